// Selective scan, bf16 tensors (ssd_selscan.cuh).
#include "ssd_selscan.cuh"

namespace ssd {
cudaError_t launch_scan_bf16(const ScanParams &p, cudaStream_t stream) { return scan::launch_io<__nv_bfloat16>(p, stream); }
}  // namespace ssd
