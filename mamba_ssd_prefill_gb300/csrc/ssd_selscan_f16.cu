// Selective scan, f16 tensors (ssd_selscan.cuh).
#include "ssd_selscan.cuh"

namespace ssd {
cudaError_t launch_scan_f16(const ScanParams &p, cudaStream_t stream) { return scan::launch_io<__half>(p, stream); }
}  // namespace ssd
