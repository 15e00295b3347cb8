// Selective scan, f32 tensors (ssd_selscan.cuh).
#include "ssd_selscan.cuh"

namespace ssd {
cudaError_t launch_scan_f32(const ScanParams &p, cudaStream_t stream) { return scan::launch_io<float>(p, stream); }
}  // namespace ssd
