// Group norm, f16 tensors (ssd_norm.cuh).
#include "ssd_norm.cuh"

namespace ssd {
cudaError_t launch_norm_f16(const NormParams &p, int sms, cudaStream_t stream) { return norm::launch_io<__half>(p, sms, stream); }
}  // namespace ssd
