// Group norm, f32 tensors (ssd_norm.cuh).
#include "ssd_norm.cuh"

namespace ssd {
cudaError_t launch_norm_f32(const NormParams &p, int sms, cudaStream_t stream) { return norm::launch_io<float>(p, sms, stream); }
}  // namespace ssd
