// Group norm, bf16 tensors (ssd_norm.cuh).
#include "ssd_norm.cuh"

namespace ssd {
cudaError_t launch_norm_bf16(const NormParams &p, int sms, cudaStream_t stream) { return norm::launch_io<__nv_bfloat16>(p, sms, stream); }
}  // namespace ssd
