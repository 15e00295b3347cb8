// Group norm with an activation, channels last, statistics per token and group (include/ssd.h has the formulas).
//
// First form: one CTA per token and group, which reads its channels once for the mean, once for the variance (of
// the differences from the mean, not from sums of squares) and once for the output.
#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += red[i];
    return s;
}

template <typename IO>
__global__ void __launch_bounds__(kThreads) norm_kernel(NormParams p) {
    __shared__ float red[kThreads / 32];
    const int64_t gs = p.D / p.G;
    for (int64_t item = blockIdx.x; item < p.rows * p.G; item += gridDim.x) {
        const int64_t row = item / p.G, c0 = (item % p.G) * gs;
        const IO *x = static_cast<const IO *>(p.x) + row * p.x_row + c0;
        const IO *z = p.z ? static_cast<const IO *>(p.z) + row * p.z_row + c0 : nullptr;
        auto act = [&](float v) { return p.silu ? silu_f32(v) : v; };
        auto in = [&](int64_t i) {
            const float v = to_f32(x[i]);
            return p.gate_first ? v * act(to_f32(z[i])) : v;
        };
        float mean = 0.f;
        if (p.center) {
            float s = 0.f;
            for (int64_t i = threadIdx.x; i < gs; i += kThreads) s += in(i);
            mean = block_sum(s, red) / (float)gs;
        }
        float s = 0.f;
        for (int64_t i = threadIdx.x; i < gs; i += kThreads) {
            const float v = in(i) - mean;
            s = fmaf(v, v, s);
        }
        const float r = rsqrtf(block_sum(s, red) / (float)gs + p.eps);
        auto value = [&](int64_t i) {
            const int64_t c = c0 + i;
            const float v = fmaf((in(i) - mean) * r, p.w ? p.w[c] : 1.f, p.bias ? p.bias[c] : 0.f);
            return !z ? act(v) : p.gate_first ? v : v * act(to_f32(z[i]));
        };
        if (!p.scales) {
            IO *y = static_cast<IO *>(p.y) + row * p.y_row + c0;
            for (int64_t i = threadIdx.x; i < gs; i += kThreads) y[i] = from_f32<IO>(value(i));
        } else {  // a warp takes a block of 128 channels, four a lane
            uint8_t *y = static_cast<uint8_t *>(p.y) + row * p.y_row + c0;
            const int lane = threadIdx.x % 32;
            for (int64_t b = threadIdx.x / 32; b * 128 < gs; b += kThreads / 32) {
                float v[4], m = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t i = b * 128 + lane + j * 32;
                    v[j] = i < gs ? value(i) : 0.f;
                    m = max_nan(m, fabsf(v[j]));
                }
#pragma unroll
                for (int o = 16; o > 0; o /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                float scale, inv;
                e4m3_scale(m, scale, inv);
                if (lane == 0)
                    *chk(p.scales, row * ((p.D + 127) / 128) + (c0 / 128 + b), 1, p.rows * ((p.D + 127) / 128), p.hdr,
                         SITE_NORM_SCALE) = scale;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t i = b * 128 + lane + j * 32;
                    if (i < gs) y[i] = (uint8_t)e4m3x2(v[j] * inv, 0.f);
                }
            }
        }
    }
}

template <typename IO>
cudaError_t launch_t(const NormParams &p, int sms, cudaStream_t stream) {
    const int64_t grid = std::min<int64_t>(p.rows * p.G, (int64_t)sms * 64);
    norm_kernel<IO><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, int io_dtype, int sms, cudaStream_t stream) {
    if (io_dtype == SSD_F32) return launch_t<float>(p, sms, stream);
    if (io_dtype == SSD_BF16) return launch_t<__nv_bfloat16>(p, sms, stream);
    return launch_t<__half>(p, sms, stream);
}

}  // namespace ssd
