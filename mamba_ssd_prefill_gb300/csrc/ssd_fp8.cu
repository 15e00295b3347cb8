// The quantiser of the e4m3 projections: one scale per block of 128 columns and one row (activations) or 128 rows
// (weights); include/ssd.h has the formulas.
#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace {

// One warp per block of block_rows x 128 elements.
template <typename IO>
__global__ void __launch_bounds__(256) quantize_kernel(QuantParams p) {
    const int lane = threadIdx.x % 32;
    const int64_t kb = (p.cols + 127) / 128, rb = (p.rows + p.block_rows - 1) / p.block_rows;
    const IO *x = static_cast<const IO *>(p.x);
    for (int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; w < rb * kb; w += (int64_t)gridDim.x * 8) {
        const int64_t r0 = w / kb * p.block_rows, c0 = w % kb * 128;
        const int64_t r1 = r0 + p.block_rows < p.rows ? r0 + p.block_rows : p.rows;
        const int n = (int)(p.cols - c0 < 128 ? p.cols - c0 : 128);
        float m = 0.f;
        for (int64_t r = r0; r < r1; ++r)
            for (int i = lane; i < n; i += 32) m = max_nan(m, fabsf(to_f32(x[r * p.x_row + c0 + i])));
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        float scale, inv;
        e4m3_scale(m, scale, inv);
        if (lane == 0) *chk(p.scales, w, 1, rb * kb, p.hdr, SITE_FP8_SCALE) = scale;
        for (int64_t r = r0; r < r1; ++r)
            for (int i = lane; i < n; i += 32)
                *chk(p.q, r * p.cols + c0 + i, 1, p.rows * p.cols, p.hdr, SITE_FP8_OUT) =
                    (uint8_t)e4m3x2(to_f32(x[r * p.x_row + c0 + i]) * inv, 0.f);
    }
}

}  // namespace

cudaError_t launch_quantize(const QuantParams &p, int io_dtype, int sms, cudaStream_t stream) {
    const int64_t blocks = (p.rows + p.block_rows - 1) / p.block_rows * ((p.cols + 127) / 128);
    const int64_t grid = std::min<int64_t>((blocks + 7) / 8, (int64_t)sms * 64);
    if (io_dtype == SSD_F32)
        quantize_kernel<float><<<(unsigned)grid, 256, 0, stream>>>(p);
    else if (io_dtype == SSD_BF16)
        quantize_kernel<__nv_bfloat16><<<(unsigned)grid, 256, 0, stream>>>(p);
    else
        quantize_kernel<__half><<<(unsigned)grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace ssd
