// The quantiser of the e4m3 projections: one scale per block of 128 columns and one row (activations) or 128 rows
// (weights); include/ssd.h has the formulas. HBM-bound: with rows of 8-element pieces 16 lanes hold a block of one row
// in registers from its one read to its write (16384 x 2560 bf16: 26 us, 4.8 TB/s). Weights, quantised once, and other rows
// are read twice, an element a lane (10576 x 2560: fp32 319 us, bf16 193; rows of 2561 bf16 elements 105).
#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace {

// One warp per block of block_rows x 128 elements.
template <typename IO>
__global__ void __launch_bounds__(256) quantize_kernel(QuantParams p) {
    after_previous();
    const int lane = threadIdx.x % 32;
    const int64_t kb = (p.cols + 127) / 128, rb = (p.rows + p.block_rows - 1) / p.block_rows;
    const int64_t xn = (p.rows - 1) * p.x_row + p.cols;
    (void)xn;
    for (int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; w < rb * kb; w += (int64_t)gridDim.x * 8) {
        const int64_t r0 = w / kb * p.block_rows, c0 = w % kb * 128;
        const int64_t r1 = r0 + p.block_rows < p.rows ? r0 + p.block_rows : p.rows;
        const int n = (int)(p.cols - c0 < 128 ? p.cols - c0 : 128);
        const IO *x = chk_rows(static_cast<const IO *>(p.x), r0 * p.x_row + c0, r1 - r0, p.x_row, n, xn, p.hdr, SITE_FP8_IN);
        float m = 0.f;
        for (int64_t r = r0; r < r1; ++r)
            for (int i = lane; i < n; i += 32) m = max_nan(m, fabsf(to_f32(x[(r - r0) * p.x_row + i])));
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        float scale, inv;
        e4m3_scale(m, scale, inv);
        if (lane == 0) *chk(p.scales, w, 1, rb * kb, p.hdr, SITE_FP8_SCALE) = scale;
        for (int64_t r = r0; r < r1; ++r)
            for (int i = lane; i < n; i += 32)
                *chk(p.q, r * p.cols + c0 + i, 1, p.rows * p.cols, p.hdr, SITE_FP8_OUT) =
                    (uint8_t)e4m3x2(to_f32(x[(r - r0) * p.x_row + i]) * inv, 0.f);
    }
}

// block_rows = 1, rows of 8-element pieces: a half-warp per block, N blocks each, all loaded before the first is written.
template <typename IO, int N>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantParams p) {
    const int lane = threadIdx.x % 16;
    const int64_t kb = (p.cols + 127) / 128, blocks = p.rows * kb;
    const int64_t b0 = ((int64_t)blockIdx.x * 16 + threadIdx.x / 16) * N;
    const IO *x = static_cast<const IO *>(p.x);
    const int64_t xn = (p.rows - 1) * p.x_row + p.cols;
    (void)xn;
    after_previous();
    Raw<IO, 8> r[N];
    int64_t col0, row0 = quick_div(b0, kb, col0), row = row0, col = col0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t c = col * 128 + lane * 8;
        if (b0 + i < blocks && c < p.cols) r[i].load(chk(x, row * p.x_row + c, 8, xn, p.hdr, SITE_FP8_IN));
        else r[i].zero();
        if (++col == kb) col = 0, ++row;
    }
    row = row0, col = col0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t c = col * 128 + lane * 8;
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max_nan(m, fabsf(r[i].get(k)));
#pragma unroll
        for (int d = 8; d > 0; d /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
        float scale, inv;
        e4m3_scale(m, scale, inv);
        if (b0 + i < blocks) {
            if (lane == 0) *chk(p.scales, b0 + i, 1, blocks, p.hdr, SITE_FP8_SCALE) = scale;
            if (c < p.cols) {
                uint32_t q[2];
#pragma unroll
                for (int k = 0; k < 8; k += 4)
                    q[k / 4] = (uint32_t)e4m3x2(r[i].get(k) * inv, r[i].get(k + 1) * inv) |
                               (uint32_t)e4m3x2(r[i].get(k + 2) * inv, r[i].get(k + 3) * inv) << 16;
                *reinterpret_cast<uint2 *>(chk(p.q, row * p.cols + c, 8, p.rows * p.cols, p.hdr, SITE_FP8_OUT)) =
                    make_uint2(q[0], q[1]);
            }
        }
        if (++col == kb) col = 0, ++row;
    }
}

template <typename IO> cudaError_t launch_t(const QuantParams &p, int sms, cudaStream_t stream) {
    const int64_t blocks = (p.rows + p.block_rows - 1) / p.block_rows * ((p.cols + 127) / 128);
    if (p.block_rows == 1 && p.vec) {
        if (blocks < (int64_t)sms * 64) {  // few blocks: one a half-warp
            return launch_after(quantize_rows_kernel<IO, 1>, (blocks + 15) / 16, 256, 0, stream, p);
        }
        const int64_t grid = (blocks + 63) / 64;
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        return launch_after(quantize_rows_kernel<IO, 4>, grid, 256, 0, stream, p);
    }
    const int64_t grid = std::min<int64_t>((blocks + 7) / 8, (int64_t)sms * 64);
    return launch_after(quantize_kernel<IO>, grid, 256, 0, stream, p);
}

}  // namespace

cudaError_t launch_quantize(const QuantParams &p, int io_dtype, int sms, cudaStream_t stream) {
    if (io_dtype == SSD_F32) return launch_t<float>(p, sms, stream);
    if (io_dtype == SSD_BF16) return launch_t<__nv_bfloat16>(p, sms, stream);
    return launch_t<__half>(p, sms, stream);
}

}  // namespace ssd
