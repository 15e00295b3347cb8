// Projections in e4m3 with a scale per block of 128 (include/ssd.h has the formulas): the quantiser and the product.
//
// First form of the product: 64 x 64 tiles in shared memory, fp32 arithmetic on the CUDA cores.
#include <cuda_fp8.h>

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

constexpr int TM = 64, TN = 64, TK = 32;

__device__ __forceinline__ float from_e4m3(uint8_t v) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3)));
}

template <typename OUT>
__global__ void __launch_bounds__(256) matmul_kernel(MatmulParams p) {
    __shared__ float sa[TK][TM + 1], sb[TK][TN + 1];
    const int64_t m0 = (int64_t)blockIdx.y * TM, n0 = (int64_t)blockIdx.x * TN, kb = (p.k + 127) / 128;
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.k; k0 += TK) {
        for (int i = tid; i < TM * TK; i += 256) {
            const int r = i / TK, c = i % TK;
            const bool inA = m0 + r < p.m && k0 + c < p.k, inB = n0 + r < p.n && k0 + c < p.k;
            sa[c][r] = inA ? from_e4m3(p.a[(m0 + r) * p.k + k0 + c]) * p.sa[(m0 + r) * kb + k0 / 128] : 0.f;
            sb[c][r] = inB ? from_e4m3(p.b[(n0 + r) * p.k + k0 + c]) * p.sb[(n0 + r) / 128 * kb + k0 / 128] : 0.f;
        }
        __syncthreads();
        for (int c = 0; c < TK; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[c][ty + i * 16], sb[c][tx + j * 16], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + i * 16, n = n0 + tx + j * 16;
            if (m < p.m && n < p.n)
                *chk(static_cast<OUT *>(p.out), m * p.out_row + n, 1, (p.m - 1) * p.out_row + p.n, p.hdr,
                     SITE_FP8_OUT) = from_f32<OUT>(acc[i][j] + (p.bias ? p.bias[n] : 0.f));
        }
}

template <typename OUT>
cudaError_t launch_t(const MatmulParams &p, cudaStream_t stream) {
    const int64_t my = (p.m + TM - 1) / TM;
    for (int64_t y = 0; y < my; y += 65535) {
        MatmulParams q = p;
        q.a += y * TM * p.k;
        q.sa += y * TM * ((p.k + 127) / 128);
        q.m -= y * TM;
        q.out = static_cast<OUT *>(p.out) + y * TM * p.out_row;
        matmul_kernel<OUT><<<dim3((unsigned)((p.n + TN - 1) / TN), (unsigned)std::min<int64_t>(my - y, 65535)), 256, 0,
                             stream>>>(q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
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

cudaError_t launch_matmul(const MatmulParams &p, int out_dtype, int, cudaStream_t stream) {
    if (out_dtype == SSD_F32) return launch_t<float>(p, stream);
    if (out_dtype == SSD_BF16) return launch_t<__nv_bfloat16>(p, stream);
    return launch_t<__half>(p, stream);
}

}  // namespace ssd
