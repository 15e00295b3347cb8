// Causal depthwise convolution over the tokens by itself, rows at any stride, regular or packed sequences:
//
//   out[t, c] = act(bias[c] + sum_j w[c, j] x[t - (k - 1) + j, c]),   x before a sequence from its cache
//
// First form: one thread per token and channel, and a second kernel for the cache.
#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

// The sequence that holds packed token t: the last s with cu[s] <= t (empty sequences before it share its start).
__device__ __forceinline__ int64_t seq_of(const int32_t *cu, int64_t nseq, int64_t t) {
    int64_t lo = 0, hi = nseq - 1;
    while (lo < hi) {
        const int64_t m = (lo + hi + 1) / 2;
        if (cu[m] <= t) lo = m;
        else hi = m - 1;
    }
    return lo;
}

// Input tp (may be negative: the cache) of sequence s, whose token 0 is row `row0` of the tensor.
template <typename IO>
__device__ __forceinline__ float conv_input(const RowConvParams &p, int64_t s, int64_t seq, int64_t row0, int64_t tp,
                                            int64_t c) {
    if (tp >= 0) return to_f32(static_cast<const IO *>(p.x)[seq * p.x_seq + (row0 + tp) * p.x_tok + c]);
    if (!p.state || tp < -(p.k - 1)) return 0.f;
    return to_f32(*chk(static_cast<const IO *>(p.state), (s * p.D + c) * (p.k - 1) + (p.k - 1) + tp, 1,
                       p.nseq * p.D * (p.k - 1), p.hdr, SITE_RCONV_STATE));
}

template <typename IO>
__global__ void __launch_bounds__(kThreads) row_conv_kernel(RowConvParams p) {
    if (p.cu && blockIdx.x == 0) check_offsets(p.cu, p.nseq, p.T, p.hdr);
    const int64_t total = p.T * p.D;
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < total; e += (int64_t)gridDim.x * kThreads) {
        const int64_t c = e % p.D, tok = e / p.D;
        int64_t s, seq, row0;
        if (p.cu) {
            s = seq_of(p.cu, p.nseq, tok);
            seq = 0;
            int64_t end;
            packed_range(p.cu, s, p.T, row0, end);
            if (tok < row0) row0 = tok;  // malformed offsets
        } else {
            s = seq = tok / p.L;
            row0 = 0;
        }
        const int64_t t = p.cu ? tok - row0 : tok % p.L;
        float acc = p.bias ? p.bias[c] : 0.f;
        for (int j = 0; j < p.k; ++j)
            acc = fmaf(p.w[c * p.k + j], conv_input<IO>(p, s, seq, row0, t - (p.k - 1) + j, c), acc);
        if (p.silu) acc = silu_f32(acc);
        static_cast<IO *>(p.out)[seq * p.out_seq + (row0 + t) * p.out_tok + c] = from_f32<IO>(acc);
    }
}

// The last k - 1 inputs of every sequence. A thread owns a (sequence, channel): its old entries are read before any
// is written, so the cache may be updated in place.
template <typename IO>
__global__ void __launch_bounds__(kThreads) row_conv_state_kernel(RowConvParams p) {
    const int64_t total = p.nseq * p.D;
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < total; e += (int64_t)gridDim.x * kThreads) {
        const int64_t s = e / p.D, c = e % p.D;
        int64_t row0 = 0, end = p.L;
        if (p.cu) packed_range(p.cu, s, p.T, row0, end);
        float v[7];
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < p.k - 1) v[j] = conv_input<IO>(p, s, p.cu ? 0 : s, row0, end - row0 - (p.k - 1) + j, c);
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < p.k - 1)
                *chk(static_cast<IO *>(p.state_out), e * (p.k - 1) + j, 1, total * (p.k - 1), p.hdr,
                     SITE_RCONV_STATE) = from_f32<IO>(v[j]);
    }
}

template <typename IO>
cudaError_t launch_t(const RowConvParams &p, int sms, cudaStream_t stream) {
    if (p.T > 0) {
        const int64_t grid = std::min<int64_t>((p.T * p.D + kThreads - 1) / kThreads, (int64_t)sms * 64);
        row_conv_kernel<IO><<<(unsigned)grid, kThreads, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (p.state_out && p.k > 1) {
        const int64_t grid = std::min<int64_t>((p.nseq * p.D + kThreads - 1) / kThreads, (int64_t)sms * 64);
        row_conv_state_kernel<IO><<<(unsigned)grid, kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_row_conv(const RowConvParams &p, int io_dtype, int sms, cudaStream_t stream) {
    if (io_dtype == SSD_F32) return launch_t<float>(p, sms, stream);
    if (io_dtype == SSD_BF16) return launch_t<__nv_bfloat16>(p, sms, stream);
    return launch_t<__half>(p, sms, stream);
}

}  // namespace ssd
