// Selective scan ("Mamba hardware-aware algorithms", fused selective scan: discretise, scan and contract with C in
// one kernel): per sequence and channel c, with dt = softplus(dt_raw + dt_bias),
//
//   h[n] <- exp(dt A[c, n]) h[n] + dt x[c] B[n],     y[c] = (sum_n C[n] h[n] + D[c] x[c]) z[c] sigmoid(z[c])
//
// First form: S lanes hold the states of a channel, four each, in registers, and walk the tokens.
#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

template <typename IO, typename ST, int S, int R>
__global__ void __launch_bounds__(kThreads) scan_kernel(ScanParams p) {
    constexpr int CT = kThreads / S;  // channels per CTA
    const int64_t ctiles = (p.D_ + CT - 1) / CT;
    const int64_t sq = blockIdx.x / ctiles, c = (blockIdx.x % ctiles) * CT + threadIdx.x / S;
    const int n0 = (threadIdx.x % S) * R;
    if (p.cu && blockIdx.x == 0) check_offsets(p.cu, p.nseq, p.T, p.hdr);
    int64_t t0 = 0, t1 = p.L;
    if (p.cu) packed_range(p.cu, sq, p.T, t0, t1);
    const int64_t seq = p.cu ? 0 : sq;
    const bool live = c < p.D_;
    const int64_t cc = live ? c : 0, g = cc / p.cpg;
    const IO *x = static_cast<const IO *>(p.x) + seq * p.x_seq + cc;
    const IO *dt = static_cast<const IO *>(p.dt) + seq * p.dt_seq + cc;
    const IO *z = static_cast<const IO *>(p.z) + (p.z ? seq * p.z_seq + cc : 0);
    const IO *B = static_cast<const IO *>(p.B) + seq * p.b_seq + g * p.N;
    const IO *C = static_cast<const IO *>(p.C) + seq * p.c_seq + g * p.N;
    IO *y = static_cast<IO *>(p.y) + seq * p.y_seq + cc;
    float a[R], h[R];
    const int64_t s0 = (sq * p.D_ + cc) * p.N;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool in = n0 + i < p.N;
        a[i] = in ? p.A[cc * p.N + n0 + i] * kLog2e : 0.f;
        h[i] = in && p.init ? to_f32(*chk(static_cast<const ST *>(p.init), s0 + n0 + i, 1, p.nseq * p.D_ * p.N, p.hdr,
                                          SITE_SCAN_STATE))
                            : 0.f;
    }
    const float bias = p.dt_bias ? p.dt_bias[cc] : 0.f, Dc = p.D ? p.D[cc] : 0.f;
    for (int64_t t = t0; t < t1; ++t) {
        const float xv = to_f32(x[t * p.x_tok]);
        float d = to_f32(dt[t * p.dt_tok]) + bias;
        if (p.softplus) d = softplus_fast(d);
        const float u = d * xv;
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t n = n0 + i < p.N ? n0 + i : 0;
            const float b = n0 + i < p.N ? to_f32(B[t * p.b_tok + n]) : 0.f;
            const float cv = n0 + i < p.N ? to_f32(C[t * p.c_tok + n]) : 0.f;
            h[i] = fmaf(ex2(d * a[i]), h[i], u * b);
            acc = fmaf(h[i], cv, acc);
        }
#pragma unroll
        for (int o = S / 2; o > 0; o /= 2) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (live && threadIdx.x % S == 0) {
            float v = fmaf(Dc, xv, acc);
            if (p.z) v *= silu_f32(to_f32(z[t * p.z_tok]));
            y[t * p.y_tok] = from_f32<IO>(v);
        }
    }
    if (live && p.fin)
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (n0 + i < p.N)
                *chk(static_cast<ST *>(p.fin), s0 + n0 + i, 1, p.nseq * p.D_ * p.N, p.hdr, SITE_SCAN_STATE) =
                    from_f32<ST>(h[i]);
}

template <typename IO, typename ST, int S, int R>
cudaError_t launch_s(const ScanParams &p, cudaStream_t stream) {
    constexpr int CT = kThreads / S;
    const int64_t grid = (p.D_ + CT - 1) / CT * p.nseq;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    scan_kernel<IO, ST, S, R><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename IO, typename ST>
cudaError_t launch_n(const ScanParams &p, cudaStream_t stream) {
    if (p.N <= 4) return launch_s<IO, ST, 1, 4>(p, stream);
    if (p.N <= 16) return launch_s<IO, ST, 4, 4>(p, stream);
    if (p.N <= 64) return launch_s<IO, ST, 16, 4>(p, stream);
    return launch_s<IO, ST, 32, 8>(p, stream);
}
template <typename IO>
cudaError_t launch_st(const ScanParams &p, int state_dtype, cudaStream_t stream) {
    return state_dtype == SSD_F32 ? launch_n<IO, float>(p, stream) : launch_n<IO, __half>(p, stream);
}

}  // namespace

cudaError_t launch_scan(const ScanParams &p, int io_dtype, int state_dtype, int, cudaStream_t stream) {
    if (io_dtype == SSD_F32) return launch_st<float>(p, state_dtype, stream);
    if (io_dtype == SSD_BF16) return launch_st<__nv_bfloat16>(p, state_dtype, stream);
    return launch_st<__half>(p, state_dtype, stream);
}

}  // namespace ssd
