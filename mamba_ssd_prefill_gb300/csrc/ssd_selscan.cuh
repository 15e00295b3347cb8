// Selective scan ("Mamba hardware-aware algorithms", fused selective scan: discretise, scan and contract with C in
// one kernel): per sequence and channel c, with dt = softplus(dt_raw + dt_bias),
//
//   h[n] <- exp(dt A[c, n]) h[n] + dt x[c] B[n],     y[c] = (sum_n C[n] h[n] + D[c] x[c]) z[c] sigmoid(z[c])
//
// Every (token, channel, state) costs one exponential and five flops, against 8 bytes per (token, channel) in 16-bit
// types: at 16 states the special-function and issue rates bound it, not HBM. So the states stay in registers and the
// work per element is kept to the recurrence itself:
//
//  - A CTA owns CT channels (of one group) and walks tokens in tiles of TT. A tile's x, dt, z, B and C are loaded to
//    registers one tile ahead (16 bytes a thread and tensor), and turned into shared memory once: (dt, dt, dt x, dt x)
//    per token and channel, ready for packed fp32 pairs, B and C in fp32. The step's softplus is so taken once per
//    (token, channel), not once per state.
//  - S lanes share a channel, R states each, in packed pairs (f32x2): per pair one multiply for the exponent, two
//    exponentials, one multiply for dt x B, one fused multiply-add for h, one for y.
//  - The sum over a channel's lanes is taken for TG tokens at once, each shuffle halving the tokens a lane holds, so
//    that S - 1 shuffles serve S tokens.
//
// Where (sequences x channel tiles) do not fill the GPU, the tokens are cut into segments: scan_kernel<SUM> first
// computes every segment's leaving state from a zero state and its summed dt (the state's decay over a segment is
// exp(A sum dt), exactly), and each segment of the main pass folds the segments before it. That costs the state part
// of the work twice. Packed sequences are segmented on the packed axis, whatever their lengths; a segment restarts
// its chain wherever a sequence begins inside it.
#pragma once

#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace scan {

typedef unsigned long long f2;  // two packed fp32

__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ float load_state(const ScanParams &p, const void *s, int64_t i) {
    const int64_t n = p.nseq * p.D_ * p.N;
    return p.state_f16 ? to_f32(*chk(static_cast<const __half *>(s), i, 1, n, p.hdr, SITE_SCAN_STATE))
                       : *chk(static_cast<const float *>(s), i, 1, n, p.hdr, SITE_SCAN_STATE);
}
__device__ __forceinline__ void store_state(const ScanParams &p, void *s, int64_t i, float v) {
    const int64_t n = p.nseq * p.D_ * p.N;
    if (p.state_f16) *chk(static_cast<__half *>(s), i, 1, n, p.hdr, SITE_SCAN_STATE) = __float2half_rn(v);
    else *chk(static_cast<float *>(s), i, 1, n, p.hdr, SITE_SCAN_STATE) = v;
}

// K consecutive elements as they lie, in registers
template <typename IO, int K> struct Raw {
    static constexpr int W = K * (int)sizeof(IO) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    // all K elements; p is aligned for them
    __device__ __forceinline__ void load(const IO *p) {
        if constexpr (W == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        }
    }
    // the first n of K elements (the others zero); vec: p is aligned for K elements
    __device__ __forceinline__ void load(const IO *p, int n, bool vec) {
        if (vec && n >= K) {
            load(p);
        } else {
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const uint32_t b = i < n ? bits(p[i]) : 0;
                if constexpr (sizeof(IO) == 4) w[i] = b;
                else if (i % 2 == 0) w[i / 2] = b;
                else w[i / 2] |= b << 16;
            }
        }
    }
    static __device__ __forceinline__ uint32_t bits(IO v) {
        if constexpr (sizeof(IO) == 4) return __float_as_uint(v);
        else return *reinterpret_cast<const uint16_t *>(&v);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(IO) == 4) {
            return __uint_as_float(w[i]);
        } else {
            const uint16_t h = (uint16_t)(i % 2 ? w[i / 2] >> 16 : w[i / 2]);
            return to_f32(*reinterpret_cast<const IO *>(&h));
        }
    }
};

// v[0 .. TG) of each of a channel's S lanes -> the total of item q TG / S, q the lane's place among them.
template <int S, int TG> __device__ __forceinline__ float reduce_lanes(float (&v)[TG], int q) {
    int m = TG;
#pragma unroll
    for (int o = S / 2; o > 0; o /= 2) {
        if (m > 1) {
            m /= 2;
            const bool upper = q & o;
#pragma unroll
            for (int i = 0; i < TG / 2; ++i)
                if (i < m) {
                    const float send = upper ? v[i] : v[i + m], keep = upper ? v[i + m] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return v[0];
}

// The last sequence whose start is at or before packed token t (empty ones before it share its start).
__device__ __forceinline__ int64_t seq_at(const int32_t *cu, int64_t nseq, int64_t t) {
    int64_t lo = 0, hi = nseq - 1;
    while (lo < hi) {
        const int64_t m = (lo + hi + 1) / 2;
        if (cu[m] <= t) lo = m;
        else hi = m - 1;
    }
    return lo;
}

template <int S_, int R_, int NT_, int TT_> struct Shape {
    static constexpr int S = S_, R = R_, NT = NT_, TT = TT_;
    static constexpr int CT = NT / S, NP = S * R, TG = S < 8 ? S : 8, CV = CT / 8;
    static constexpr int VPT = (TT * CV + NT - 1) / NT;         // vectors of 8 channels a thread loads per tensor
    static constexpr int NV = NP / 4;                           // vectors of 4 states per token
    static constexpr int YS = CT + 8;                           // row of y: tokens of a reduction on different banks
    static constexpr size_t smem(bool sum) {
        return (size_t)TT * CT * 16 + (size_t)TT * NP * 4 * (sum ? 1 : 2) + (sum ? 0 : (size_t)TT * YS * 4) + CT * 8;
    }
};

template <typename IO, typename T, bool SUM>
__global__ void __launch_bounds__(T::NT) scan_kernel(ScanParams p) {
    constexpr int S = T::S, R = T::R, NT = T::NT, TT = T::TT, CT = T::CT, NP = T::NP, TG = T::TG, CV = T::CV,
                  VPT = T::VPT, NV = T::NV, YS = T::YS;
    constexpr int BPT = (TT * NV * (SUM ? 1 : 2) + NT - 1) / NT;
    extern __shared__ __align__(16) uint8_t smem[];
    ulonglong2 *du = reinterpret_cast<ulonglong2 *>(smem);                 // [TT][CT] (dt, dt, dt x, dt x)
    float *Bs = reinterpret_cast<float *>(smem + (size_t)TT * CT * 16);    // [TT][NP]
    float *Cs = Bs + TT * NP;                                              // [TT][NP], not for SUM
    float *ys = SUM ? Cs : Cs + TT * NP;                                   // [TT][YS], not for SUM
    float *bias_s = SUM ? ys : ys + TT * YS, *D_s = bias_s + CT;           // [CT] each
    const int tid = threadIdx.x;
    const int64_t per_group = (p.cpg + CT - 1) / CT, ctiles = per_group * p.G;
    const int64_t item = blockIdx.x / ctiles, ct = blockIdx.x % ctiles, g = ct / per_group;
    const int64_t c0 = g * p.cpg + ct % per_group * CT;                    // first channel
    const int64_t left = (g + 1) * p.cpg - c0;                             // channels of the group from c0 on
    const int ch = tid / S, q = tid % S;                                   // this lane's channel and place
    const bool live = ch < left;
    const bool packed = p.cu != nullptr;

    // tokens [t0, t1) of sequence `sq` (packed: of the packed axis, sq the sequence that holds t0)
    int64_t sq, k, t0, t1, qe = 0;
    const int64_t nseg = SUM ? p.nseg - 1 : p.nseg;  // the last segment's leaving state is not needed
    bool fresh;                                      // the chain begins from a sequence's initial state
    if (packed) {
        k = item;
        t0 = k * p.seg_len;
        t1 = t0 + p.seg_len < p.T ? t0 + p.seg_len : p.T;
        int64_t qb;
        sq = seq_at(p.cu, p.nseq, SUM ? t1 - 1 : t0);
        packed_range(p.cu, sq, p.T, qb, qe);
        if (SUM) {
            if (qe <= t1) return;  // no sequence goes on past this segment
            fresh = qb >= t0;
            if (fresh) t0 = qb < t1 ? qb : t1;
        } else {
            fresh = qb >= t0;
            if (qe <= t0) qe = p.T;  // malformed offsets
            if (item == 0 && ct == 0) check_offsets(p.cu, p.nseq, p.T, p.hdr);
            if (p.fin)  // empty sequences keep their states; each segment's CTAs look after some of them
                for (int64_t s = item; s < p.nseq; s += p.nseg)
                    if (p.cu[s] == p.cu[s + 1])
                        for (int64_t e = tid; e < CT * p.N; e += NT)
                            if (e / p.N < left) {
                                const int64_t i = (s * p.D_ + c0) * p.N + e;
                                store_state(p, p.fin, i, p.init ? load_state(p, p.init, i) : 0.f);
                            }
        }
    } else {
        sq = item / nseg;
        k = item % nseg;
        t0 = k * p.seg_len;
        t1 = t0 + p.seg_len < p.L ? t0 + p.seg_len : p.L;
        fresh = k == 0;
    }
    const int64_t row = packed ? 0 : sq;  // leading index of the token tensors
    const IO *x = static_cast<const IO *>(p.x) + row * p.x_seq + c0;
    const IO *dt = static_cast<const IO *>(p.dt) + row * p.dt_seq + c0;
    const IO *z = SUM || !p.z ? nullptr : static_cast<const IO *>(p.z) + row * p.z_seq + c0;
    const IO *B = static_cast<const IO *>(p.B) + row * p.b_seq + g * p.N;
    const IO *C = static_cast<const IO *>(p.C) + row * p.c_seq + g * p.N;

    for (int i = tid; i < CT; i += NT) {
        bias_s[i] = p.dt_bias && i < left ? p.dt_bias[c0 + i] : 0.f;
        D_s[i] = p.D && i < left ? p.D[c0 + i] : 0.f;
    }

    f2 a[R / 2], h[R / 2];
    const int64_t cN = (c0 + (live ? ch : 0)) * p.N;
    const int n0 = q * R;
    auto get2 = [&](auto f) {  // f(n) for this lane's states, 0 past the last and for missing channels
#pragma unroll
        for (int i = 0; i < R / 2; ++i) {
            const int n = n0 + 2 * i;
            h[i] = pack2(live && n < p.N ? f(n) : 0.f, live && n + 1 < p.N ? f(n + 1) : 0.f);
        }
    };
    get2([&](int n) { return p.A[cN + n] * kLog2e; });
#pragma unroll
    for (int i = 0; i < R / 2; ++i) a[i] = h[i];
    auto initial = [&](int64_t s) {
        get2([&](int n) { return p.init ? load_state(p, p.init, s * p.D_ * p.N + cN + n) : 0.f; });
    };
    auto final_state = [&](int64_t s) {
        if (p.fin && live)
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                const int n = n0 + 2 * i;
                const float2 v = unpack2(h[i]);
                if (n < p.N) store_state(p, p.fin, s * p.D_ * p.N + cN + n, v.x);
                if (n + 1 < p.N) store_state(p, p.fin, s * p.D_ * p.N + cN + n + 1, v.y);
            }
    };
    if (fresh) {
        initial(sq);
    } else if (SUM) {
        get2([](int) { return 0.f; });
    } else {  // the segments before, from the one in which the sequence began
        int64_t j = 0, first = sq * (p.nseg - 1);
        if (packed) {
            int64_t qb, e;
            packed_range(p.cu, sq, p.T, qb, e);
            j = qb / p.seg_len;
            first = 0;
        }
        const int64_t extent = p.seg_items * p.D_ * p.N;
        auto leaving = [&](int64_t i, int n) {
            return *chk(p.seg_state, (first + i) * p.D_ * p.N + cN + n, 1, extent, p.hdr, SITE_SCAN_SEG);
        };
        get2([&](int n) { return leaving(j, n); });
        for (++j; j < k; ++j) {
            const float d = live ? p.seg_dt[(first + j) * p.D_ + c0 + ch] : 0.f;
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                const int n = n0 + 2 * i;
                const float2 e = unpack2(mul2(a[i], pack2(d, d)));
                h[i] = fma2(pack2(ex2(e.x), ex2(e.y)), h[i],
                            pack2(live && n < p.N ? leaving(j, n) : 0.f, live && n + 1 < p.N ? leaving(j, n + 1) : 0.f));
            }
        }
    }

    // loads of one tile: 8 channels of a token per vector, and 4 states of a token of B or C
    const int cv = tid % CV, trow = tid / CV;             // channel vector and first token of this thread
    const int clive = (int)(left - cv * 8 < 0 ? 0 : left - cv * 8 < 8 ? left - cv * 8 : 8);
    Raw<IO, 8> rx[VPT], rd[VPT], rz[VPT];
    Raw<IO, 4> rb[BPT];
    const int64_t xn = (p.rows - 1) * p.x_seq + (p.L - 1) * p.x_tok + p.D_;
    const int64_t dn = (p.rows - 1) * p.dt_seq + (p.L - 1) * p.dt_tok + p.D_;
    const int64_t zn = (p.rows - 1) * p.z_seq + (p.L - 1) * p.z_tok + p.D_;
    const int64_t yn = (p.rows - 1) * p.y_seq + (p.L - 1) * p.y_tok + p.D_;
    const int64_t bn = (p.rows - 1) * p.b_seq + (p.L - 1) * p.b_tok + p.G * p.N;
    const int64_t cn = (p.rows - 1) * p.c_seq + (p.L - 1) * p.c_tok + p.G * p.N;
    (void)xn, (void)dn, (void)zn, (void)yn, (void)bn, (void)cn;
    auto at = [&](const IO *base, const void *whole, int64_t off, int n, int64_t extent) {
        const IO *w = static_cast<const IO *>(whole);
        return (const IO *)chk(w, base + off - w, n, extent, p.hdr, SITE_SCAN_IN);
    };
    auto load = [&](int64_t tile) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int t = trow + v * (NT / CV);
            rx[v].zero();
            rd[v].zero();
            rz[v].zero();
            if ((TT * CV % NT == 0 || t < TT) && tile + t < t1 && clive > 0) {
                const int64_t tk = tile + t;
                rx[v].load(at(x, p.x, tk * p.x_tok + cv * 8, clive, xn), clive, p.vec);
                rd[v].load(at(dt, p.dt, tk * p.dt_tok + cv * 8, clive, dn), clive, p.vec);
                if (!SUM && z) rz[v].load(at(z, p.z, tk * p.z_tok + cv * 8, clive, zn), clive, p.vec);
            }
        }
#pragma unroll
        for (int v = 0; v < BPT; ++v) {
            const int e = tid + v * NT, t = e / NV % TT, n = e % NV * 4, nl = (int)(p.N - n);
            rb[v].zero();
            if (e < TT * NV * (SUM ? 1 : 2) && tile + t < t1 && nl > 0) {
                const int64_t tk = tile + t;
                if (SUM || e < TT * NV) rb[v].load(at(B, p.B, tk * p.b_tok + n, nl < 4 ? nl : 4, bn), nl, p.vec_bc);
                else rb[v].load(at(C, p.C, tk * p.c_tok + n, nl < 4 ? nl : 4, cn), nl, p.vec_bc);
            }
        }
    };
    // slot of a channel in a row of du: 8-channel vectors written by different threads fall on different banks
    auto slot = [](int c) { return (c & ~7) | ((c ^ (c >> 3)) & 7); };
    const int my_slot = slot(ch);
    float dt_sum = 0.f;

    // tokens [lo, hi) of the tile in shared memory; MASK: other tokens of the groups of TG leave the state alone
    auto run = [&](auto mask, int lo, int hi) {
        constexpr bool MASK = decltype(mask)::value;
        float part_dt = 0.f;
#pragma unroll 2
        for (int g0 = lo / TG * TG; g0 < hi; g0 += TG) {
            float v[TG];
#pragma unroll
            for (int i = 0; i < TG; ++i) {
                const int t = g0 + i;
                const bool in = !MASK || (t >= lo && t < hi);
                const ulonglong2 d = du[t * CT + my_slot];
                const ulonglong2 *b = reinterpret_cast<const ulonglong2 *>(Bs + t * NP + n0);
                const ulonglong2 *c = reinterpret_cast<const ulonglong2 *>(Cs + t * NP + n0);
                f2 y = 0;
#pragma unroll
                for (int j = 0; j < R / 4; ++j) {
                    const ulonglong2 bb = b[j];
                    const float2 e0 = unpack2(mul2(d.x, a[2 * j])), e1 = unpack2(mul2(d.x, a[2 * j + 1]));
                    const f2 h0 = fma2(pack2(ex2(e0.x), ex2(e0.y)), h[2 * j], mul2(d.y, bb.x));
                    const f2 h1 = fma2(pack2(ex2(e1.x), ex2(e1.y)), h[2 * j + 1], mul2(d.y, bb.y));
                    h[2 * j] = in ? h0 : h[2 * j];
                    h[2 * j + 1] = in ? h1 : h[2 * j + 1];
                    if (!SUM) {
                        const ulonglong2 cc = c[j];
                        y = j == 0 ? mul2(h[0], cc.x) : fma2(h[2 * j], cc.x, y);
                        y = fma2(h[2 * j + 1], cc.y, y);
                    }
                }
                if (SUM) part_dt += in ? unpack2(d.x).x : 0.f;
                const float2 yy = unpack2(y);
                v[i] = yy.x + yy.y;
            }
            if (!SUM) {
                const float total = reduce_lanes<S, TG>(v, q);
                const int t = g0 + q * TG / S;
                if ((S <= TG || q % (S / TG) == 0) && (!MASK || (t >= lo && t < hi))) ys[t * YS + ch] = total;
            }
        }
        dt_sum += part_dt;
    };

    load(t0);
    for (int64_t tile = t0; tile < t1; tile += TT) {
        const int n = (int)(t1 - tile < TT ? t1 - tile : TT);
        if (tile == t0) __syncthreads();  // bias_s and D_s
        // (dt, dt, dt x, dt x); tokens past the end: a decay of 1 and nothing added
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int t = trow + v * (NT / CV);
            if (TT * CV % NT == 0 || t < TT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float d = rd[v].get(i) + bias_s[cv * 8 + i];
                    if (p.softplus) d = softplus_fast(d);
                    if (t >= n) d = 0.f;
                    const float u = d * rx[v].get(i);
                    du[t * CT + slot(cv * 8 + i)] = make_ulonglong2(pack2(d, d), pack2(u, u));
                }
            }
        }
#pragma unroll
        for (int v = 0; v < BPT; ++v) {
            const int e = tid + v * NT;
            if (TT * NV * (SUM ? 1 : 2) % NT == 0 || e < TT * NV * (SUM ? 1 : 2))
                *reinterpret_cast<float4 *>(Bs + e * 4) =  // C follows B
                    make_float4(rb[v].get(0), rb[v].get(1), rb[v].get(2), rb[v].get(3));
        }
        Raw<IO, 8> cx[VPT], cz[VPT];  // this tile's x and z, for its output
#pragma unroll
        for (int v = 0; v < VPT; ++v) cx[v] = rx[v], cz[v] = rz[v];
        if (tile + TT < t1) load(tile + TT);
        __syncthreads();
        if (SUM || !packed || qe > tile + n) {
            run(std::integral_constant<bool, false>(), 0, TT);
        } else {  // sequences end in this tile
            int pos = 0;
            while (pos < n) {
                const int e = qe - tile < n ? (int)(qe - tile) : n;
                run(std::integral_constant<bool, true>(), pos, e);
                pos = e;
                if (tile + e == qe) {
                    final_state(sq);
                    int64_t qb = 0;
                    do {
                        if (++sq >= p.nseq) break;
                        packed_range(p.cu, sq, p.T, qb, qe);
                    } while (qe <= tile + e);
                    if (sq >= p.nseq) {  // the end, or malformed offsets
                        sq = p.nseq - 1;
                        qe = p.T + 1;
                        if (tile + e >= p.T) break;
                    }
                    initial(sq);
                }
            }
        }
        __syncthreads();
        if (!SUM) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int t = trow + v * (NT / CV);
                if (t < n && clive > 0) {
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[i] = fmaf(D_s[cv * 8 + i], cx[v].get(i), ys[t * YS + cv * 8 + i]);
                        if (z) o[i] *= silu_f32(cz[v].get(i));
                    }
                    IO *out = chk(static_cast<IO *>(p.y), row * p.y_seq + (tile + t) * p.y_tok + c0 + cv * 8, clive, yn,
                                  p.hdr, SITE_SCAN_Y);
                    if (p.vec && clive == 8) {
                        Raw<IO, 8> w;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t b = Raw<IO, 8>::bits(from_f32<IO>(o[i]));
                            if constexpr (sizeof(IO) == 4) w.w[i] = b;
                            else if (i % 2 == 0) w.w[i / 2] = b;
                            else w.w[i / 2] |= b << 16;
                        }
#pragma unroll
                        for (int i = 0; i < Raw<IO, 8>::W / 4; ++i)
                            reinterpret_cast<uint4 *>(out)[i] =
                                make_uint4(w.w[4 * i], w.w[4 * i + 1], w.w[4 * i + 2], w.w[4 * i + 3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i < clive) out[i] = from_f32<IO>(o[i]);
                    }
                }
            }
        }
    }
    if (SUM) {
        if (live) {
            const int64_t i0 = packed ? item : sq * (p.nseg - 1) + k;
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                const int n = n0 + 2 * i;
                const float2 v = unpack2(h[i]);
                if (n < p.N) {
                    float *s = chk(p.seg_state, i0 * p.D_ * p.N + cN + n, n + 1 < p.N ? 2 : 1,
                                   p.seg_items * p.D_ * p.N, p.hdr, SITE_SCAN_SEG);
                    s[0] = v.x;
                    if (n + 1 < p.N) s[1] = v.y;
                }
            }
            if (q == 0) p.seg_dt[i0 * p.D_ + c0 + ch] = dt_sum;
        }
    } else if (!packed && t1 == p.L) {
        final_state(sq);
    }
}

// One token for every sequence: the states are read and written once, from and to HBM, which bounds it. A thread keeps
// the A of its R states for TG sequences, whose states are all in flight together; of a channel's S lanes each
// discretises and gates for one of the sequences (as in the transposed sum above, which serves here too).
template <typename IO, int S, int R>
__global__ void __launch_bounds__(256) step_kernel(ScanParams p) {
    constexpr int CT = 256 / S, TG = S < 8 ? S : 8;
    const int64_t ctiles = (p.D_ + CT - 1) / CT;
    const int ch = threadIdx.x / S, q = threadIdx.x % S, n0 = q * R;
    const int64_t c = blockIdx.x % ctiles * CT + ch, s0 = blockIdx.x / ctiles * TG;
    const bool live = c < p.D_;
    const int64_t cc = live ? c : 0, cN = cc * p.N, g = cc / p.cpg;
    const int nl = live ? (int)(p.N - n0) : 0;  // states of this lane (may be negative)
    const int64_t total = p.nseq * p.D_ * p.N;
    (void)total;
    float h[TG][R], b[R], cs[R], a[R];
#pragma unroll
    for (int j = 0; j < TG; ++j) {
        const int64_t i = (s0 + j) * p.D_ * p.N + cN + n0;
        if (p.init && s0 + j < p.nseq && nl > 0) {
            if (p.vec_state && nl >= R) {
                if (p.state_f16) {
                    Raw<__half, R> r;
                    r.load(chk(static_cast<const __half *>(p.init), i, R, total, p.hdr, SITE_SCAN_STATE));
#pragma unroll
                    for (int k = 0; k < R; ++k) h[j][k] = r.get(k);
                } else {
                    Raw<float, R> r;
                    r.load(chk(static_cast<const float *>(p.init), i, R, total, p.hdr, SITE_SCAN_STATE));
#pragma unroll
                    for (int k = 0; k < R; ++k) h[j][k] = r.get(k);
                }
            } else {
#pragma unroll
                for (int k = 0; k < R; ++k) h[j][k] = k < nl ? load_state(p, p.init, i + k) : 0.f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < R; ++k) h[j][k] = 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) a[k] = k < nl ? p.A[cN + n0 + k] * kLog2e : 0.f;
    // lane q discretises for sequence mine (of the group of TG)
    const int mine = q * TG / S;
    float xv = 0.f, d = 0.f, zv = 0.f;
    if (s0 + mine < p.nseq && live) {
        const int64_t s = s0 + mine;
        xv = to_f32(static_cast<const IO *>(p.x)[s * p.x_seq + cc]);
        d = to_f32(static_cast<const IO *>(p.dt)[s * p.dt_seq + cc]) + (p.dt_bias ? p.dt_bias[cc] : 0.f);
        if (p.z) zv = to_f32(static_cast<const IO *>(p.z)[s * p.z_seq + cc]);
        if (p.softplus) d = softplus_fast(d);
    }
    const float u = d * xv;
    float v[TG];
#pragma unroll
    for (int j = 0; j < TG; ++j) {
        const int src = j * (S / TG);
        const float dj = __shfl_sync(0xffffffffu, d, src, S), uj = __shfl_sync(0xffffffffu, u, src, S);
        float acc = 0.f;
        if (s0 + j < p.nseq) {
            const int64_t s = s0 + j;
            const IO *B = static_cast<const IO *>(p.B) + s * p.b_seq + g * p.N + n0;
            const IO *C = static_cast<const IO *>(p.C) + s * p.c_seq + g * p.N + n0;
            if (p.vec_bc && nl >= R) {
                Raw<IO, R> rb, rc;
                rb.load(B);
                rc.load(C);
#pragma unroll
                for (int k = 0; k < R; ++k) b[k] = rb.get(k), cs[k] = rc.get(k);
            } else {
#pragma unroll
                for (int k = 0; k < R; ++k) b[k] = k < nl ? to_f32(B[k]) : 0.f, cs[k] = k < nl ? to_f32(C[k]) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                h[j][k] = fmaf(ex2(dj * a[k]), h[j][k], uj * b[k]);
                acc = fmaf(h[j][k], cs[k], acc);
            }
            if (p.fin && nl > 0) {
                const int64_t i = s * p.D_ * p.N + cN + n0;
                if (p.vec_state && nl >= R) {
                    if (p.state_f16) {
                        __half *o = chk(static_cast<__half *>(p.fin), i, R, total, p.hdr, SITE_SCAN_STATE);
                        __half2 w[R / 2];
#pragma unroll
                        for (int k = 0; k < R / 2; ++k) w[k] = __floats2half2_rn(h[j][2 * k], h[j][2 * k + 1]);
                        if constexpr (R == 4) *reinterpret_cast<uint2 *>(o) = *reinterpret_cast<const uint2 *>(w);
                        else *reinterpret_cast<uint4 *>(o) = *reinterpret_cast<const uint4 *>(w);
                    } else {
                        float *o = chk(static_cast<float *>(p.fin), i, R, total, p.hdr, SITE_SCAN_STATE);
#pragma unroll
                        for (int k = 0; k < R; k += 4)
                            *reinterpret_cast<float4 *>(o + k) = make_float4(h[j][k], h[j][k + 1], h[j][k + 2], h[j][k + 3]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < R; ++k)
                        if (k < nl) store_state(p, p.fin, i + k, h[j][k]);
                }
            }
        }
        v[j] = acc;
    }
    float y = fmaf(p.D ? p.D[cc] : 0.f, xv, reduce_lanes<S, TG>(v, q));
    if (p.z) y *= silu_f32(zv);
    if (live && s0 + mine < p.nseq && (S <= TG || q % (S / TG) == 0))
        *chk(static_cast<IO *>(p.y), (s0 + mine) * p.y_seq + cc, 1, (p.rows - 1) * p.y_seq + p.D_, p.hdr,
             SITE_SCAN_Y) = from_f32<IO>(y);
}

template <typename IO, typename T, bool SUM>
cudaError_t launch_pass(const ScanParams &p, int64_t items, cudaStream_t stream) {
    const int64_t grid = items * ((p.cpg + T::CT - 1) / T::CT) * p.G;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    auto k = scan_kernel<IO, T, SUM>;
    constexpr size_t smem = T::smem(SUM);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    k<<<(unsigned)grid, T::NT, smem, stream>>>(p);
    return cudaGetLastError();
}
template <typename IO, typename T>
cudaError_t launch_shape(const ScanParams &p, cudaStream_t stream) {
    if (p.nseg > 1) {
        const cudaError_t e = launch_pass<IO, T, true>(p, p.seg_items, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_pass<IO, T, false>(p, p.cu ? p.nseg : p.nseq * p.nseg, stream);
}
template <typename IO, int S, int R>
cudaError_t launch_step_kernel(const ScanParams &p, cudaStream_t stream) {
    constexpr int CT = 256 / S, TG = S < 8 ? S : 8;
    const int64_t grid = (p.D_ + CT - 1) / CT * ((p.nseq + TG - 1) / TG);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    step_kernel<IO, S, R><<<(unsigned)grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

using Shape4 = Shape<1, 4, 64, 32>;     // up to 4 states
using Shape8 = Shape<2, 4, 128, 32>;    // up to 8
using Shape16 = Shape<4, 4, 256, 32>;   // up to 16
using Shape32 = Shape<4, 8, 256, 32>;
using Shape64 = Shape<8, 8, 256, 32>;
using Shape128 = Shape<16, 8, 256, 32>;
using Shape256 = Shape<32, 8, 256, 16>;

template <typename IO> cudaError_t launch_io(const ScanParams &p, cudaStream_t stream) {
    if (!p.cu && p.L == 1) {
        if (p.N <= 4) return launch_step_kernel<IO, 1, 4>(p, stream);
        if (p.N <= 8) return launch_step_kernel<IO, 2, 4>(p, stream);
        if (p.N <= 16) return launch_step_kernel<IO, 4, 4>(p, stream);
        if (p.N <= 32) return launch_step_kernel<IO, 8, 4>(p, stream);
        if (p.N <= 64) return launch_step_kernel<IO, 16, 4>(p, stream);
        if (p.N <= 128) return launch_step_kernel<IO, 32, 4>(p, stream);
        return launch_step_kernel<IO, 32, 8>(p, stream);
    }
    if (p.N <= 4) return launch_shape<IO, Shape4>(p, stream);
    if (p.N <= 8) return launch_shape<IO, Shape8>(p, stream);
    if (p.N <= 16) return launch_shape<IO, Shape16>(p, stream);
    if (p.N <= 32) return launch_shape<IO, Shape32>(p, stream);
    if (p.N <= 64) return launch_shape<IO, Shape64>(p, stream);
    if (p.N <= 128) return launch_shape<IO, Shape128>(p, stream);
    return launch_shape<IO, Shape256>(p, stream);
}

}  // namespace scan
}  // namespace ssd
