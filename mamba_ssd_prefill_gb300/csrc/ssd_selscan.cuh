// Selective scan ("Mamba hardware-aware algorithms", fused selective scan: discretise, scan and contract with C in
// one kernel): per sequence and channel c, with dt = softplus(dt_raw + dt_bias),
//
//   h[n] <- exp(dt A[c, n]) h[n] + dt x[c] B[n],     y[c] = (sum_n C[n] h[n] + D[c] x[c]) z[c] sigmoid(z[c])
//
// Every (token, channel, state) costs one exponential and four multiply-adds, against 8 bytes per (token, channel) in
// 16-bit types: at 16 states the FMA and special-function pipes bound it, not HBM. A packed f32x2 instruction takes two
// cycles of a quarter's FMA pipe, an exponential four of the other and 1.5 of the issue beside it: 5.7 cycles an element
// and quarter for the recurrence alone. So the states stay in registers, and what is around it is kept small:
//
//  - A CTA owns CT channels (of one group) and walks tokens in tiles of TT. A tile's x, dt and z are copied to shared
//    memory one tile ahead (asynchronous copies of 16, 8 or 4 bytes as rows are aligned, or through registers); each
//    thread turns the vectors that it copied into (dt, dt x)
//    per token and channel, B and C are kept in fp32. The softplus is so taken once per (token, channel).
//  - A thread holds CH channels x R states in packed pairs, S lanes share the states of its channels. A shared memory
//    load costs its bytes per lane, broadcast or not (an LDS.128 four cycles of the SM's pipe), and B and C are eight
//    bytes for every element: with one channel a thread they took 3.4 cycles an element and bounded the kernel. CH = 4,
//    R = 8 (128 registers) and CH = 2, R = 8 (96) measure the same where segments fill the GPU (16384 x 5120 x 16:
//    0.73 ms); where they are not needed the smaller one has more warps and is taken (32 x 4096 x 1536 x 16, both in one
//    build: CH = 4 1.75 ms, CH = 2 1.28; the present build takes 1.48). Up to 8 states a tile is 4 tokens and not 8, of
//    which fewer CTAs would fit in shared memory (4 x 4096 x 1536 x 4: 131 us against 178; 12824 x 4000 x 8: 330
//    against 380).
//  - States are padded to 4, 8, 16, 24, 32, 64, 128 or 256: 4 x 4096 x 1536 with 32 states takes 437 us, with 33 1035,
//    with 64 932, with 128 1689, with 256 3186.
//  - The sum over a channel's lanes is taken for the thread's channels at once, each shuffle halving the channels a
//    lane holds.
//
// Where (sequences x channel tiles) do not fill the GPU, the tokens are cut into segments: scan_kernel<SUM> first
// computes every segment's leaving state from a zero state, and its summed dt (the state's decay over a segment is
// exp(A sum dt), exactly); join_kernel turns them into the states that enter the segments, and the main pass starts
// every segment from its own. The state part of the work is done twice. Packed sequences are segmented on the packed
// axis, whatever their lengths; a segment restarts its chain wherever a sequence begins inside it.
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

// v[0 .. TG), the shares of TG items in each of a channel's S lanes -> totals: lane q is left with the items q TG / S
// onwards, TG / S of them (one where S >= TG) in v[0 ..].
template <int S, int TG> __device__ __forceinline__ void reduce_lanes(float (&v)[TG], int q) {
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
}

// The last sequence whose start is at or before packed token t (empty ones before it share its start): the whole CTA
// counts the starts, since a search would wait for memory at every step.
__device__ __forceinline__ int64_t seq_at(const int32_t *cu, int64_t nseq, int64_t t) {
    int64_t n = 0;
    for (int64_t s = 0; s < nseq; s += blockDim.x) {
        const int64_t i = s + threadIdx.x;
        n += __syncthreads_count(i < nseq && cu[i] <= t);
    }
    return n > 0 ? n - 1 : 0;  // malformed offsets may start past t
}

template <int S_, int R_, int CH_, int NT_, int TT_, int MINB_, int SINGLE_> struct Shape {
    static constexpr int S = S_, R = R_, CH = CH_, NT = NT_, TT = TT_, MINB = MINB_;
    static constexpr int MINB_SINGLE = SINGLE_;  // CTAs an SM holds of the instances of UNIT 0
    static constexpr int CT = NT / S * CH, NP = S * R, CV = CT / 8;  // channels, states, 8-channel vectors of a CTA
    static constexpr int VPT = (TT * CV + NT - 1) / NT;              // vectors a thread copies per tensor
    static constexpr int NV = NP / 4;                                // 4-state vectors per token
    static constexpr size_t smem(bool sum, size_t es) {
        return (size_t)TT * CT * (8 + (sum ? 0 : 4)) + (size_t)TT * NP * 4 * (sum ? 1 : 2) +
               2 * (size_t)TT * CT * es * (sum ? 2 : 3) + CT * 8;
    }
};

// UNIT: bytes that rows are copied by: 16, 4 (and 8; 4 x 4096 x 1540 x 16: 296 us, by single elements 371), or 0 for
// single elements, 16-bit rows of odd widths or addresses. These wait one by one in registers: held to the same registers
// those instances would spill, so they keep fewer CTAs (12824 x 3981 x 8: 0.49 ms against 0.60).
template <typename IO, typename T, bool SUM, int UNIT>
__global__ void __launch_bounds__(T::NT, UNIT ? T::MINB : T::MINB_SINGLE) scan_kernel(ScanParams p) {
    constexpr int S = T::S, R = T::R, NT = T::NT, TT = T::TT, CT = T::CT, NP = T::NP, CV = T::CV, VPT = T::VPT,
                  NV = T::NV, P = R / 2, kCH = T::CH;
    constexpr int BPT = (TT * NV * (SUM ? 1 : 2) + NT - 1) / NT;
    constexpr int RAW = TT * CT;  // elements of a staged tensor
    extern __shared__ __align__(16) uint8_t smem[];
    float4 *du = reinterpret_cast<float4 *>(smem);                         // [TT][CT / 2] (dt, dt x) of two channels
    float *Bs = reinterpret_cast<float *>(smem + (size_t)TT * CT * 8);     // [TT][NP]
    float *Cs = Bs + TT * NP;                                              // [TT][NP], not for SUM
    float *ys = SUM ? Cs : Cs + TT * NP;                                   // [TT][CT], not for SUM
    float *bias_s = SUM ? ys : ys + TT * CT, *D_s = bias_s + CT;           // [CT] each
    IO *raw = reinterpret_cast<IO *>(D_s + CT);                            // [2][x, dt, z][TT][CT]
    const int tid = threadIdx.x;
    const int64_t per_group = (p.cpg + CT - 1) / CT, ctiles = per_group * p.G;
    int64_t ct, in_group;
    const int64_t item = quick_div(blockIdx.x, ctiles, ct), g = quick_div(ct, per_group, in_group);
    const int64_t c0 = g * p.cpg + in_group * CT;                          // first channel
    const int left = (int)((g + 1) * p.cpg - c0 < CT ? (g + 1) * p.cpg - c0 : CT);  // channels of this CTA
    const int ch = tid / S * kCH, q = tid % S;                             // this thread's first channel, its lane's place
    const int clive = left - ch < 0 ? 0 : left - ch < kCH ? left - ch : kCH;
    const bool packed = p.cu != nullptr;
    after_previous();

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
        packed_range(p.cu, p.nseq, sq, p.T, p.hdr, qb, qe);
        fresh = qb >= t0;
        if (SUM) {
            if (fresh) t0 = qb < t1 ? qb : t1;
            if (qe <= t1) {  // no sequence goes on past this segment
                auto mark = [&](int i) {  // (a loop from tid on made the prompts' passes 1.7 % slower: 742 against 729 us)
                    if (i < left)
                        *chk(p.seg_dt, item * p.D_ + c0 + i, 1, p.seg_items * p.D_, p.hdr, SITE_SCAN_SEG) =
                            __int_as_float(0x7fffffff);
                };
#pragma unroll
                for (int i = 0; i < CT; i += NT) mark(tid + i);
                return;
            }
        } else {
            if (qe <= t0) qe = p.T;  // malformed offsets
            if (item == 0 && ct == 0) check_offsets(p.cu, p.nseq, p.T, p.hdr);
            if (p.fin)  // empty sequences keep their states; each segment's CTAs look after some of them
                for (int64_t s = item; s < p.nseq; s += p.nseg)
                    if (const int32_t *o = chk(p.cu, s, 2, p.nseq + 1, p.hdr, SITE_OFFSETS); o[0] == o[1])
                        for (int64_t e = tid; e < left * p.N; e += NT) {
                            const int64_t i = (s * p.D_ + c0) * p.N + e;
                            store_state(p, p.fin, i, p.init ? load_state(p, p.init, i) : 0.f);
                        }
        }
    } else {
        sq = quick_div(item, nseg, k);
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

    // copies of one tile: vectors of 8 channels of a token; a thread later reads the vectors that it copied itself
    const int cv = tid % CV * 8, trow = tid / CV;  // first channel of this thread's vectors, first token
    const int vlive = left - cv < 0 ? 0 : left - cv < 8 ? left - cv : 8;
    constexpr int TSTEP = NT / CV;
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
    auto copy = [&](IO *dst, const IO *src) {
        if (vlive == 8) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(IO) / 2; ++i) {
                uint8_t *d = reinterpret_cast<uint8_t *>(dst) + 16 * i;
                const uint8_t *s = reinterpret_cast<const uint8_t *>(src) + 16 * i;
                if constexpr (UNIT == 16) {
                    cp_async16(d, s);
                } else if (p.unit == 8) {
                    cp_async<8>(d, s);
                    cp_async<8>(d + 8, s + 8);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) cp_async<4>(d + j, s + j);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = i < vlive ? src[i] : from_f32<IO>(0.f);
        }
    };
    // element offsets of this thread's first vectors in the tile that is copied next, stepped from tile to tile
    int64_t ox = (t0 + trow) * p.x_tok + cv, od = (t0 + trow) * p.dt_tok + cv, oz = (t0 + trow) * p.z_tok + cv;
    const int b_t = tid / NV % TT, b_n = tid % NV * 4;
    Raw<IO, 8> ahead[UNIT ? 1 : SUM ? 2 : 3][UNIT ? 1 : VPT];
    auto load = [&](int64_t tile, int stage) {
        IO *st = raw + stage * (SUM ? 2 : 3) * RAW + trow * CT + cv;
        const int n = (int)(t1 - tile < TT ? t1 - tile : TT);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int t = trow + v * TSTEP;
            if (t < n && vlive > 0) {
                const IO *px = at(x, p.x, ox + v * TSTEP * p.x_tok, vlive, xn);
                const IO *pd = at(dt, p.dt, od + v * TSTEP * p.dt_tok, vlive, dn);
                const IO *pz = !SUM && z ? at(z, p.z, oz + v * TSTEP * p.z_tok, vlive, zn) : nullptr;
                if constexpr (UNIT != 0) {
                    copy(st + v * TSTEP * CT, px);
                    copy(st + RAW + v * TSTEP * CT, pd);
                    if (!SUM && pz) copy(st + 2 * RAW + v * TSTEP * CT, pz);
                } else {  // element by element, to registers: on their way while the tile before is worked on
                    if (vlive == 8) {
                        ahead[0][v].load_each(px);
                        ahead[1][v].load_each(pd);
                        if (!SUM && pz) ahead[SUM ? 1 : 2][v].load_each(pz);
                    } else {
                        ahead[0][v].load(px, vlive, false);
                        ahead[1][v].load(pd, vlive, false);
                        if (!SUM && pz) ahead[SUM ? 1 : 2][v].load(pz, vlive, false);
                    }
                }
            }
        }
        ox += TT * p.x_tok;
        od += TT * p.dt_tok;
        if (!SUM) oz += TT * p.z_tok;
        asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
        for (int v = 0; v < BPT; ++v) {
            const int e = tid + v * NT, t = BPT == 1 ? b_t : e / NV % TT, n4 = BPT == 1 ? b_n : e % NV * 4;
            const int nl = (int)(p.N - n4);
            rb[v].zero();
            if (e < TT * NV * (SUM ? 1 : 2) && t < n && nl > 0) {
                const int64_t tk = tile + t;
                if (SUM || e < TT * NV) rb[v].load(at(B, p.B, tk * p.b_tok + n4, nl < 4 ? nl : 4, bn), nl, p.vec_bc);
                else rb[v].load(at(C, p.C, tk * p.c_tok + n4, nl < 4 ? nl : 4, cn), nl, p.vec_bc);
            }
        }
    };
    load(t0, 0);

    for (int i = tid; i < CT; i += NT) {
        bias_s[i] = p.dt_bias && i < left ? *chk(p.dt_bias, c0 + i, 1, p.D_, p.hdr, SITE_WEIGHT) : 0.f;
        D_s[i] = p.D && i < left ? *chk(p.D, c0 + i, 1, p.D_, p.hdr, SITE_WEIGHT) : 0.f;
    }
    f2 a[kCH][P], h[kCH][P];
    const int n0 = q * R;
    auto get2 = [&](auto f) {  // f(c, n) for this lane's channels and states, 0 past the last
#pragma unroll
        for (int c = 0; c < kCH; ++c)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int n = n0 + 2 * i;
                h[c][i] = pack2(c < clive && n < p.N ? f(c0 + ch + c, n) : 0.f,
                                c < clive && n + 1 < p.N ? f(c0 + ch + c, n + 1) : 0.f);
            }
    };
    // whole vectors of this lane's channels and states: rows of N at `base`
    const bool vec_rows = p.vec_state && clive == kCH && n0 + R <= p.N;
    auto get_rows = [&](const auto *base, int64_t i, int64_t n, uint32_t site) {  // i: the first channel's row
        using E = typename std::remove_cv<typename std::remove_reference<decltype(*base)>::type>::type;
#pragma unroll
        for (int c = 0; c < kCH; ++c)
#pragma unroll
            for (int j = 0; j < R; j += 4) {
                Raw<E, 4> r;
                r.load(chk(base, (i + c) * p.N + n0 + j, 4, n, p.hdr, site));
                const float2 u = r.pair(0), w = r.pair(2);
                h[c][j / 2] = pack2(u.x, u.y);
                h[c][j / 2 + 1] = pack2(w.x, w.y);
            }
    };
    if (vec_rows) get_rows(p.A, c0 + ch, p.D_ * p.N, SITE_WEIGHT);
    else get2([&](int64_t c, int n) { return *chk(p.A, c * p.N + n, 1, p.D_ * p.N, p.hdr, SITE_WEIGHT); });
#pragma unroll
    for (int c = 0; c < kCH; ++c)
#pragma unroll
        for (int i = 0; i < P; ++i) a[c][i] = mul2(h[c][i], pack2(kLog2e, kLog2e));
    auto initial = [&](int64_t s) {
        if (!p.init) get2([](int64_t, int) { return 0.f; });
        else if (!vec_rows) get2([&](int64_t c, int n) { return load_state(p, p.init, (s * p.D_ + c) * p.N + n); });
        else if (p.state_f16)
            get_rows(static_cast<const __half *>(p.init), s * p.D_ + c0 + ch, p.nseq * p.D_ * p.N, SITE_SCAN_STATE);
        else
            get_rows(static_cast<const float *>(p.init), s * p.D_ + c0 + ch, p.nseq * p.D_ * p.N, SITE_SCAN_STATE);
    };
    auto each_state = [&](auto f) {  // f(c, n, h) for this lane's channels and states
#pragma unroll
        for (int c = 0; c < kCH; ++c)
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int n = n0 + 2 * i;
                const float2 v = unpack2(h[c][i]);
                if (c < clive && n < p.N) f(c0 + ch + c, n, v.x);
                if (c < clive && n + 1 < p.N) f(c0 + ch + c, n + 1, v.y);
            }
    };
    auto final_state = [&](int64_t s) {
        if (p.fin) each_state([&](int64_t c, int n, float v) { store_state(p, p.fin, (s * p.D_ + c) * p.N + n, v); });
    };
    const int64_t extent = p.seg_items * p.D_ * p.N;
    (void)extent;
    if (fresh) {
        initial(sq);
    } else if (SUM) {
        get2([](int64_t, int) { return 0.f; });
    } else {  // the state that enters this segment
        const int64_t i0 = (packed ? 0 : sq * (p.nseg - 1)) + k - 1;
        if (vec_rows) get_rows(static_cast<const float *>(p.seg_state), i0 * p.D_ + c0 + ch, extent, SITE_SCAN_SEG);
        else
            get2([&](int64_t c, int n) {
                return *chk(p.seg_state, (i0 * p.D_ + c) * p.N + n, 1, extent, p.hdr, SITE_SCAN_SEG);
            });
    }

    // places of a two-channel unit in a row of du, of a four-channel unit in a row of ys: threads that write and threads
    // that read neighbouring units fall on different banks
    auto du_at = [](int t, int unit) { return t * (CT / 2) + (unit ^ ((unit >> 3) & 3)); };
    auto ys_at = [](int t, int unit) { return t * CT + (unit ^ ((unit >> 3) & 1)) * 4; };
    float dt_sum[kCH] = {};

    // tokens [lo, hi) of the tile in shared memory; MASK: the others leave the state alone
    auto run = [&](auto mask, int lo, int hi) {
        constexpr bool MASK = decltype(mask)::value;
        float part[kCH] = {};
#pragma unroll 2
        for (int t = MASK ? lo : 0; t < (MASK ? hi : TT); ++t) {
            float d[kCH], u[kCH];
#pragma unroll
            for (int c = 0; c < kCH; c += 2) {
                const float4 w = du[du_at(t, (ch + c) / 2)];
                d[c] = w.x, u[c] = w.y, d[c + 1] = w.z, u[c + 1] = w.w;
            }
            const ulonglong2 *bp = reinterpret_cast<const ulonglong2 *>(Bs + t * NP + n0);
            const ulonglong2 *cp = reinterpret_cast<const ulonglong2 *>(Cs + t * NP + n0);
            f2 b[P], cc[P];
#pragma unroll
            for (int j = 0; j < P / 2; ++j) {
                const ulonglong2 w = bp[j];
                b[2 * j] = w.x;
                b[2 * j + 1] = w.y;
            }
            if (!SUM)
#pragma unroll
                for (int j = 0; j < P / 2; ++j) {
                    const ulonglong2 w = cp[j];
                    cc[2 * j] = w.x;
                    cc[2 * j + 1] = w.y;
                }
            float v[kCH];
#pragma unroll
            for (int c = 0; c < kCH; ++c) {
                const f2 dd = pack2(d[c], d[c]), uu = pack2(u[c], u[c]);
                f2 y = 0;
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const float2 e = unpack2(mul2(dd, a[c][j]));
                    h[c][j] = fma2(pack2(ex2(e.x), ex2(e.y)), h[c][j], mul2(uu, b[j]));
                    if (!SUM) y = j == 0 ? mul2(h[c][j], cc[j]) : fma2(h[c][j], cc[j], y);
                }
                const float2 yy = unpack2(y);
                v[c] = yy.x + yy.y;
                if (SUM) part[c] += d[c];
            }
            if (!SUM) {
                reduce_lanes<S, kCH>(v, q);
                constexpr int LEFT = S < kCH ? kCH / S : 1;  // channels left in this lane
                const int c = ch + q * kCH / S;
                float *o = ys + ys_at(t, c / 4) + c % 4;
                if constexpr (LEFT == 4) *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
                else if constexpr (LEFT == 2) *reinterpret_cast<float2 *>(o) = make_float2(v[0], v[1]);
                else if (S <= kCH || q % (S / kCH) == 0) o[0] = v[0];
            }
        }
        if (SUM)
#pragma unroll
            for (int c = 0; c < kCH; ++c) dt_sum[c] += part[c];
    };

    int64_t oy = row * p.y_seq + (t0 + trow) * p.y_tok + c0 + cv;
    int stage = 0;
    for (int64_t tile = t0; tile < t1; tile += TT, stage ^= 1, oy += TT * p.y_tok) {
        const int n = (int)(t1 - tile < TT ? t1 - tile : TT);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (tile == t0) __syncthreads();  // bias_s and D_s
        IO *st = raw + stage * (SUM ? 2 : 3) * RAW;
        if constexpr (UNIT == 0) {
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int t = trow + v * TSTEP;
                if (t < n && vlive > 0) {
                    ahead[0][v].store(st + t * CT + cv);
                    ahead[1][v].store(st + RAW + t * CT + cv);
                    if (!SUM && z) ahead[SUM ? 1 : 2][v].store(st + 2 * RAW + t * CT + cv);
                }
            }
        }
        // (dt, dt x); tokens past the end: a decay of 1 and nothing added
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int t = trow + v * TSTEP;
            if (TT * CV % NT == 0 || t < TT) {
                Raw<IO, 8> rx, rd;
                rx.load(st + t * CT + cv);
                rd.load(st + RAW + t * CT + cv);
                if (t < n) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 r2 = rd.pair(i), x2 = rx.pair(i);
                        const float2 b2 = *reinterpret_cast<const float2 *>(bias_s + cv + i);
                        float d0 = r2.x + b2.x, d1 = r2.y + b2.y;
                        if (p.softplus) d0 = softplus_fast(d0), d1 = softplus_fast(d1);
                        du[du_at(t, (cv + i) / 2)] = make_float4(d0, d0 * x2.x, d1, d1 * x2.y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) du[du_at(t, (cv + i) / 2)] = make_float4(0.f, 0.f, 0.f, 0.f);
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
        if (tile + TT < t1) load(tile + TT, stage ^ 1);
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
                        packed_range(p.cu, p.nseq, sq, p.T, p.hdr, qb, qe);
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
                const int t = trow + v * TSTEP;
                if (t < n && vlive > 0) {
                    Raw<IO, 8> rx, rz;
                    rx.load(st + t * CT + cv);
                    if (z) rz.load(st + 2 * RAW + t * CT + cv);
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const float4 y4 = *reinterpret_cast<const float4 *>(ys + ys_at(t, (cv + i) / 4));
                        const float4 D4 = *reinterpret_cast<const float4 *>(D_s + cv + i);
                        const float2 xa = rx.pair(i), xb = rx.pair(i + 2);
                        o[i] = fmaf(D4.x, xa.x, y4.x);
                        o[i + 1] = fmaf(D4.y, xa.y, y4.y);
                        o[i + 2] = fmaf(D4.z, xb.x, y4.z);
                        o[i + 3] = fmaf(D4.w, xb.y, y4.w);
                    }
                    if (z)
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float2 g = rz.pair(i);
                            o[i] *= silu_f32(g.x);
                            o[i + 1] *= silu_f32(g.y);
                        }
                    IO *out = chk(static_cast<IO *>(p.y), oy + v * TSTEP * p.y_tok, vlive, yn, p.hdr, SITE_SCAN_Y);
                    if (UNIT == 0 && vlive == 8) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) out[i] = from_f32<IO>(o[i]);
                    } else if (vlive == 8) {
                        Raw<IO, 8> w;
#pragma unroll
                        for (int i = 0; i < 8; i += 2) w.set_pair(i, o[i], o[i + 1]);
#pragma unroll
                        for (int i = 0; i < Raw<IO, 8>::W / 4; ++i) {
                            if constexpr (UNIT == 16) {
                                reinterpret_cast<uint4 *>(out)[i] =
                                    make_uint4(w.w[4 * i], w.w[4 * i + 1], w.w[4 * i + 2], w.w[4 * i + 3]);
                            } else {
#pragma unroll
                                for (int j = 4 * i; j < 4 * i + 4; ++j) reinterpret_cast<uint32_t *>(out)[j] = w.w[j];
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i < vlive) out[i] = from_f32<IO>(o[i]);
                    }
                }
            }
        }
    }
    if (SUM) {
        const int64_t i0 = packed ? item : sq * (p.nseg - 1) + k;
        each_state([&](int64_t c, int n, float v) {
            *chk(p.seg_state, (i0 * p.D_ + c) * p.N + n, 1, extent, p.hdr, SITE_SCAN_SEG) = v;
        });
        // a segment in which a sequence begins does not take up the state before it: its sum is NaN
#pragma unroll
        for (int c = 0; c < kCH; ++c)
            if (q == 0 && c < clive)
                *chk(p.seg_dt, i0 * p.D_ + c0 + ch + c, 1, p.seg_items * p.D_, p.hdr, SITE_SCAN_SEG) =
                    packed && fresh ? __int_as_float(0x7fffffff) : dt_sum[c];
    } else if (!packed && t1 == p.L) {
        final_state(sq);
    }
}

// seg_state[i], the leaving state of segment i from a zero state -> from its true entering state (which is what enters
// segment i + 1). A chain is a state of a channel through the segments of a sequence (packed: of the axis). What bounds
// it is waiting for memory: so a thread takes kJoin segments that are all on their way at once, and up to kJoinThreads
// threads share a chain, each first joining its own segments from a zero state (9001 x 1000 x 24: 76 segments 12 us from
// cold memory; one thread a chain took 90 for 188).
constexpr int kJoin = 16, kJoinThreads = 8, kJoinChains = 32;

static __global__ void __launch_bounds__(kJoinChains *kJoinThreads) join_kernel(ScanParams p) {
    __shared__ float2 part[2][kJoinThreads][kJoinChains];  // (sum of dt, leaving state) of the threads' segments
    after_previous();
    const int64_t e = (int64_t)blockIdx.x * kJoinChains + threadIdx.x, dn = p.D_ * p.N;
    const int64_t chains = p.cu ? 1 : p.nseq, segs = p.nseg - 1;
    const bool live = e < chains * dn;
    int64_t i = 0, c = 0, base = 0, rest;
    if (live) {
        base = quick_div(e, dn, i) * segs;
        c = quick_div(i, p.N, rest);
    }
    const float a = live ? *chk(p.A, i, 1, dn, p.hdr, SITE_WEIGHT) * kLog2e : 0.f;
    const int64_t extent = p.seg_items * dn;
    (void)extent;
    // (d, v) leaves h as exp(a d) h + v; as v where d is NaN: a segment in which a sequence begins
    auto pass = [&](float d, float v, float h) { return d != d ? v : fmaf(ex2(a * d), h, v); };
    float enter = 0.f;  // the state that enters this round's segments
    int parity = 0;
    for (int64_t r0 = 0; r0 < segs; r0 += kJoin * blockDim.y, parity ^= 1) {
        const int64_t j0 = r0 + threadIdx.y * kJoin;
        const int n = !live || j0 >= segs ? 0 : (int)(segs - j0 < kJoin ? segs - j0 : kJoin);
        float v[kJoin], d[kJoin];
        float *s = chk(p.seg_state, n ? (base + j0) * dn + i : 0, n ? (n - 1) * dn + 1 : 0, extent, p.hdr, SITE_SCAN_SEG);
        const float *sd = chk_rows(p.seg_dt, n ? (base + j0) * p.D_ + c : 0, n, p.D_, 1, p.seg_items * p.D_, p.hdr,
                                   SITE_SCAN_SEG);
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            v[j] = d[j] = 0.f;
            if (j < n) v[j] = s[j * dn], d[j] = sd[j * p.D_];
        }
        if (j0 == 0) d[0] = __int_as_float(0x7fffffff);
        if (blockDim.y > 1) {
            float h = 0.f, sum = 0.f;
#pragma unroll
            for (int j = 0; j < kJoin; ++j) {
                if (j < n) h = pass(d[j], v[j], h);
                sum += d[j];
            }
            part[parity][threadIdx.y][threadIdx.x] = make_float2(sum, h);
            __syncthreads();
            float all = enter, mine = enter;
            for (int y = 0; y < (int)blockDim.y && r0 + y * kJoin < segs; ++y) {
                if (y == (int)threadIdx.y) mine = all;
                const float2 w = part[parity][y][threadIdx.x];
                all = pass(w.x, w.y, all);
            }
            enter = all;
            h = mine;
#pragma unroll
            for (int j = 0; j < kJoin; ++j)
                if (j < n) s[j * dn] = h = pass(d[j], v[j], h);
        } else {
#pragma unroll
            for (int j = 0; j < kJoin; ++j)
                if (j < n) s[j * dn] = enter = pass(d[j], v[j], enter);
        }
    }
}

// One token for every sequence: the states are read and written once, from and to HBM, which bounds it. A thread takes
// its R states of a channel through kSeqs sequences, whose states, B and C are all on their way before the first is used;
// of a channel's S lanes each discretises and gates for some of the sequences (the sums over the lanes are transposed to
// match), so that no softplus is taken twice.
constexpr int kSeqs = 8;

template <typename IO, typename ST, int S, int R>
__global__ void __launch_bounds__(128) step_kernel(ScanParams p) {
    constexpr int CT = 128 / S, PER = kSeqs / S > 0 ? kSeqs / S : 1;  // channels of a CTA, sequences a lane gates for
    const int64_t ctiles = (p.D_ + CT - 1) / CT;
    const int ch = threadIdx.x / S, q = threadIdx.x % S, n0 = q * R;
    int64_t ct, rest;
    const int64_t s0 = quick_div(blockIdx.x, ctiles, ct) * kSeqs, c = ct * CT + ch;
    const bool live = c < p.D_;
    const int64_t cc = live ? c : 0, cN = cc * p.N, g = quick_div(cc, p.cpg, rest);
    const int nl = live ? (int)(p.N - n0) : 0;  // states of this lane (may be negative)
    const int ns = (int)(p.nseq - s0 < kSeqs ? p.nseq - s0 : kSeqs);
    const int64_t total = p.nseq * p.D_ * p.N, seq_states = p.D_ * p.N;
    (void)total;
    const bool whole = nl >= R;
    const int mine_n = whole ? R : nl < 0 ? 0 : nl;
    (void)mine_n;
    after_previous();
    const int mine = q * kSeqs / S;  // this lane discretises and gates for the sequences mine, mine + 1, ..
    const int64_t i0 = s0 * seq_states + cN + n0;
    const float bias = p.dt_bias ? *chk(p.dt_bias, cc, 1, p.D_, p.hdr, SITE_WEIGHT) : 0.f;
    const float Dc = p.D ? *chk(p.D, cc, 1, p.D_, p.hdr, SITE_WEIGHT) : 0.f;
    float a[R];
#pragma unroll
    for (int k = 0; k < R; ++k) a[k] = k < nl ? *chk(p.A, cN + n0 + k, 1, p.D_ * p.N, p.hdr, SITE_WEIGHT) * kLog2e : 0.f;

    // FAST: all of the group's sequences and of this lane's states exist, and whole vectors are aligned
    auto body = [&](auto fast) {
        constexpr bool FAST = decltype(fast)::value;
        Raw<ST, R> rh[kSeqs];
        Raw<IO, R> rb[kSeqs], rc[kSeqs];
        const ST *init = static_cast<const ST *>(p.init);
        if (init) {
            const ST *hp = chk_rows(init, i0, ns, seq_states, mine_n, total, p.hdr, SITE_SCAN_STATE);
#pragma unroll
            for (int j = 0; j < kSeqs; ++j) {
                if constexpr (FAST) {
                    rh[j].load(hp + j * seq_states);
                } else {
                    rh[j].zero();
                    if (j < ns && nl > 0) rh[j].load(hp + j * seq_states, nl, p.vec_state);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSeqs; ++j) rh[j].zero();
        }
        float x[PER], d[PER], z[PER], u[PER];
        {
            auto rows = [&](const void *q, int64_t seq) {  // this channel in the lane's sequences
                return chk_rows(static_cast<const IO *>(q), (s0 + mine) * seq + cc, ns - mine < PER ? ns - mine : PER,
                                seq, 1, (p.rows - 1) * seq + p.D_, p.hdr, SITE_SCAN_IN);
            };
            const IO *xp = rows(p.x, p.x_seq), *dp = rows(p.dt, p.dt_seq);
            const IO *zp = p.z ? rows(p.z, p.z_seq) : nullptr;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                x[j] = d[j] = z[j] = 0.f;
                if (FAST || mine + j < ns) {
                    x[j] = to_f32(xp[j * p.x_seq]);
                    d[j] = to_f32(dp[j * p.dt_seq]) + bias;
                    if (zp) z[j] = to_f32(zp[j * p.z_seq]);
                }
            }
        }
        {
            auto rows = [&](const void *q, int64_t seq) {  // this lane's states in the sequences
                return chk_rows(static_cast<const IO *>(q), s0 * seq + g * p.N + n0, ns, seq, mine_n,
                                (p.rows - 1) * seq + p.G * p.N, p.hdr, SITE_SCAN_IN);
            };
            const IO *B = rows(p.B, p.b_seq), *C = rows(p.C, p.c_seq);
#pragma unroll
            for (int j = 0; j < kSeqs; ++j) {
                if constexpr (FAST) {
                    rb[j].load(B + j * p.b_seq);
                    rc[j].load(C + j * p.c_seq);
                } else {
                    rb[j].zero();
                    rc[j].zero();
                    if (j < ns && nl > 0) {
                        rb[j].load(B + j * p.b_seq, nl, p.vec_bc);
                        rc[j].load(C + j * p.c_seq, nl, p.vec_bc);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (p.softplus) d[j] = softplus_fast(d[j]);
            u[j] = d[j] * x[j];
        }
        float v[kSeqs];
        ST *fp = static_cast<ST *>(p.fin);
        if (fp) fp = chk_rows(fp, i0, ns, seq_states, mine_n, total, p.hdr, SITE_SCAN_STATE);
#pragma unroll
        for (int j = 0; j < kSeqs; ++j) {
            const int src = j * S / kSeqs;  // the lane that discretised for sequence j
            const float dj = __shfl_sync(0xffffffffu, d[j % PER], src, S);
            const float uj = __shfl_sync(0xffffffffu, u[j % PER], src, S);
            float h[R], acc = 0.f;
#pragma unroll
            for (int k = 0; k < R; k += 2) {
                const float2 h2 = rh[j].pair(k), b2 = rb[j].pair(k), c2 = rc[j].pair(k);
                h[k] = fmaf(ex2(dj * a[k]), h2.x, uj * b2.x);
                h[k + 1] = fmaf(ex2(dj * a[k + 1]), h2.y, uj * b2.y);
                acc = fmaf(h[k + 1], c2.y, fmaf(h[k], c2.x, acc));
            }
            v[j] = acc;
            if (fp && (FAST || (j < ns && nl > 0))) {
                ST *o = fp + j * seq_states;
                if (FAST || (p.vec_state && whole)) {
                    Raw<ST, R> w;
#pragma unroll
                    for (int k = 0; k < R; k += 2) w.set_pair(k, h[k], h[k + 1]);
                    if constexpr (Raw<ST, R>::W == 2) {
                        *reinterpret_cast<uint2 *>(o) = make_uint2(w.w[0], w.w[1]);
                    } else {
#pragma unroll
                        for (int k = 0; k < Raw<ST, R>::W; k += 4)
                            reinterpret_cast<uint4 *>(o)[k / 4] =
                                make_uint4(w.w[k], w.w[k + 1], w.w[k + 2], w.w[k + 3]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < R; ++k)
                        if (k < nl) o[k] = from_f32<ST>(h[k]);
                }
            }
        }
        reduce_lanes<S, kSeqs>(v, q);
        if (live && (S <= kSeqs || q % (S / kSeqs) == 0))
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (FAST || mine + j < ns) {
                    float y = fmaf(Dc, x[j], v[j]);
                    if (p.z) y *= silu_f32(z[j]);
                    *chk(static_cast<IO *>(p.y), (s0 + mine + j) * p.y_seq + cc, 1, (p.rows - 1) * p.y_seq + p.D_, p.hdr,
                         SITE_SCAN_Y) = from_f32<IO>(y);
                }
    };
    // the same for all lanes of a warp, which exchange values inside
    if (__all_sync(0xffffffffu, ns == kSeqs && live && whole && p.vec_state && p.vec_bc))
        body(std::integral_constant<bool, true>());
    else
        body(std::integral_constant<bool, false>());
}

template <typename IO, typename T, bool SUM, int UNIT>
cudaError_t launch_pass(const ScanParams &p, int64_t items, cudaStream_t stream) {
    const int64_t grid = items * ((p.cpg + T::CT - 1) / T::CT) * p.G;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    auto k = scan_kernel<IO, T, SUM, UNIT>;
    constexpr size_t smem = T::smem(SUM, sizeof(IO));
    if constexpr (smem > 48 * 1024) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(k, smem, done);
        if (e != cudaSuccess) return e;
    }
    if (p.nseg == 1) {
        // Whole chains, fewer CTAs than fit, start once the kernel before has left every SM: started as its CTAs leave,
        // they crowd on the SMs that come free first (32 x 4096 x 1536 x 16, 384 CTAs: 2.00 ms against 1.48).
        k<<<(unsigned)grid, T::NT, smem, stream>>>(p);
        return cudaGetLastError();
    }
    return launch_after(k, grid, T::NT, smem, stream, p);
}
template <typename IO, typename T, bool SUM>
cudaError_t launch_rows(const ScanParams &p, int64_t items, cudaStream_t stream) {
    if constexpr (sizeof(IO) < 4)
        if (p.unit == 0) return launch_pass<IO, T, SUM, 0>(p, items, stream);
    return p.unit == 16 ? launch_pass<IO, T, SUM, 16>(p, items, stream) : launch_pass<IO, T, SUM, 4>(p, items, stream);
}
template <typename IO, typename T>
cudaError_t launch_shape(const ScanParams &p, cudaStream_t stream) {
    if (p.nseg > 1) {
        cudaError_t e = launch_rows<IO, T, true>(p, p.seg_items, stream);
        if (e != cudaSuccess) return e;
        if (p.nseg > 2) {
            const int64_t grid = ((p.cu ? 1 : p.nseq) * p.D_ * p.N + kJoinChains - 1) / kJoinChains;
            if (grid > INT32_MAX) return cudaErrorInvalidValue;
            const int64_t share = (p.nseg - 1 + kJoin - 1) / kJoin;
            e = launch_after(join_kernel, grid, dim3(kJoinChains, (unsigned)std::min<int64_t>(share, kJoinThreads)), 0,
                             stream, p);
            if (e != cudaSuccess) return e;
        }
    }
    const int64_t items = p.cu ? p.nseg : p.nseq * p.nseg;
    return launch_rows<IO, T, false>(p, items, stream);
}
template <typename IO, int S, int R>
cudaError_t launch_step_kernel(const ScanParams &p, cudaStream_t stream) {
    constexpr int CT = 128 / S;
    const int64_t grid = (p.D_ + CT - 1) / CT * ((p.nseq + kSeqs - 1) / kSeqs);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return p.state_f16 ? launch_after(step_kernel<IO, __half, S, R>, grid, 128, 0, stream, p)
                       : launch_after(step_kernel<IO, float, S, R>, grid, 128, 0, stream, p);
}

// By the number of states; scan_cta (ssd_internal.h) tells the planner their channels and threads.
using Shape4 = Shape<1, 4, 4, 32, 4, 16, 12>;
using Shape8 = Shape<1, 8, 2, 64, 4, 8, 7>;
using Shape16 = Shape<2, 8, 2, 128, 8, 5, 4>;
using Shape24 = Shape<2, 12, 2, 128, 8, 4, 3>;
using Shape32 = Shape<4, 8, 2, 256, 8, 2, 1>;
using Shape64 = Shape<8, 8, 2, 256, 8, 2, 1>;
using Shape128 = Shape<16, 8, 2, 256, 8, 2, 1>;
using Shape256 = Shape<32, 8, 2, 256, 8, 2, 1>;

template <typename IO, typename T> cudaError_t launch_checked(const ScanParams &p, cudaStream_t stream) {
    const ScanCta c = scan_cta(p.N);
    const bool agree = c.channels == T::CT && c.threads == T::NT && c.resident == T::MINB &&
                       c.resident_single == T::MINB_SINGLE;
    return agree ? launch_shape<IO, T>(p, stream) : cudaErrorInvalidValue;
}

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
    if (p.N <= 4) return launch_checked<IO, Shape4>(p, stream);
    if (p.N <= 8) return launch_checked<IO, Shape8>(p, stream);
    if (p.N <= 16) return launch_checked<IO, Shape16>(p, stream);
    if (p.N <= 24) return launch_checked<IO, Shape24>(p, stream);
    if (p.N <= 32) return launch_checked<IO, Shape32>(p, stream);
    if (p.N <= 64) return launch_checked<IO, Shape64>(p, stream);
    if (p.N <= 128) return launch_checked<IO, Shape128>(p, stream);
    return launch_checked<IO, Shape256>(p, stream);
}

}  // namespace scan
}  // namespace ssd
