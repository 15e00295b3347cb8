// Causal depthwise convolution over the tokens by itself, rows at any stride, regular or packed sequences:
//
//   out[t, c] = act(bias[c] + sum_j w[c, j] x[t - (k - 1) + j, c]),   x before a sequence from its cache
//
// HBM-bound: one read and one write of every row. A thread owns 16 bytes of channels and walks up to 64 tokens with the
// taps and the last k - 1 inputs in fp32 registers; the k - 1 rows before its tokens are read again (from L2). Its rows
// come through a ring of 16-byte asynchronous copies in shared memory, four stages of four tokens, in slots that no
// other thread touches: 32 KB a CTA in flight without a register or a barrier (loads to registers, eight ahead, kept
// 168 registers and 12 warps and ran 8 x 8192 x 5376 channels in 396 us; the ring with a predicate on every token 361;
// whole stages without one, so that the window of inputs is renamed and not moved, 216 us, 6.5 TB/s). Rows that are
// not 16-byte multiples are copied in units of 4 bytes (5378 channels: 296 us); 16-bit rows of odd widths or addresses
// take one channel a thread from registers (5377 channels: 399 us).
// The cache leaves with the thread that walks a sequence's last token, so a prompt takes one launch, and a single token
// too: its thread reads the old cache before it writes the new one. Only where the cache is updated in place and another
// thread reads its old entries does a second kernel write it.
#include <string.h>

#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 128;

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

// What a thread walks: tokens [t0, t1) of the row axis of `row`, in sequence s on [start, end).
struct Walk {
    int64_t s, row, t0, t1, start, end;
};
__device__ __forceinline__ Walk walk_of(const RowConvParams &p, int64_t item, int64_t tiles, int tl) {
    Walk w;
    if (p.cu) {
        w.row = 0;
        w.t0 = item * tl;
        w.t1 = w.t0 + tl < p.T ? w.t0 + tl : p.T;
        w.s = seq_of(p.cu, p.nseq, w.t0);
        packed_range(p.cu, p.nseq, w.s, p.T, p.hdr, w.start, w.end);
        if (w.start > w.t0) w.start = w.t0;  // malformed offsets
        if (w.end <= w.t0) w.end = p.T + 1;
    } else {
        int64_t tile;
        w.s = w.row = quick_div(item, tiles, tile);
        w.t0 = tile * tl;
        w.t1 = w.t0 + tl < p.L ? w.t0 + tl : p.L;
        w.start = 0;
        w.end = p.L;
    }
    return w;
}
// The sequence that begins at packed token t, after the one that ended there.
__device__ __forceinline__ void next_sequence(const RowConvParams &p, Walk &w, int64_t t) {
    do {
        if (++w.s >= p.nseq) break;
        packed_range(p.cu, p.nseq, w.s, p.T, p.hdr, w.start, w.end);
    } while (w.end <= t);
    if (w.s >= p.nseq) w.s = p.nseq - 1, w.start = t, w.end = p.T + 1;  // malformed offsets
}

// V channels a thread (16 bytes; V = 1: single elements), rows copied by UNIT bytes (16 or 4). The rows come through a ring in shared
// memory, kGroup tokens a stage, in slots that only their thread writes and reads (no barrier); V = 1 loads a stage's
// tokens to registers instead.
// CTAs an SM: by registers; with more the wider windows spill (8 x 8192 x 5376, width 5: 4 CTAs 279 us, 3 268; width 8: 3
// 506, 2 464; width 7: 3 339, 2 378).
constexpr int kStages = 4;

template <typename IO, int K, int V, int UNIT>
__global__ void __launch_bounds__(kThreads, V == 1 ? 8 : K > 7 ? 2 : K > 4 ? 3 : 4)
    row_conv_kernel(RowConvParams p, int tl, int64_t tiles, int write_state) {
    constexpr int KH = K > 1 ? K - 1 : 1, P = V > 1 ? V / 2 : 1, G = V > 1 ? 4 : 8;  // P: channel pairs, G: tokens a stage
    __shared__ uint4 ring[V > 1 ? kStages * G : 1][V > 1 ? kThreads : 1];
    constexpr bool PART = V > 1 && UNIT < 16;       // a row's last thread may hold fewer channels
    constexpr int E = 4 / (int)sizeof(IO);          // elements of 4 bytes
    const int64_t nvec = (p.D + V - 1) / V, idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    after_previous();
    if (p.cu && blockIdx.x == 0) check_offsets(p.cu, p.nseq, p.T, p.hdr);
    int64_t cvec;
    const int64_t item = quick_div(idx, nvec, cvec), c = cvec * V;
    if (item >= (p.cu ? tiles : p.nseq * tiles)) return;
    const int live = PART && p.D - c < V ? (int)(p.D - c) : V;
    Walk wk = walk_of(p, item, tiles, tl);
    const IO *x = static_cast<const IO *>(p.x);
    const IO *state = static_cast<const IO *>(p.state);
    IO *sout = static_cast<IO *>(p.state_out);
    const int64_t xn = (p.rows - 1) * p.x_seq + (p.L - 1) * p.x_tok + p.D, sn = p.nseq * p.D * (K - 1);
    const int64_t on = (p.rows - 1) * p.out_seq + (p.L - 1) * p.out_tok + p.D;
    (void)xn, (void)sn, (void)on;
    const int64_t xo = wk.row * p.x_seq + c;

    // the first rows of the walk are on their way while the taps and the inputs before them are read
    int64_t xt = xo + wk.t0 * p.x_tok, fetched = wk.t0;
    auto fetch = [&](int stage) {
        if constexpr (V > 1) {
#pragma unroll
            for (int u = 0; u < G; ++u)
                if (fetched + u < wk.t1) {
                    const IO *s = chk(x, xt + u * p.x_tok, live, xn, p.hdr, SITE_RCONV_IN);
                    uint4 *d = &ring[stage * G + u][threadIdx.x];
                    if constexpr (PART) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j * E < live) cp_async<4>(reinterpret_cast<uint32_t *>(d) + j, s + j * E);
                    } else {
                        cp_async16(d, s);
                    }
                }
            asm volatile("cp.async.commit_group;" ::: "memory");
            xt += G * p.x_tok;
            fetched += G;
        }
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);

    float2 hist[KH][P];  // hist[j]: the input of token t - 1 - j (V = 1: its .x)
    // inputs before token t of sequence q on [begin, ..)
    auto load_hist = [&](int64_t q, int64_t t, int64_t begin) {
        if (V > 1 && !PART && K > 1 && t == begin && state && p.vec_state) {  // all of them cached: whole vectors
            Raw<IO, V * KH> r;
            r.load(chk(state, (q * p.D + c) * (K - 1), V * (K - 1), sn, p.hdr, SITE_RCONV_STATE));
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int i = 0; i < P; ++i)
                    hist[j][i] = make_float2(r.get(2 * i * KH + K - 2 - j), r.get((2 * i + 1) * KH + K - 2 - j));
            return;
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int64_t tp = t - 1 - j;
            float v[2 * P];
            if (tp >= begin) {
                const IO *r = chk(x, xo + tp * p.x_tok, live, xn, p.hdr, SITE_RCONV_IN);
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = i < live ? to_f32(r[i]) : 0.f;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[i] = state && i < live ? to_f32(*chk(state, (q * p.D + c + i) * (K - 1) + (K - 1) + (tp - begin), 1, sn,
                                               p.hdr, SITE_RCONV_STATE))
                                 : 0.f;
            }
#pragma unroll
            for (int i = 0; i < P; ++i) hist[j][i] = make_float2(v[2 * i], V > 1 ? v[2 * i + 1] : 0.f);
        }
    };
    // what the cache of sequence q holds after the inputs in hist
    auto save = [&](int64_t q) {
        if constexpr (K > 1) {
            IO v[V * KH];
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
                    v[i * KH + j] = from_f32<IO>(i % 2 ? hist[K - 2 - j][i / 2].y : hist[K - 2 - j][i / 2].x);
            IO *o = chk(sout, (q * p.D + c) * (K - 1), live * (K - 1), sn, p.hdr, SITE_RCONV_STATE);
            if (V > 1 && !PART && p.vec_state) {
#pragma unroll
                for (int i = 0; i < V * KH * (int)sizeof(IO) / 16; ++i) {
                    uint4 u;
                    memcpy(&u, v + i * (16 / (int)sizeof(IO)), 16);
                    reinterpret_cast<uint4 *>(o)[i] = u;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V * KH; ++i)
                    if (i < live * KH) o[i] = v[i];
            }
        }
    };
    if (p.cu && write_state && K > 1)  // empty sequences keep their cache; each tile's threads look after some of them
        for (int64_t q = item; q < p.nseq; q += tiles)
            if (const int32_t *o = chk(p.cu, q, 2, p.nseq + 1, p.hdr, SITE_OFFSETS); o[0] == o[1]) {
                load_hist(q, 0, 0);
                save(q);
            }

    float2 w[K][P], bias[P];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float t[K];
        const int64_t ci = i < live ? c + i : c;
        const float *wc = chk(p.w, ci * K, K, p.D * K, p.hdr, SITE_WEIGHT);
        if constexpr (K == 4) {
            if (p.vec_w) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(wc));
                t[0] = u.x, t[1] = u.y, t[2] = u.z, t[3] = u.w;
            } else {
#pragma unroll
                for (int j = 0; j < K; ++j) t[j] = wc[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < K; ++j) t[j] = wc[j];
        }
        const float b = p.bias ? *chk(p.bias, ci, 1, p.D, p.hdr, SITE_WEIGHT) : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (i % 2) w[j][i / 2].y = t[j];
            else w[j][i / 2] = make_float2(t[j], 0.f);
        if (i % 2) bias[i / 2].y = b;
        else bias[i / 2] = make_float2(b, 0.f);
    }
    load_hist(wk.s, wk.t0, wk.start);
    IO *out = static_cast<IO *>(p.out);
    int64_t oo = wk.row * p.out_seq + wk.t0 * p.out_tok + c;
    int stage = 0;
    // token u of the stage, in[K - 1] its input and in[j] the ones before it
    auto token = [&](const float2 (&in)[KH + 1][P], int u) {
        float2 acc[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if constexpr (V > 1) {
                acc[i] = bias[i];
#pragma unroll
                for (int j = 0; j < K; ++j) acc[i] = fma2(w[j][i], in[KH + 1 - K + j][i], acc[i]);
            } else {
                acc[i] = bias[i];
#pragma unroll
                for (int j = 0; j < K; ++j) acc[i].x = fmaf(w[j][i].x, in[KH + 1 - K + j][i].x, acc[i].x);
            }
            if (p.silu) {
                acc[i].x = silu_f32(acc[i].x);
                if (V > 1) acc[i].y = silu_f32(acc[i].y);
            }
        }
        IO *dst = chk(out, oo + u * p.out_tok, live, on, p.hdr, SITE_RCONV_OUT);
        if constexpr (V > 1) {
            Raw<IO, V> o;
#pragma unroll
            for (int i = 0; i < P; ++i) o.set_pair(2 * i, acc[i].x, acc[i].y);
            if constexpr (PART) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j * E < live) reinterpret_cast<uint32_t *>(dst)[j] = o.w[j];
            } else {
                *reinterpret_cast<uint4 *>(dst) = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
            }
        } else {
            *dst = from_f32<IO>(acc[0].x);
        }
    };
    for (int64_t t = wk.t0; t < wk.t1; t += G) {
        const int n = (int)(wk.t1 - t < G ? wk.t1 - t : G);
        IO one[V > 1 ? 1 : G];
        if constexpr (V > 1) {
            fetch((stage + kStages - 1) % kStages);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        } else {
#pragma unroll
            for (int u = 0; u < G; ++u) {
                one[u] = from_f32<IO>(0.f);
                if (u < n) one[u] = *chk(x, xt + u * p.x_tok, 1, xn, p.hdr, SITE_RCONV_IN);
            }
            xt += G * p.x_tok;
        }
        auto input = [&](float2 (&v)[P], int u) {
            if constexpr (V > 1) {
                Raw<IO, V> r;
                const uint4 q = ring[stage * G + u][threadIdx.x];
                r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = r.pair(2 * i);
            } else {
                v[0] = make_float2(to_f32(one[V > 1 ? 0 : u]), 0.f);
            }
        };
        if (n == G && (!p.cu || wk.end >= t + G)) {  // a whole stage of one sequence
            float2 win[G + KH][P];
#pragma unroll
            for (int j = 0; j < KH; ++j)
#pragma unroll
                for (int i = 0; i < P; ++i) win[j][i] = hist[KH - 1 - j][i];
#pragma unroll
            for (int u = 0; u < G; ++u) {
                input(win[KH + u], u);
                token(reinterpret_cast<const float2(&)[KH + 1][P]>(win[u]), u);
            }
#pragma unroll
            for (int j = 0; j < KH; ++j)
#pragma unroll
                for (int i = 0; i < P; ++i) hist[j][i] = win[G + KH - 1 - j][i];
        } else {
#pragma unroll
            for (int u = 0; u < G; ++u) {
                if (u < n) {
                    if (p.cu && t + u == wk.end) {
                        if (write_state) save(wk.s);
                        next_sequence(p, wk, t + u);
                        load_hist(wk.s, wk.start, wk.start);
                    }
                    float2 win[KH + 1][P];
#pragma unroll
                    for (int j = 0; j < KH; ++j)
#pragma unroll
                        for (int i = 0; i < P; ++i) win[j][i] = hist[KH - 1 - j][i];
                    input(win[KH], u);
                    token(win, u);
#pragma unroll
                    for (int j = 0; j < KH; ++j)
#pragma unroll
                        for (int i = 0; i < P; ++i) hist[j][i] = win[KH - j][i];
                }
            }
        }
        oo += G * p.out_tok;
        stage = (stage + 1) % kStages;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (write_state && wk.t1 == wk.end) save(wk.s);
}

// The last k - 1 inputs of every sequence, for a cache updated in place or a call without tokens. A thread owns a
// (sequence, channel): its old entries are read before any is written.
template <typename IO>
__global__ void __launch_bounds__(kThreads) row_conv_state_kernel(RowConvParams p) {
    after_previous();
    const int64_t total = p.nseq * p.D;
    const IO *x = static_cast<const IO *>(p.x);
    const IO *state = static_cast<const IO *>(p.state);
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < total; e += (int64_t)gridDim.x * kThreads) {
        const int64_t s = e / p.D, c = e % p.D;
        int64_t row0 = 0, end = p.L;
        if (p.cu) packed_range(p.cu, p.nseq, s, p.T, p.hdr, row0, end);
        IO v[7];
#pragma unroll
        for (int j = 0; j < 7; ++j) {
            const int64_t t = end - (p.k - 1) + j;
            v[j] = from_f32<IO>(0.f);
            if (j < p.k - 1 && t >= row0)
                v[j] = *chk(x, (p.cu ? 0 : s) * p.x_seq + t * p.x_tok + c, 1,
                            (p.rows - 1) * p.x_seq + (p.L - 1) * p.x_tok + p.D, p.hdr, SITE_RCONV_IN);
            else if (j < p.k - 1 && state)
                v[j] = *chk(state, e * (p.k - 1) + (p.k - 1) + (t - row0), 1, total * (p.k - 1), p.hdr,
                            SITE_RCONV_STATE);
        }
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < p.k - 1)
                *chk(static_cast<IO *>(p.state_out), e * (p.k - 1) + j, 1, total * (p.k - 1), p.hdr,
                     SITE_RCONV_STATE) = v[j];
    }
}

template <typename IO, int K, int V, int UNIT>
cudaError_t launch_kv(const RowConvParams &p, int tl, int64_t tiles, int write_state, cudaStream_t stream) {
    const int64_t threads = (p.cu ? tiles : p.nseq * tiles) * ((p.D + V - 1) / V), grid = (threads + kThreads - 1) / kThreads;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_after(row_conv_kernel<IO, K, V, UNIT>, grid, kThreads, 0, stream, p, tl, tiles, write_state);
}
template <typename IO, int V, int UNIT>
cudaError_t launch_v(const RowConvParams &p, int tl, int64_t tiles, int write_state, cudaStream_t stream) {
    switch (p.k) {
        case 1: return launch_kv<IO, 1, V, UNIT>(p, tl, tiles, write_state, stream);
        case 2: return launch_kv<IO, 2, V, UNIT>(p, tl, tiles, write_state, stream);
        case 3: return launch_kv<IO, 3, V, UNIT>(p, tl, tiles, write_state, stream);
        case 4: return launch_kv<IO, 4, V, UNIT>(p, tl, tiles, write_state, stream);
        case 5: return launch_kv<IO, 5, V, UNIT>(p, tl, tiles, write_state, stream);
        case 6: return launch_kv<IO, 6, V, UNIT>(p, tl, tiles, write_state, stream);
        case 7: return launch_kv<IO, 7, V, UNIT>(p, tl, tiles, write_state, stream);
        default: return launch_kv<IO, 8, V, UNIT>(p, tl, tiles, write_state, stream);
    }
}

template <typename IO>
cudaError_t launch_t(const RowConvParams &p, int sms, cudaStream_t stream) {
    const size_t state_bytes = (size_t)(p.nseq * p.D * (p.k - 1)) * sizeof(IO);
    bool save_after = p.state_out && p.k > 1 && p.T == 0;
    if (p.T > 0) {
        constexpr int kVec = 16 / (int)sizeof(IO);
        const int64_t V = p.unit ? kVec : 1, L = p.cu ? p.T : p.L, chains = p.cu ? 1 : p.nseq;
        // 64 tokens a thread (8 x 8192 x 5376: 16 tokens 326 us, 32 240, 64 216, 256 234); shorter walks where those leave
        // SMs idle (4096 x 5376: 32 and 64 tokens 23.5 us, 128 31)
        int tl = 64;
        while (tl > 8 && chains * ((L + tl - 1) / tl) * (p.D / V) < (int64_t)sms * 512) tl /= 2;
        const int64_t tiles = (L + tl - 1) / tl;
        const char *a = static_cast<const char *>(p.state), *b = static_cast<const char *>(p.state_out);
        const bool shared = a && b && a < b + state_bytes && b < a + state_bytes;
        save_after = p.state_out && p.k > 1 && shared && (tiles > 1 || p.cu || a != b);
        const int write_state = p.state_out && p.k > 1 && !save_after;
        cudaError_t e;
        if (p.unit == 16) e = launch_v<IO, kVec, 16>(p, tl, tiles, write_state, stream);
        else if (p.unit == 4) e = launch_v<IO, kVec, 4>(p, tl, tiles, write_state, stream);
        else if constexpr (sizeof(IO) < 4) e = launch_v<IO, 1, 0>(p, tl, tiles, write_state, stream);
        else e = cudaErrorInvalidValue;
        if (e != cudaSuccess) return e;
    }
    if (save_after) {
        const int64_t grid = std::min<int64_t>((p.nseq * p.D + kThreads - 1) / kThreads, (int64_t)sms * 64);
        return launch_after(row_conv_state_kernel<IO>, grid, kThreads, 0, stream, p);
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
