// Group norm with an activation, channels last, statistics per token and group (include/ssd.h has the formulas).
//
// HBM-bound: x and z are read once and y written once. W warps hold a token's group in registers, up to three 16-byte
// vectors a lane, so the variance is taken of the differences from the mean, not from sums of squares; a group that one
// warp holds needs no barrier. CTAs of 512 threads an SM stay (weight and bias come from L1), and the
// next token's vectors are loaded under the sums of this one: without that 16384 x 1536 channels with a gate took 39 us
// however many warps there were, with it 28; four or more vectors a lane leave too few warps (39 us). In e4m3 the 16
// (fp32: 32) lanes that hold 128 channels find their largest magnitude by shuffles. Rows that are not 16-byte multiples
// go by pairs (16384 x 1538: 57 us) or single elements (1537: 84). Longer groups (over 24576 channels, in fp32 12288, by
// pairs and elements 8192), and e4m3 of unaligned rows, take the kernel that reads a group three times.
#pragma once

#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace norm {

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
__global__ void __launch_bounds__(kThreads) norm_long_kernel(NormParams p) {
    after_previous();
    __shared__ float red[kThreads / 32];
    const int64_t gs = p.D / p.G;
    for (int64_t item = blockIdx.x; item < p.rows * p.G; item += gridDim.x) {
        const int64_t row = item / p.G, c0 = (item % p.G) * gs;
        const IO *x = chk(static_cast<const IO *>(p.x), row * p.x_row + c0, gs, (p.rows - 1) * p.x_row + p.D, p.hdr,
                          SITE_NORM_IN);
        const IO *z = !p.z ? nullptr
                           : chk(static_cast<const IO *>(p.z), row * p.z_row + c0, gs, (p.rows - 1) * p.z_row + p.D,
                                 p.hdr, SITE_NORM_IN);
        const int64_t yn = (p.rows - 1) * p.y_row + p.D;
        (void)yn;
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
            const float v = fmaf((in(i) - mean) * r, p.w ? *chk(p.w, c, 1, p.D, p.hdr, SITE_WEIGHT) : 1.f,
                                 p.bias ? *chk(p.bias, c, 1, p.D, p.hdr, SITE_WEIGHT) : 0.f);
            return !z ? act(v) : p.gate_first ? v : v * act(to_f32(z[i]));
        };
        if (!p.scales) {
            IO *y = chk(static_cast<IO *>(p.y), row * p.y_row + c0, gs, yn, p.hdr, SITE_NORM_OUT);
            for (int64_t i = threadIdx.x; i < gs; i += kThreads) y[i] = from_f32<IO>(value(i));
        } else {  // a warp takes a block of 128 channels, four a lane
            uint8_t *y = chk(static_cast<uint8_t *>(p.y), row * p.y_row + c0, gs, yn, p.hdr, SITE_NORM_OUT);
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

// Sum over a group's W warps (W = 1: over the warp), the same in all its lanes.
__device__ __forceinline__ float group_sum(float v, float *red, int W, int warp) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (W == 1) return v;
    if (threadIdx.x % 32 == 0) red[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < W; ++i) s += red[i];
    return s;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "mul.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "add.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 silu2(float2 v) {
    const float2 e = mul2(v, both(-kLog2e));
    const float2 d = add2(make_float2(ex2(e.x), ex2(e.y)), both(1.f));
    return mul2(v, make_float2(rcp(d.x), rcp(d.y)));
}

constexpr int kMostWarps = 16;
enum Gate { kNone, kFirst, kAfter };

// W warps a group: W = 1, four groups in a CTA of 128 threads; else one, in a CTA of 32 W threads. V: elements of a
// vector (16 bytes, 4 bytes of 16-bit types, or 1); a lane's values are in packed pairs, of one vector or (V = 1) of neighbouring single elements.
template <typename IO, int V, int NV, bool Q, int GATE>
__global__ void __launch_bounds__(32 * kMostWarps, 1) norm_kernel(NormParams p, int W) {
    constexpr int P = NV * V / 2, PV = V / 2;  // pairs of a lane, of a vector
    __shared__ float red[4][32];  // by sum and by parity of the item: one barrier a sum separates its writers and readers
    int parity = 0;
    const int lane = threadIdx.x % 32, warp = W == 1 ? 0 : threadIdx.x / 32;
    after_previous();
    const int64_t gs = p.D / p.G;
    const int nvec = (int)(gs / V);
    const int64_t step = W == 1 ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t xn = (p.rows - 1) * p.x_row + p.D, zn = (p.rows - 1) * p.z_row + p.D, yn = (p.rows - 1) * p.y_row + p.D;
    (void)xn, (void)zn, (void)yn;
    const float inv_n = 1.f / (float)gs;
    const IO *x = static_cast<const IO *>(p.x), *z = static_cast<const IO *>(p.z);
    int64_t grp, row = quick_div(W == 1 ? (int64_t)blockIdx.x * 4 + threadIdx.x / 32 : blockIdx.x, p.G, grp);
    int64_t step_grp, step_row = quick_div(step, p.G, step_grp);
    // this lane's vectors: e0, e0 + 32 W, ..
    const int e0 = warp * 32 + lane, apart = 32 * W, mine = e0 < nvec ? (nvec - e0 + apart - 1) / apart : 0;
    Raw<IO, V> rx[NV], rz[GATE != kNone ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        rx[i].zero();
        if (GATE != kNone) rz[i].zero();
    }
    auto load = [&](int64_t r, int64_t g) {  // what lies past the group stays zero
        if (r >= p.rows) return;
        const int64_t xi = r * p.x_row + g * gs + e0 * V, zi = r * p.z_row + g * gs + e0 * V;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < mine) {
                rx[i].load(chk(x, xi + i * apart * V, V, xn, p.hdr, SITE_NORM_IN));
                if (GATE != kNone) rz[i].load(chk(z, zi + i * apart * V, V, zn, p.hdr, SITE_NORM_IN));
            }
    };
    auto value = [&](const auto &r, int k) {  // pair k of a lane
        if constexpr (V == 1) return make_float2(r[2 * k].get(0), r[2 * k + 1].get(0));
        else return r[k / (PV ? PV : 1)].pair(2 * (k % (PV ? PV : 1)));
    };
    load(row, grp);
    for (; row < p.rows; parity ^= 1) {
        const int64_t c0 = grp * gs;
        float2 v[P];
        Raw<IO, V> gate[GATE != kNone ? NV : 1];
        auto act2 = [&](float2 u) { return p.silu ? silu2(u) : u; };
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = value(rx, k);
        if constexpr (GATE != kNone) {
#pragma unroll
            for (int i = 0; i < NV; ++i) gate[i] = rz[i];
        }
        int64_t next_row = row + step_row, next_grp = grp + step_grp;
        if (next_grp >= p.G) next_grp -= p.G, ++next_row;
        load(next_row, next_grp);  // under this token's arithmetic
        if constexpr (GATE == kFirst) {
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] = mul2(v[k], act2(value(gate, k)));
        }
        if (p.center) {
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < P; ++k) s = add2(s, v[k]);
            const float mean = group_sum(s.x + s.y, red[2 * parity], W, warp) * inv_n;
            // what lies past the group stays 0
            if constexpr (V == 1) {
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    v[k].x -= 2 * k < mine ? mean : 0.f;
                    v[k].y -= 2 * k + 1 < mine ? mean : 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float2 m = both(i < mine ? -mean : 0.f);
#pragma unroll
                    for (int k = 0; k < PV; ++k) v[i * PV + k] = add2(v[i * PV + k], m);
                }
            }
        }
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < P; ++k) s = fma2(v[k], v[k], s);
        const float r = rsqrtf(group_sum(s.x + s.y, red[2 * parity + 1], W, warp) * inv_n + p.eps);
        const int64_t ci = c0 + e0 * V, yi = row * p.y_row + ci;
        // weight and bias of a pair's channels (only read where they exist: i < mine)
        auto scale_shift = [&](int i, float2 *o) {
            const float *wp = chk(p.w, ci + i * apart * V, V, p.D, p.hdr, SITE_WEIGHT);
            const float *bp = chk(p.bias, ci + i * apart * V, V, p.D, p.hdr, SITE_WEIGHT);
            if constexpr (V == 1) {
                if (p.w) o[0].x *= __ldg(wp);
                if (p.bias) o[0].x += __ldg(bp);
            } else if constexpr (V == 2) {
                if (p.w) o[0] = mul2(o[0], __ldg(reinterpret_cast<const float2 *>(wp)));
                if (p.bias) o[0] = add2(o[0], __ldg(reinterpret_cast<const float2 *>(bp)));
            } else {
                if (p.w)
#pragma unroll
                    for (int k = 0; k < V; k += 4) {
                        const float4 f = __ldg(reinterpret_cast<const float4 *>(wp + k));
                        o[k / 2] = mul2(o[k / 2], make_float2(f.x, f.y));
                        o[k / 2 + 1] = mul2(o[k / 2 + 1], make_float2(f.z, f.w));
                    }
                if (p.bias)
#pragma unroll
                    for (int k = 0; k < V; k += 4) {
                        const float4 f = __ldg(reinterpret_cast<const float4 *>(bp + k));
                        o[k / 2] = add2(o[k / 2], make_float2(f.x, f.y));
                        o[k / 2 + 1] = add2(o[k / 2 + 1], make_float2(f.z, f.w));
                    }
            }
        };
        if constexpr (V == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < mine) {
                    float2 o = make_float2((i % 2 ? v[i / 2].y : v[i / 2].x) * r, 0.f);
                    scale_shift(i, &o);
                    if (GATE == kNone && p.silu) o.x = silu_f32(o.x);
                    if constexpr (GATE == kAfter) o.x *= p.silu ? silu_f32(gate[i].get(0)) : gate[i].get(0);
                    *chk(static_cast<IO *>(p.y), yi + i * apart, 1, yn, p.hdr, SITE_NORM_OUT) = from_f32<IO>(o.x);
                }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool in = i < mine;
                float2 o[PV];
#pragma unroll
                for (int k = 0; k < PV; ++k) o[k] = mul2(v[i * PV + k], both(r));
                if (in) {
                    scale_shift(i, o);
                    if constexpr (GATE == kNone) {
#pragma unroll
                        for (int k = 0; k < PV; ++k) o[k] = act2(o[k]);
                    } else if constexpr (GATE == kAfter) {
#pragma unroll
                        for (int k = 0; k < PV; ++k) o[k] = mul2(o[k], act2(gate[i].pair(2 * k)));
                    }
                }
                if constexpr (!Q) {
                    if (in) {
                        Raw<IO, V> t;
#pragma unroll
                        for (int k = 0; k < PV; ++k) t.set_pair(2 * k, o[k].x, o[k].y);
                        IO *y = chk(static_cast<IO *>(p.y), yi + i * apart * V, V, yn, p.hdr, SITE_NORM_OUT);
                        if constexpr (V == 2) *reinterpret_cast<uint32_t *>(y) = t.w[0];
                        else *reinterpret_cast<uint4 *>(y) = make_uint4(t.w[0], t.w[1], t.w[2], t.w[3]);
                    }
                } else {
                    constexpr int LANES = 128 / V;  // lanes of a block; lanes past the group hold zeros
                    float m = 0.f;
#pragma unroll
                    for (int k = 0; k < PV; ++k) m = max_nan(max_nan(m, fabsf(o[k].x)), fabsf(o[k].y));
#pragma unroll
                    for (int d = LANES / 2; d > 0; d /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
                    float scale, inv;
                    e4m3_scale(m, scale, inv);
                    if (in) {
                        const int64_t kb = (p.D + 127) / 128;
                        if (lane % LANES == 0)
                            *chk(p.scales, row * kb + (ci + i * apart * V) / 128, 1, p.rows * kb, p.hdr,
                                 SITE_NORM_SCALE) = scale;
                        uint8_t *y = chk(static_cast<uint8_t *>(p.y), yi + i * apart * V, V, yn, p.hdr, SITE_NORM_OUT);
                        uint32_t q[PV / 2];
#pragma unroll
                        for (int k = 0; k < PV; k += 2) {
                            const float2 a = mul2(o[k], both(inv)), b = mul2(o[k + 1], both(inv));
                            q[k / 2] = (uint32_t)e4m3x2(a.x, a.y) | (uint32_t)e4m3x2(b.x, b.y) << 16;
                        }
                        if constexpr (V == 8) *reinterpret_cast<uint2 *>(y) = make_uint2(q[0], q[1]);
                        else *reinterpret_cast<uint32_t *>(y) = q[0];
                    }
                }
            }
        }
        row = next_row;
        grp = next_grp;
    }
}

template <typename IO, int V, int NV, bool Q, int GATE>
cudaError_t launch_gate(const NormParams &p, int W, int sms, cudaStream_t stream) {
    const int threads = W == 1 ? 128 : 32 * W;
    const int64_t items = p.rows * p.G, ctas = W == 1 ? (items + 3) / 4 : items;
    // 512 threads an SM: more of them, where they fit, ran the same or slower
    const int64_t grid = std::min<int64_t>(ctas, (int64_t)sms * std::max(1, 512 / threads));
    if (grid == ctas) return launch_after(norm_kernel<IO, V, NV, Q, GATE>, grid, threads, 0, stream, p, W);
    // CTAs that walk rows start once the kernel before has left every SM: started as its CTAs leave, more than their
    // share would gather on the SMs that come free first (8191 x 5120 and the product behind it: 172 us against 160)
    norm_kernel<IO, V, NV, Q, GATE><<<(unsigned)grid, threads, 0, stream>>>(p, W);
    return cudaGetLastError();
}
template <typename IO, int V, int NV, bool Q>
cudaError_t launch_q(const NormParams &p, int W, int sms, cudaStream_t stream) {
    if (!p.z) return launch_gate<IO, V, NV, Q, kNone>(p, W, sms, stream);
    return p.gate_first ? launch_gate<IO, V, NV, Q, kFirst>(p, W, sms, stream)
                        : launch_gate<IO, V, NV, Q, kAfter>(p, W, sms, stream);
}
template <typename IO, int V, int NV>
cudaError_t launch_nv(const NormParams &p, int W, int sms, cudaStream_t stream) {
    if constexpr (V > 2)
        if (p.scales) return launch_q<IO, V, NV, true>(p, W, sms, stream);
    return launch_q<IO, V, NV, false>(p, W, sms, stream);
}

template <typename IO> cudaError_t launch_io(const NormParams &p, int sms, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(IO);
    const int64_t gs = p.D / p.G;
    // a CTA holds 16 warps at most, a lane up to 3 vectors (6 of longer groups), or 4 pairs (8), or 8 single elements
    // (16; with 4 of them 16384 x 1537 took 112 us)
    const int64_t nvec = p.unit == 16 ? gs / V : p.unit == 4 ? gs / 2 : gs;
    const int few = p.unit == 16 ? 3 : p.unit == 4 ? 4 : 8, many = p.unit == 16 ? 6 : p.unit == 4 ? 8 : 16;
    if (nvec <= kMostWarps * 32 * many && (p.unit == 16 || !p.scales)) {
        const int most = nvec <= kMostWarps * 32 * few ? few : many;
        const int W = (int)((nvec + 32 * most - 1) / (32 * most));
        const int NV = (int)((nvec + 32 * W - 1) / (32 * W));
        if (p.unit == 16) switch (NV) {
            case 1: return launch_nv<IO, V, 1>(p, W, sms, stream);
            case 2: return launch_nv<IO, V, 2>(p, W, sms, stream);
            case 3: return launch_nv<IO, V, 3>(p, W, sms, stream);
            default: return launch_nv<IO, V, 6>(p, W, sms, stream);
        }
        if constexpr (sizeof(IO) == 2)
            if (p.unit == 4)
                return NV <= 4 ? launch_nv<IO, 2, 4>(p, W, sms, stream) : launch_nv<IO, 2, 8>(p, W, sms, stream);
        return NV <= 8 ? launch_nv<IO, 1, 8>(p, W, sms, stream) : launch_nv<IO, 1, 16>(p, W, sms, stream);
    }
    const int64_t grid = std::min<int64_t>(p.rows * p.G, (int64_t)sms * 64);
    norm_long_kernel<IO><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace norm
}  // namespace ssd
