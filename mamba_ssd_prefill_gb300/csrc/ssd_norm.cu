// Group norm with an activation, channels last, statistics per token and group (include/ssd.h has the formulas).
//
// HBM-bound: x and z are read once and y written once. W warps hold a token's group in registers, up to three 16-byte
// vectors a lane, so the variance is taken of the differences from the mean, not from sums of squares; a group that one
// warp holds needs no barrier. The CTAs that fit the SMs stay (512 threads an SM; weight and bias come from L1), and the
// next token's vectors are loaded under the sums of this one: without that 16384 x 1536 channels with a gate took 39 us
// however many warps there were, with it 29; four or more vectors a lane leave too few warps (39 us). In e4m3 the 16
// (fp32: 32) lanes that hold 128 channels find their largest magnitude by shuffles. Rows that are not 16-byte multiples
// go by single elements. Longer groups (over 24576 channels, in fp32 12288, by elements 8192), and e4m3 of unaligned rows, take the
// kernel that reads a group three times.
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
__global__ void __launch_bounds__(kThreads) norm_long_kernel(NormParams p) {
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

// Keeps a branch that all threads take alike a branch: as selects the modes not taken would cost an instruction a value
// each.
#define BRANCH() asm volatile("")

// W warps a group: W = 1, four groups in a CTA of 128 threads; else one, in a CTA of 32 W threads. V: elements of a
// vector (16 bytes, or 1).
constexpr int kMostWarps = 16;

template <typename IO, int V, int NV, bool Q>
__global__ void __launch_bounds__(32 * kMostWarps) norm_kernel(NormParams p, int W) {
    __shared__ float red[4][32];  // by sum and by parity of the item: one barrier a sum separates its writers and readers
    int parity = 0;
    const int lane = threadIdx.x % 32, warp = W == 1 ? 0 : threadIdx.x / 32;
    const int64_t gs = p.D / p.G;
    const int nvec = (int)(gs / V);
    const int64_t step = W == 1 ? (int64_t)gridDim.x * 4 : gridDim.x;
    const int64_t xn = (p.rows - 1) * p.x_row + p.D, zn = (p.rows - 1) * p.z_row + p.D, yn = (p.rows - 1) * p.y_row + p.D;
    (void)xn, (void)zn, (void)yn;
    const float inv_n = 1.f / (float)gs;
    const IO *x = static_cast<const IO *>(p.x), *z = static_cast<const IO *>(p.z);
    int64_t grp, row = quick_div(W == 1 ? (int64_t)blockIdx.x * 4 + threadIdx.x / 32 : blockIdx.x, p.G, grp);
    int64_t step_grp, step_row = quick_div(step, p.G, step_grp);
    auto advance = [&](int64_t &r, int64_t &g) {
        r += step_row;
        g += step_grp;
        if (g >= p.G) g -= p.G, ++r;
    };
    Raw<IO, V> rx[NV], rz[NV];
    // this lane's vectors: e0, e0 + 32 W, ..
    const int e0 = warp * 32 + lane, apart = 32 * W, mine = e0 < nvec ? (nvec - e0 + apart - 1) / apart : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        rx[i].zero();
        rz[i].zero();
    }
    auto load = [&](int64_t r, int64_t g) {  // what lies past the group stays zero
        if (r >= p.rows) return;
        const int64_t xi = r * p.x_row + g * gs + e0 * V, zi = r * p.z_row + g * gs + e0 * V;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i < mine) {
                rx[i].load(chk(x, xi + i * apart * V, V, xn, p.hdr, SITE_NORM_IN));
                if (z) rz[i].load(chk(z, zi + i * apart * V, V, zn, p.hdr, SITE_NORM_IN));
            }
    };
    load(row, grp);
    for (; row < p.rows; parity ^= 1) {
        const int64_t c0 = grp * gs;
        float v[NV][V], gate[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) v[i][k] = rx[i].get(k), gate[i][k] = rz[i].get(k);
        int64_t next_row = row, next_grp = grp;
        advance(next_row, next_grp);
        load(next_row, next_grp);  // under this token's sums
        if (z && p.silu) {
            BRANCH();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) gate[i][k] = silu_f32(gate[i][k]);
        }
        if (p.gate_first) {
            BRANCH();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) v[i][k] *= gate[i][k];
        }
        if (p.center) {
            BRANCH();
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) s += v[i][k];
            const float mean = group_sum(s, red[2 * parity], W, warp) * inv_n;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i < mine)  // what lies past the group stays 0
#pragma unroll
                    for (int k = 0; k < V; ++k) v[i][k] -= mean;
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) s = fmaf(v[i][k], v[i][k], s);
        const float r = rsqrtf(group_sum(s, red[2 * parity + 1], W, warp) * inv_n + p.eps);
        const int64_t ci = c0 + e0 * V, yi = row * p.y_row + ci;
        const float *wp = p.w + (p.w ? ci : 0), *bp = p.bias + (p.bias ? ci : 0);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = i < mine;
            float o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = v[i][k] * r;
            if (in) {
                auto params = [&](const float *src, float (&dst)[V]) {
                    if constexpr (V == 1) {
                        dst[0] = __ldg(src + i * apart * V);
                    } else {
#pragma unroll
                        for (int k = 0; k < V; k += 4) {
                            const float4 f = __ldg(reinterpret_cast<const float4 *>(src + i * apart * V + k));
                            dst[k] = f.x, dst[k + 1] = f.y, dst[k + 2] = f.z, dst[k + 3] = f.w;
                        }
                    }
                };
                float t[V];
                if (p.w) {
                    BRANCH();
                    params(wp, t);
#pragma unroll
                    for (int k = 0; k < V; ++k) o[k] *= t[k];
                }
                if (p.bias) {
                    BRANCH();
                    params(bp, t);
#pragma unroll
                    for (int k = 0; k < V; ++k) o[k] += t[k];
                }
                if (!z && p.silu) {
                    BRANCH();
#pragma unroll
                    for (int k = 0; k < V; ++k) o[k] = silu_f32(o[k]);
                }
                if (z && !p.gate_first) {
                    BRANCH();
#pragma unroll
                    for (int k = 0; k < V; ++k) o[k] *= gate[i][k];
                }
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) o[k] = 0.f;
            }
            if constexpr (!Q) {
                if (in) {
                    IO *y = chk(static_cast<IO *>(p.y), yi + i * apart * V, V, yn, p.hdr, SITE_NORM_OUT);
                    if constexpr (V == 1) {
                        *y = from_f32<IO>(o[0]);
                    } else {
                        Raw<IO, V> t;
#pragma unroll
                        for (int k = 0; k < V; k += 2) t.set_pair(k, o[k], o[k + 1]);
                        *reinterpret_cast<uint4 *>(y) = make_uint4(t.w[0], t.w[1], t.w[2], t.w[3]);
                    }
                }
            } else {
                constexpr int LANES = 128 / V;  // lanes of a block
                float m = 0.f;
#pragma unroll
                for (int k = 0; k < V; ++k) m = max_nan(m, fabsf(o[k]));
#pragma unroll
                for (int d = LANES / 2; d > 0; d /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
                float scale, inv;
                e4m3_scale(m, scale, inv);
                if (in) {
                    const int64_t kb = (p.D + 127) / 128;
                    if (lane % LANES == 0)
                        *chk(p.scales, row * kb + (ci + i * apart * V) / 128, 1, p.rows * kb, p.hdr, SITE_NORM_SCALE) = scale;
                    uint8_t *y = chk(static_cast<uint8_t *>(p.y), yi + i * apart * V, V, yn, p.hdr, SITE_NORM_OUT);
                    uint32_t q[V / 4];
#pragma unroll
                    for (int k = 0; k < V; k += 4)
                        q[k / 4] = (uint32_t)e4m3x2(o[k] * inv, o[k + 1] * inv) |
                                   (uint32_t)e4m3x2(o[k + 2] * inv, o[k + 3] * inv) << 16;
                    if constexpr (V == 8) *reinterpret_cast<uint2 *>(y) = make_uint2(q[0], q[1]);
                    else *reinterpret_cast<uint32_t *>(y) = q[0];
                }
            }
        }
        row = next_row;
        grp = next_grp;
    }
}

template <typename IO, int V, int NV>
cudaError_t launch_nv(const NormParams &p, int W, int sms, cudaStream_t stream) {
    const int64_t items = p.rows * p.G, ctas = W == 1 ? (items + 3) / 4 : items;
    const int threads = W == 1 ? 128 : 32 * W;
    const int64_t grid = std::min<int64_t>(ctas, (int64_t)sms * std::max(1, (V > 1 ? 512 : 1024) / threads));
    if constexpr (V > 1)
        if (p.scales) {
            norm_kernel<IO, V, NV, true><<<(unsigned)grid, threads, 0, stream>>>(p, W);
            return cudaGetLastError();
        }
    norm_kernel<IO, V, NV, false><<<(unsigned)grid, threads, 0, stream>>>(p, W);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_t(const NormParams &p, int sms, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(IO);
    const int64_t gs = p.D / p.G;
    // a CTA holds 16 warps at most, a lane up to 3 vectors (6 of longer groups), or 4 single elements (16)
    const int64_t nvec = p.vec ? gs / V : gs;
    if (nvec <= kMostWarps * 32 * (p.vec ? 6 : 16) && (p.vec || !p.scales)) {
        const int few = p.vec ? 3 : 4, most = nvec <= kMostWarps * 32 * few ? few : p.vec ? 6 : 16;
        const int W = (int)((nvec + 32 * most - 1) / (32 * most));
        const int NV = (int)((nvec + 32 * W - 1) / (32 * W));
        if (p.vec) switch (NV) {
            case 1: return launch_nv<IO, V, 1>(p, W, sms, stream);
            case 2: return launch_nv<IO, V, 2>(p, W, sms, stream);
            case 3: return launch_nv<IO, V, 3>(p, W, sms, stream);
            default: return launch_nv<IO, V, 6>(p, W, sms, stream);
        }
        return NV <= 4 ? launch_nv<IO, 1, 4>(p, W, sms, stream) : launch_nv<IO, 1, 16>(p, W, sms, stream);
    }
    const int64_t grid = std::min<int64_t>(p.rows * p.G, (int64_t)sms * 64);
    norm_long_kernel<IO><<<(unsigned)grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, int io_dtype, int sms, cudaStream_t stream) {
    if (io_dtype == SSD_F32) return launch_t<float>(p, sms, stream);
    if (io_dtype == SSD_BF16) return launch_t<__nv_bfloat16>(p, sms, stream);
    return launch_t<__half>(p, sms, stream);
}

}  // namespace ssd
