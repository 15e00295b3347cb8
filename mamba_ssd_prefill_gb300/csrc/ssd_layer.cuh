// Device helpers of the operators around the SSD (selective scan, convolution by
// itself, group norm, e4m3 projections).
#pragma once

#include <type_traits>

#include "ssd_common.cuh"

namespace ssd {

// a / b and a % b of non-negative numbers; a 64-bit division takes some ten times a 32-bit one.
__device__ __forceinline__ int64_t quick_div(int64_t a, int64_t b, int64_t &rest) {
    if (((a | b) >> 32) == 0) {
        const uint32_t q = (uint32_t)a / (uint32_t)b;
        rest = (uint32_t)a - q * (uint32_t)b;
        return q;
    }
    const int64_t q = a / b;
    rest = a - q * b;
    return q;
}

// Kernels that launch_after launches may start while the one before them in the stream still runs, so that the time it
// takes to start them is hidden (a quantiser and a product of 16 tokens: 9.3 us against 13.4 a pair, a convolution of one
// token 5.9 against 8.1). Each lets the next one start at once, and calls this before it touches memory: it waits until
// the kernels before it are done and all that they wrote is visible. A kernel launched in the ordinary way passes through.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int64_t grid, dim3 threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float v) {  // 2^v, relative error 2^-22
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp(float v) {  // 1 / v, relative error 2^-23; 0 above 2^126
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1]. log(1 + e) is e times a polynomial of degree 8 in e
// (the minimax one of log(1 + e) / e on [0, 1], found by exchange, 6.5e-8 relative), so that the small steps (v around -7)
// that layers learn keep their relative accuracy, which a logarithm of the rounded 1 + e would lose. The relative error is
// at most (1.3 |v| + 8) 2^-24 for v from -87 up to 0, and 8 units above: the exponent's argument |v| log2(e) is rounded
// once, with a rounded constant (1.3 |v| units of e), 2^x has 4 units, the polynomial and its evaluation 4. Below -87 it
// is 0. -inf -> 0, inf -> inf, NaN stays.
__device__ __forceinline__ float softplus_fast(float v) {
    const float e = ex2(fminf(v, -v) * kLog2e);
    float q = fmaf(e, 0.00523269409f, -0.0295052398f);
    q = fmaf(e, q, 0.0782259554f);
    q = fmaf(e, q, -0.136632457f);
    q = fmaf(e, q, 0.191060066f);
    q = fmaf(e, q, -0.24842982f);
    q = fmaf(e, q, 0.333190978f);
    q = fmaf(e, q, -0.499994934f);
    q = fmaf(e, q, 0.99999994f);
    return fmaf(e, q, v < 0.f ? 0.f : v);
}

// v sigmoid(v) in fp32: 8 units of 2^-24 relative for v >= 0, (1.3 |v| + 8) for v < 0 (the exponent's argument, as above);
// 0 below about -88.
__device__ __forceinline__ float silu_f32(float v) { return v * rcp(1.f + ex2(v * -kLog2e)); }

// K consecutive elements as they lie, in registers
template <typename IO, int K> struct Raw {
    static constexpr int W = K * (int)sizeof(IO) < 4 ? 1 : K * (int)sizeof(IO) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    // all K elements; p is aligned for them
    __device__ __forceinline__ void load(const IO *p) {
        if constexpr (K == 1) {
            w[0] = bits(*p);
        } else if constexpr (W == 1) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else if constexpr (W == 2) {
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
    // all K elements, one by one
    __device__ __forceinline__ void load_each(const IO *p) {
        IO e[K];
#pragma unroll
        for (int i = 0; i < K; ++i) e[i] = p[i];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if constexpr (sizeof(IO) == 4) w[i] = bits(e[i]);
            else if (i % 2 == 0) w[i / 2] = bits(e[i]);
            else w[i / 2] |= bits(e[i]) << 16;
        }
    }
    __device__ __forceinline__ void store(IO *p) const {  // all K, 16 bytes at a time
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
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
    __device__ __forceinline__ float2 pair(int i) const {  // elements i and i + 1, i even
        if constexpr (sizeof(IO) == 4) {
            return make_float2(__uint_as_float(w[i]), __uint_as_float(w[i + 1]));
        } else if constexpr (std::is_same<IO, __nv_bfloat16>::value) {
            return make_float2(__uint_as_float(w[i / 2] << 16), __uint_as_float(w[i / 2] & 0xffff0000u));
        } else {
            return __half22float2(*reinterpret_cast<const __half2 *>(&w[i / 2]));
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (K == 1) {
            if constexpr (sizeof(IO) == 4) return __uint_as_float(w[0]);
            const uint16_t h = (uint16_t)w[0];
            return to_f32(*reinterpret_cast<const IO *>(&h));
        }
        const float2 v = pair(i & ~1);
        return i & 1 ? v.y : v.x;
    }
    __device__ __forceinline__ void set_pair(int i, float x, float y) {
        if constexpr (sizeof(IO) == 4) {
            w[i] = __float_as_uint(x), w[i + 1] = __float_as_uint(y);
        } else if constexpr (std::is_same<IO, __nv_bfloat16>::value) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            w[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(x, y);
            w[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}

template <int BYTES> __device__ __forceinline__ void cp_async(void *dst, const void *src) {  // 4 or 8
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "n"(BYTES)
                 : "memory");
}

// Two fp32 fused multiply-adds in one instruction, each rounded like a scalar fmaf.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 pa, pb, pc, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "mov.b64 pc, {%6, %7};\n\tfma.rn.f32x2 pd, pa, pb, pc;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Two values as e4m3 bytes (lo in the low byte), rounded to nearest even, saturating at 448; NaN -> 0x7f.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Scale of a block whose largest magnitude is m (NaN where the block holds a NaN or an infinity), and the factor
// its values are multiplied with. Below m = 1.3e-36 the quotient 448 / m is infinite and the largest finite factor is
// taken instead: such a block comes back too small.
constexpr float kE4m3Max = 448.f;
__device__ __forceinline__ void e4m3_scale(float m, float &scale, float &inv) {
    if (m == 0.f) {
        scale = inv = 1.f;
    } else if (m <= 3.402823466e38f) {
        scale = __fdiv_rn(m, kE4m3Max);
        inv = fminf(__fdiv_rn(kE4m3Max, m), 3.402823466e38f);
    } else {
        scale = inv = __int_as_float(0x7fffffff);
    }
}
// max that keeps a NaN of either side
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// `count` rows of `width` elements `stride` apart, the first at element idx of a buffer of n: their address. The bounds-checked
// builds look at the whole span, and at nothing where there are no rows.
template <typename T>
__device__ __forceinline__ T *chk_rows(T *base, int64_t idx, int64_t count, int64_t stride, int64_t width, int64_t n,
                                       WsHeader *hdr, uint32_t site) {
#ifdef SSD_BOUNDS_CHECK
    return count > 0 && width > 0 ? chk(base, idx, (count - 1) * stride + width, n, hdr, site) : base;
#else
    return base + idx;
#endif
}

// Packed sequences: the token range of sequence s, kept inside [0, T] whatever the offsets hold.
__device__ __forceinline__ void packed_range(const int32_t *cu, int64_t nseq, int64_t s, int64_t T, WsHeader *hdr,
                                             int64_t &begin, int64_t &end) {
    const int32_t *at = chk(cu, s, 2, nseq + 1, hdr, SITE_OFFSETS);
    const int64_t b = at[0], e = at[1];
    begin = b < 0 ? 0 : b > T ? T : b;
    end = e < begin ? begin : e > T ? T : e;
}
// Record malformed offsets (first != 0, last != T, or decreasing). Called by one CTA of a launch.
__device__ __forceinline__ void check_offsets(const int32_t *cu, int64_t nseq, int64_t T, WsHeader *hdr) {
    bool bad = false;
    for (int64_t s = threadIdx.x; s < nseq; s += blockDim.x) bad |= cu[s + 1] < cu[s];
    if (threadIdx.x == 0) bad |= cu[0] != 0 || cu[nseq] != T;
    if (bad && hdr) atomicCAS(&hdr->status, 0u, (uint32_t)DEV_BAD_SEQLENS);
}

}  // namespace ssd
