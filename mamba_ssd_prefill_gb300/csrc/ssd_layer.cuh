// Device helpers of the operators around the SSD (selective scan, convolution by
// itself, group norm, e4m3 projections).
#pragma once

#include "ssd_common.cuh"

namespace ssd {

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
// (the minimax one of log(1 + e) / e on [0, 1], found by exchange, 3e-8 relative): a few ulp relative wherever v is,
// which a logarithm of the rounded 1 + e would lose for the small steps (v around -7) that layers learn.
// -inf -> 0, inf -> inf, NaN stays.
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

// v sigmoid(v) in fp32 (a few ulp; 0 below about -88).
__device__ __forceinline__ float silu_f32(float v) { return v * rcp(1.f + ex2(v * -kLog2e)); }

// Two values as e4m3 bytes (lo in the low byte), rounded to nearest even, saturating at 448; NaN -> 0x7f.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Scale of a block whose largest magnitude is m (NaN where the block holds a NaN or an infinity), and the factor
// its values are multiplied with. A subnormal m would make 448 / m infinite: the largest finite factor is taken.
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

// Packed sequences: the token range of sequence s, kept inside [0, T] whatever the offsets hold.
__device__ __forceinline__ void packed_range(const int32_t *cu, int64_t s, int64_t T, int64_t &begin, int64_t &end) {
    const int64_t b = cu[s], e = cu[s + 1];
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
