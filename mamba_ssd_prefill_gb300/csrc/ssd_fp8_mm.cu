// Product of e4m3 matrices with block scales (include/ssd.h):
//
//   out[m, n] = bias[n] + sum_j sa[m, j] sb[n / 128, j] sum_{k in block j} a[m, k] b[n, k]
//
// The inner sums run on the tensor cores (tcgen05.mma, kind f8f6f4: four instructions of K = 32 a block), each block
// into TMEM afresh; the scales differ from block to block, so the outer sum is taken in fp32 registers while the
// tensor cores work on the next block in the other half of TMEM.
//
// Two kernels. wide_kernel: tokens are the 128 rows (TMEM lanes) of a tile, 256 weights its columns; one persistent
// CTA per SM, TMA into four stages of 48 KB, two blocks in TMEM (256 columns each). What bounds it is the turn of a TMEM
// half: MMA (512 clocks), read, FMA and back, so a warp reads 64 columns at a time and gives the half back before it adds
// the last 64 (16 columns at a time 16384 x 10576 x 2560 took 369 us, so 341 to 348: 2.6 PFLOP/s; 16384 x 8192 x 8192:
// 2.9). The tensor pipe is active for 52 % of the time (4096 x 10576 x 2560). In seconds of such products the power limit
// takes the SM clock to 1.75 GHz and the time to 382 us; at that clock a full pipe would take 211.
// fp32 output writes twice the bytes: 563 us with a bias.
// narrow_kernel, for few tokens: weights are the 128 rows and TN tokens the columns, so no row of the tensor core idles;
// K is split over the CTAs of a cluster, whose partial sums are joined through distributed shared memory in rank order
// (no atomics: the result does not depend on timing). 16 x 10576 x 2560: 7.3 us, the weights at 3.7 TB/s.
#include "sm100_ptx.cuh"
#include "ssd_internal.h"
#include "ssd_layer.cuh"

namespace ssd {
namespace {

using namespace sm100;

constexpr int kBK = 128;          // bytes (= elements) of K per stage: one scale block, one 128-byte swizzle row
constexpr uint32_t kTileA = 128 * kBK;

// D[tmem] (+)= A[smem] B[smem], e4m3 operands (format 0 in the instruction descriptor), fp32 accumulation, K = 32
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Wait for the TMEM loads before it; the registers they fill pass through, so no use of them moves above it.
__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
// Warp-collective: 64 consecutive columns of the calling warp's TMEM lanes.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
          "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
          "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait64(uint32_t (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]),
                   "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]), "+r"(r[40]), "+r"(r[41]), "+r"(r[42]),
                   "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]), "+r"(r[48]), "+r"(r[49]),
                   "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]), "+r"(r[56]),
                   "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
                 :
                 : "memory");
}
// acc += s * r, C columns
template <int C> __device__ __forceinline__ void add_scaled(float *acc, const uint32_t (&r)[C], float2 s) {
#pragma unroll
    for (int j = 0; j < C; j += 2) {
        const float2 v = fma2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), s,
                              make_float2(acc[j], acc[j + 1]));
        acc[j] = v.x;
        acc[j + 1] = v.y;
    }
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}

// Bounded wait on a barrier's phase; on timeout it records SSD_ERR_DEVICE and raises the CTA's abort flag, after which
// every other wait of the CTA gives up at once.
__device__ __forceinline__ bool mm_wait_slow(uint64_t *bar, uint32_t parity, int32_t *abort_flag, WsHeader *hdr) {
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 0; it < kMaxSpinIters; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 15u) == 15u) {
            if (*reinterpret_cast<volatile int32_t *>(abort_flag)) return false;
            if (globaltimer() - t0 > kDefaultTimeoutNs) break;
        }
    }
    *reinterpret_cast<volatile int32_t *>(abort_flag) = 1;
    if (atomicCAS(&hdr->status, 0u, (uint32_t)DEV_PIPE) == 0u) hdr->err_where = WAIT_PIPE;
    return false;
}
__device__ __forceinline__ bool mm_wait(uint64_t *bar, uint32_t parity, int32_t *abort_flag, WsHeader *hdr) {
    return mbar_try_wait(bar, parity) || mm_wait_slow(bar, parity, abort_flag, hdr);
}
// After an early stop: the copies still in flight land before the CTA exits (bounded).
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 < 100000000ull) {
    }
}

template <typename OUT> __device__ __forceinline__ uint4 pack16(const float *v);  // 16 bytes of OUT
template <> __device__ __forceinline__ uint4 pack16<float>(const float *v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <> __device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <> __device__ __forceinline__ uint4 pack16<__half>(const float *v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------------------------------------ wide_kernel

constexpr int kWS = 4;                        // stages
constexpr uint32_t kWTileB = 256 * kBK;
constexpr uint32_t kWStage = kTileA + kWTileB;
// Warp 0 copies, warp 1 issues MMAs, warps 4 .. 11 hold the sums (128 fp32 a thread) and write the output. At launch a
// thread has 168 registers (384 x 168 = 64512); the first four warps give up what the sums need:
// 128 x 40 + 256 x 232 = 64512.
constexpr int kWThreads = 384;

struct WideBars {
    uint64_t full[kWS], empty[kWS], tfull[2], tempty[2], drained;
    uint32_t tmem;
    int32_t abort;
};

struct Tile {
    int64_t m0, n0;
};
// Tiles in bands of 16 row tiles, row tiles fastest: the tiles that run side by side share A and B in L2.
__device__ __forceinline__ Tile wide_tile(int64_t t, int64_t mt, int64_t nt) {
    constexpr int64_t kBand = 16;
    const int64_t band = t / (kBand * nt), rest = t % (kBand * nt);
    const int64_t h = mt - band * kBand < kBand ? mt - band * kBand : kBand;
    return Tile{(band * kBand + rest % h) * 128, rest / h * 256};
}

template <typename OUT>
__global__ void __launch_bounds__(kWThreads, 1)
    wide_kernel(MatmulParams p, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_o, int vec) {
    extern __shared__ uint8_t dyn[];
    __shared__ WideBars sm;
    uint8_t *stages = dyn + (1024 - (smem_u32(dyn) & 1023)) % 1024;
    uint8_t *outbuf = stages + kWS * kWStage;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t mt = (p.m + 127) / 128, nt = (p.n + 255) / 256, tiles = mt * nt;
    const int nkb = (int)((p.k + kBK - 1) / kBK);
    WsHeader *hdr = p.hdr;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWS; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.tfull[i], 1);
            mbar_init(&sm.tempty[i], 8);
        }
        mbar_init(&sm.drained, 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    after_previous();

    if (warp >= 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        // TMEM lanes 32 (warp % 4) .., columns 128 half ..
        const int q = warp % 4, half = (warp - 4) / 4;
        uint8_t *buf = outbuf + (warp - 4) * 4096;
        uint32_t i = 0;
        bool ok = true;
        const int64_t nsb = (p.n + 127) / 128;
        for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            const Tile tl = wide_tile(t, mt, nt);
            const int64_t m = tl.m0 + q * 32 + lane, n0 = tl.n0 + half * 128;
            const bool live = m < p.m && n0 / 128 < nsb;
            const float *sa = chk(p.sa, live ? m * nkb : 0, nkb, p.m * nkb, hdr, SITE_FP8_SCALE);
            const float *sb = chk(p.sb, live ? n0 / 128 * nkb : 0, nkb, nsb * nkb, hdr, SITE_FP8_SCALE);
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            float va = live ? sa[0] : 0.f, vb = live ? sb[0] : 0.f;
            for (int kb = 0; kb < nkb; ++kb, ++i) {
                const float s = va * vb;
                if (kb + 1 < nkb && live) {  // the next block's, under this one's wait
                    va = sa[kb + 1];
                    vb = sb[kb + 1];
                }
                const uint32_t ts = i & 1;
                if (!mm_wait(&sm.tfull[ts], (i >> 1) & 1, &sm.abort, hdr)) ok = false;
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = tmem + ts * 256 + half * 128 + ((uint32_t)(q * 32) << 16);
                const float2 s2 = make_float2(s, s);
                uint32_t r[64];
                tmem_ld64(at, r);
                tmem_ld_wait64(r);
                add_scaled(&acc[0], r, s2);
                tmem_ld64(at + 64, r);
                tmem_ld_wait64(r);
                tc_fence_before();  // this warp has read the block
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.tempty[ts]);
                add_scaled(&acc[64], r, s2);
            }
            if (!ok) break;
            // Out of registers through a 4 KB buffer of the warp (rows of 128 bytes, 16-byte pieces swizzled as a TMA
            // store expects them); rows and columns past the end are clipped by the store. Rows that are no 16-byte
            // multiples are stored piece by piece.
            constexpr int E = 16 / (int)sizeof(OUT), CW = 8 * E;  // elements of a piece, of a row of the buffer
#pragma unroll
            for (int c = 0; c < 128 / CW; ++c) {
                if (p.bias)
#pragma unroll
                    for (int j = 0; j < CW; ++j)
                        if (n0 + c * CW + j < p.n)
                            acc[c * CW + j] += *chk(p.bias, n0 + c * CW + j, 1, p.n, hdr, SITE_WEIGHT);
                if (vec) {  // the store before this one has read the buffer
                    if (lane == 0) bulk_wait_read0();
                    __syncwarp();
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((j ^ (lane & 7)) * 16)) =
                        pack16<OUT>(&acc[c * CW + j * E]);
                if (vec) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && n0 + c * CW < p.n && tl.m0 + q * 32 < p.m) {
                        tma_store_2d(&map_o, buf, (int)(n0 + c * CW), (int)(tl.m0 + q * 32));
                        bulk_commit();
                    }
                    continue;
                }
                __syncwarp();
#pragma unroll 1
                for (int u = 0; u < 8; ++u) {
                    const int r = u * 4 + lane / 8, j = lane % 8;
                    const int64_t row = tl.m0 + q * 32 + r, col = n0 + c * CW + j * E;
                    const uint4 w = *reinterpret_cast<const uint4 *>(buf + r * 128 + ((j ^ (r & 7)) * 16));
                    if (row < p.m && col < p.n) {
                        const int64_t left = p.n - col;
                        OUT *o = chk(static_cast<OUT *>(p.out), row * p.out_row + col, left < E ? left : E,
                                     (p.m - 1) * p.out_row + p.n, hdr, SITE_FP8_OUT);
                        const OUT *e = reinterpret_cast<const OUT *>(&w);
#pragma unroll
                        for (int x = 0; x < E; ++x)
                            if (x < left) o[x] = e[x];
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0) bulk_wait0();
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0 && lane == 0) {
            prefetch_tensormap(&map_a);
            prefetch_tensormap(&map_b);
            uint32_t i = 0;  // stages filled
            bool ok = true;
            for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile tl = wide_tile(t, mt, nt);
                for (int kb = 0; kb < nkb; ++kb, ++i) {
                    const uint32_t st = i % kWS;
                    if (!mm_wait(&sm.empty[st], ((i / kWS) & 1) ^ 1, &sm.abort, hdr)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sm.full[st], kWStage);
                    tma_load_2d(stages + st * kWStage, &map_a, &sm.full[st], kb * kBK, (int)tl.m0);
                    tma_load_2d(stages + st * kWStage + kTileA, &map_b, &sm.full[st], kb * kBK, (int)tl.n0);
                }
            }
            for (uint32_t j = 0; j < (uint32_t)kWS && j < i; ++j)
                drain(&sm.full[(i - 1 - j) % kWS], ((i - 1 - j) / kWS) & 1);
        }
        if (warp == 1) {
        constexpr uint32_t id = idesc_f16_f32(128, 256, false, false);  // format fields 0: e4m3 under f8f6f4
        const bool leader = elect_one();
        uint32_t i = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            for (int kb = 0; kb < nkb; ++kb, ++i) {
                const uint32_t st = i % kWS, ts = i & 1;
                if (!mm_wait(&sm.tempty[ts], ((i >> 1) & 1) ^ 1, &sm.abort, hdr) ||
                    !mm_wait(&sm.full[st], (i / kWS) & 1, &sm.abort, hdr)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (leader) {
                    const uint64_t da = desc_sw128(smem_u32(stages + st * kWStage), 16, 1024);
                    const uint64_t db = desc_sw128(smem_u32(stages + st * kWStage + kTileA), 16, 1024);
#pragma unroll
                    for (uint32_t s = 0; s < 4; ++s) mma_f8(tmem + ts * 256, da + 2 * s, db + 2 * s, id, s > 0);
                    mma_commit(&sm.empty[st]);
                    mma_commit(&sm.tfull[ts]);
                }
                __syncwarp();
            }
        }
        if (leader) {  // every MMA has completed before TMEM is released
            mma_commit(&sm.drained);
            drain(&sm.drained, 0);
        }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------------------------- narrow_kernel

constexpr int kNThreads = 192;       // TMA warp, MMA warp, 4 warps for the sums and the output
constexpr int kNScales = 3840;       // products of scales held by a CTA (TN tokens x its blocks of K); two CTAs fit an SM
constexpr uint32_t kNRing = 96 * 1024;

template <int TN> struct Narrow {
    static constexpr uint32_t kStage = kTileA + TN * kBK;
    static constexpr int kStages = (int)(kNRing / kStage) < 6 ? (int)(kNRing / kStage) : 6;
    static constexpr uint32_t kCols = 2 * TN < 32 ? 32 : 2 * TN;
    static constexpr uint32_t kDyn = kStages * kStage + 4 * kNScales + 1024;
    static_assert(TN * 128 * 4 <= kStages * kStage, "the partial sums fit the stages");
};

struct NarrowBars {
    uint64_t full[6], empty[6], tfull[2], tempty[2], drained;
    uint32_t tmem;
    int32_t abort;
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [ra];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// Grid: x = weight tiles x splits (a cluster holds the splits of one tile), y = token tiles.
template <typename OUT, int TN>
__global__ void __launch_bounds__(kNThreads)
    narrow_kernel(MatmulParams p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_t,
                  int splits, int vec) {
    using T = Narrow<TN>;
    extern __shared__ uint8_t dyn[];
    __shared__ NarrowBars sm;
    uint8_t *stages = dyn + (1024 - (smem_u32(dyn) & 1023)) % 1024;
    float *scales = reinterpret_cast<float *>(stages + T::kStages * T::kStage);
    float *part = reinterpret_cast<float *>(stages);  // [TN][128], once the last block has been read
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)(blockIdx.x % splits);
    const int64_t w0 = (int64_t)(blockIdx.x / splits) * 128, m0 = (int64_t)blockIdx.y * TN;
    const int nkb = (int)((p.k + kBK - 1) / kBK);
    const int kb0 = (int)((int64_t)nkb * rank / splits), kb1 = (int)((int64_t)nkb * (rank + 1) / splits);
    WsHeader *hdr = p.hdr;
    if (threadIdx.x == 0) {
        for (int i = 0; i < T::kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.tfull[i], 1);
            mbar_init(&sm.tempty[i], 4);
        }
        mbar_init(&sm.drained, 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem, T::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    after_previous();

    if (warp == 0) {
        if (lane == 0) {
            uint32_t i = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++i) {
                const uint32_t st = i % T::kStages;
                if (!mm_wait(&sm.empty[st], ((i / T::kStages) & 1) ^ 1, &sm.abort, hdr)) break;
                mbar_arrive_expect_tx(&sm.full[st], T::kStage);
                tma_load_2d(stages + st * T::kStage, &map_w, &sm.full[st], kb * kBK, (int)w0);
                tma_load_2d(stages + st * T::kStage + kTileA, &map_t, &sm.full[st], kb * kBK, (int)m0);
            }
            for (uint32_t j = 0; j < (uint32_t)T::kStages && j < i; ++j)
                drain(&sm.full[(i - 1 - j) % T::kStages], ((i - 1 - j) / T::kStages) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t id = idesc_f16_f32(128, TN, false, false);
        const bool leader = elect_one();
        uint32_t i = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++i) {
            const uint32_t st = i % T::kStages, ts = i & 1;
            if (!mm_wait(&sm.tempty[ts], ((i >> 1) & 1) ^ 1, &sm.abort, hdr) ||
                !mm_wait(&sm.full[st], (i / T::kStages) & 1, &sm.abort, hdr))
                break;
            tc_fence_after();
            if (leader) {
                const uint64_t da = desc_sw128(smem_u32(stages + st * T::kStage), 16, 1024);
                const uint64_t db = desc_sw128(smem_u32(stages + st * T::kStage + kTileA), 16, 1024);
#pragma unroll
                for (uint32_t s = 0; s < 4; ++s) mma_f8(tmem + ts * TN, da + 2 * s, db + 2 * s, id, s > 0);
                mma_commit(&sm.empty[st]);
                mma_commit(&sm.tfull[ts]);
            }
            __syncwarp();
        }
        if (leader) {
            mma_commit(&sm.drained);
            drain(&sm.drained, 0);
        }
        __syncwarp();
    } else {
        // warps 2 .. 5: weight rows 32 (warp % 4) .., all TN tokens
        const int q = warp % 4, tid = threadIdx.x - 64;
        for (int e = tid; e < (kb1 - kb0) * TN; e += 128) {
            const int j = e % TN, kb = kb0 + e / TN;
            scales[e] = m0 + j < p.m
                            ? *chk(p.sa, (m0 + j) * nkb + kb, 1, p.m * nkb, hdr, SITE_FP8_SCALE) *
                                  *chk(p.sb, w0 / 128 * nkb + kb, 1, (p.n + 127) / 128 * nkb, hdr, SITE_FP8_SCALE)
                            : 0.f;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        float2 acc[TN / 2];
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) acc[j] = make_float2(0.f, 0.f);
        uint32_t i = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb, ++i) {
            const uint32_t ts = i & 1;
            if (!mm_wait(&sm.tfull[ts], (i >> 1) & 1, &sm.abort, hdr)) ok = false;
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t at = tmem + ts * TN + ((uint32_t)(q * 32) << 16);
            const float4 *s4 = reinterpret_cast<const float4 *>(scales + (kb - kb0) * TN);
            uint32_t r[2][16];
            tmem_ld16(at, r[0]);
#pragma unroll
            for (int c = 0; c < TN / 16; ++c) {
                tmem_ld_wait16(r[c & 1]);
                if (c < TN / 16 - 1) tmem_ld16(at + 16 * (c + 1), r[(c + 1) & 1]);
                else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.tempty[ts]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 s = s4[c * 4 + j];
                    float2 *a = acc + c * 8 + j * 2;
                    const uint32_t *v = r[c & 1] + 4 * j;
                    a[0] = fma2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), make_float2(s.x, s.y), a[0]);
                    a[1] = fma2(make_float2(__uint_as_float(v[2]), __uint_as_float(v[3])), make_float2(s.z, s.w), a[1]);
                }
            }
        }
        // every block's MMAs have been waited for, so the stages are free
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) {
            part[(2 * j) * 128 + q * 32 + lane] = acc[j].x;
            part[(2 * j + 1) * 128 + q * 32 + lane] = acc[j].y;
        }
    }
    // the splits' sums, joined in rank order: each CTA takes every splits-th token
    if (splits > 1) cluster_sync();
    else __syncthreads();
    if (warp >= 2) {
        const int64_t n = w0 + lane * 4;
        for (int j = rank + (warp - 2) * splits; j < TN; j += 4 * splits) {
            if (m0 + j >= p.m) break;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (splits > 1) {
                for (int r = 0; r < splits; ++r) {
                    const float4 u = ld_cluster4(smem_u32(part + j * 128 + lane * 4), (uint32_t)r);
                    v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                }
            } else {
                v = *reinterpret_cast<const float4 *>(part + j * 128 + lane * 4);
            }
            float o[4] = {v.x, v.y, v.z, v.w};
            if (n >= p.n) continue;
            const int left = (int)(p.n - n < 4 ? p.n - n : 4);
            if (p.bias)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (x < left) o[x] += *chk(p.bias, n + x, 1, p.n, hdr, SITE_WEIGHT);
            OUT *out = chk(static_cast<OUT *>(p.out), (m0 + j) * p.out_row + n, left, (p.m - 1) * p.out_row + p.n, hdr,
                           SITE_FP8_OUT);
            if (vec && left == 4) {
                if constexpr (sizeof(OUT) == 4) {
                    *reinterpret_cast<float4 *>(out) = make_float4(o[0], o[1], o[2], o[3]);
                } else {
                    OUT h[4] = {from_f32<OUT>(o[0]), from_f32<OUT>(o[1]), from_f32<OUT>(o[2]), from_f32<OUT>(o[3])};
                    *reinterpret_cast<uint2 *>(out) = *reinterpret_cast<const uint2 *>(h);
                }
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (x < left) out[x] = from_f32<OUT>(o[x]);
            }
        }
    }
    tc_fence_before();
    if (splits > 1) cluster_sync();  // no CTA leaves while its sums are being read
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, T::kCols);
    }
}

// k = 0: the bias, or zeros
template <typename OUT>
__global__ void __launch_bounds__(256) bias_kernel(MatmulParams p) {
    after_previous();
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < p.m * p.n; e += (int64_t)gridDim.x * 256)
        *chk(static_cast<OUT *>(p.out), e / p.n * p.out_row + e % p.n, 1, (p.m - 1) * p.out_row + p.n, p.hdr,
             SITE_FP8_OUT) = from_f32<OUT>(p.bias ? *chk(p.bias, e % p.n, 1, p.n, p.hdr, SITE_WEIGHT) : 0.f);
}

// 2-D map over [rows, k] bytes, box [box_rows, 128 bytes], 128-byte swizzle, zeros outside
bool byte_map(CUtensorMap *map, const uint8_t *base, int64_t rows, int64_t k, int box_rows) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)k};
    const cuuint32_t box[2] = {kBK, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename OUT>
cudaError_t launch_wide(const MatmulParams &p, int sms, cudaStream_t stream) {
    CUtensorMap ma, mb;
    if (!byte_map(&ma, p.a, p.m, p.k, 128) || !byte_map(&mb, p.b, p.n, p.k, 256)) return cudaErrorInvalidValue;
    const int64_t tiles = ((p.m + 127) / 128) * ((p.n + 255) / 256);
    const size_t smem = kWS * kWStage + 8 * 4096 + 1024;
    auto k = wide_kernel<OUT>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k, smem, done);
    if (e != cudaSuccess) return e;
    // output map [m, n], box [32, 128 bytes], where rows lie on 16-byte boundaries and are made of whole 16-byte pieces: a TMA
    // store clips by pieces, and wrote the rest of a last one over what lies behind column n of wider rows
    int vec = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_row * sizeof(OUT)) |
                (uintptr_t)(p.n * sizeof(OUT))) & 15) == 0;
    CUtensorMap mo = ma;
    if (vec) {
        const cuuint64_t dims[2] = {(cuuint64_t)p.n, (cuuint64_t)p.m};
        const cuuint64_t strides[1] = {(cuuint64_t)(p.m > 1 ? p.out_row * sizeof(OUT) : (p.n * sizeof(OUT) + 15) / 16 * 16)};
        const cuuint32_t box[2] = {128 / (cuuint32_t)sizeof(OUT), 32};
        const cuuint32_t estr[2] = {1, 1};
        const CUtensorMapDataType dt = sizeof(OUT) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                       : std::is_same<OUT, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        if (strides[0] >> 40 ||
            encode_tiled_fn()(&mo, dt, 2, p.out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            vec = 0;
    }
    // Many waves start once the kernel before has ended: started as its CTAs leave, the CTAs of neighbouring tiles land on
    // SMs apart (quantiser and product, 16384 x 2560 x 10576, 35 waves: 410 us against 401; 8191 x 5120 x 2560 behind the
    // norm, four waves: 157 against 160). Nothing was measured between the two; the switch stands at twice the smaller.
    if (tiles < (int64_t)sms * 8) return launch_after(k, std::min<int64_t>(tiles, sms), kWThreads, smem, stream, p, ma, mb, mo, vec);
    k<<<(unsigned)sms, kWThreads, smem, stream>>>(p, ma, mb, mo, vec);
    return cudaGetLastError();
}

template <typename OUT, int TN>
cudaError_t launch_narrow(const MatmulParams &p, int splits, cudaStream_t stream) {
    CUtensorMap mw, mt;
    if (!byte_map(&mw, p.b, p.n, p.k, 128) || !byte_map(&mt, p.a, p.m, p.k, TN)) return cudaErrorInvalidValue;
    auto k = narrow_kernel<OUT, TN>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(k, Narrow<TN>::kDyn, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.n + 127) / 128 * splits), (unsigned)((p.m + TN - 1) / TN));
    cfg.blockDim = dim3(kNThreads);
    cfg.dynamicSmemBytes = Narrow<TN>::kDyn;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const size_t align = 4 * sizeof(OUT);
    const int vec = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_row * sizeof(OUT))) & (align - 1)) == 0;
    e = cudaLaunchKernelEx(&cfg, k, p, mw, mt, splits, vec);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// The kernel and split whose estimated time is least, in nanoseconds. Measured on 16 sizes (1 .. 1024 tokens, K 640 ..
// 8192, 640 .. 10576 outputs), each kernel and split forced in turn: a wave of the wide kernel takes 2.2 us and 0.375 a
// block of K; a narrow CTA 1.6 us and 0.17, 0.24, 0.34 or 0.6 a block for 16 .. 128 tokens, half as much again where two
// share an SM; the estimate then picks the fastest or one within 8 % of it (256 x 2560 x 5120: 64 tokens in 2 splits
// 16.1 us, 128 in 4 15.4, wide 20.0; 128 x 10576 x 2560: wide 12.9, 64 tokens 15.3).
struct Choice {
    int tn, splits;  // tn 0: wide
};
Choice choose(const MatmulParams &p, int sms) {
    const int64_t nkb = (p.k + kBK - 1) / kBK;
    const int64_t waves = (((p.m + 127) / 128) * ((p.n + 255) / 256) + sms - 1) / sms;
    Choice best{0, 1};
    double least = 2000.0 + (double)waves * (2200.0 + 375.0 * (double)nkb);
    const double block_ns[4] = {170, 240, 340, 600}, shared[4] = {1.2, 1.5, 1.4, 1.75};
    for (int i = 0, tn = 16; tn <= 128; ++i, tn *= 2) {
        const int64_t mt = (p.m + tn - 1) / tn, tiles = mt * ((p.n + 127) / 128);
        if (mt > 65535) continue;
        for (int splits = 1; splits <= 8; splits *= 2) {
            if (splits > 1 && splits * 2 > nkb) break;
            const int64_t blocks = (nkb + splits - 1) / splits;
            if (blocks * tn > kNScales || tiles * splits > (1 << 30)) continue;
            const int64_t on_sm = (tiles * splits + sms - 1) / sms;  // CTAs an SM gets, two at a time
            const double t = 3000.0 + (splits > 1 ? 500.0 + 100.0 * splits : 0.0) +
                             (double)((on_sm + 1) / 2) *
                                 (1600.0 + block_ns[i] * (double)blocks * (on_sm > 1 ? shared[i] : 1.0));
            if (t < least) {
                least = t;
                best = Choice{tn, splits};
            }
        }
    }
    return best;
}

std::atomic<int> forced_tile{-1}, forced_splits{-1};  // ssd_debug_product; -1: the library's own choice
bool runs(const MatmulParams &p, Choice c) {  // whether a forced choice holds the problem
    if (c.tn == 0) return c.splits == 1;
    const int64_t nkb = (p.k + kBK - 1) / kBK, mt = (p.m + c.tn - 1) / c.tn;
    return c.splits <= nkb && (nkb + c.splits - 1) / c.splits * c.tn <= kNScales && mt <= 65535 &&
           mt * ((p.n + 127) / 128) * c.splits <= (1 << 30);
}

template <typename OUT>
cudaError_t launch_t(const MatmulParams &p, int sms, cudaStream_t stream) {
    if (p.k == 0) {
        return launch_after(bias_kernel<OUT>, std::min<int64_t>((p.m * p.n + 255) / 256, (int64_t)sms * 8), 256, 0, stream,
                            p);
    }
    const Choice forced{forced_tile.load(std::memory_order_relaxed), forced_splits.load(std::memory_order_relaxed)};
    if (forced.tn >= 0 && !runs(p, forced)) return cudaErrorNotSupported;
    const Choice c = forced.tn >= 0 ? forced : choose(p, sms);
    switch (c.tn) {
        case 16: return launch_narrow<OUT, 16>(p, c.splits, stream);
        case 32: return launch_narrow<OUT, 32>(p, c.splits, stream);
        case 64: return launch_narrow<OUT, 64>(p, c.splits, stream);
        case 128: return launch_narrow<OUT, 128>(p, c.splits, stream);
        default: return launch_wide<OUT>(p, sms, stream);
    }
}

}  // namespace

bool force_product(int token_tile, int splits) {
    const bool own = token_tile == -1 && splits == -1;
    const bool narrow = (token_tile == 16 || token_tile == 32 || token_tile == 64 || token_tile == 128) &&
                        (splits == 1 || splits == 2 || splits == 4 || splits == 8);
    if (!own && !narrow && !(token_tile == 0 && splits == 1)) return false;
    forced_splits.store(splits, std::memory_order_relaxed);
    forced_tile.store(token_tile, std::memory_order_relaxed);
    return true;
}

cudaError_t launch_matmul(const MatmulParams &p, int out_dtype, int sms, cudaStream_t stream) {
    if (out_dtype == SSD_F32) return launch_t<float>(p, sms, stream);
    if (out_dtype == SSD_BF16) return launch_t<__nv_bfloat16>(p, sms, stream);
    return launch_t<__half>(p, sms, stream);
}

}  // namespace ssd
