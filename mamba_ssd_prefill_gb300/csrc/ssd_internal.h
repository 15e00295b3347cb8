// Host-side interfaces between the C ABI (ssd_api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "../../include/ssd.h"
#include "ssd_common.cuh"

namespace ssd {

// Workspace bytes of a regular batch with or without two-level state passing (ssd_api.cu).
ssd_status_t workspace_bytes(const ssd_problem_t *prob, bool segments, size_t *bytes);

// cuTensorMapEncodeTiled, looked up once through the runtime's driver entry points (ssd_api.cu); null when the
// driver has none
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled_fn();

// Launch-configuration overrides set by ssd_debug_knobs (test hooks; -1 = the library's own choice).
struct Knobs {
    int tc_heads_per_unit, tc_late_ticket, simt_two_pass, conv_tma;
    int tc_segment_chunks;  // -1: the library's choice, 0: one state chain per sequence, >= 1: chunks per segment
    int tc_head_flags;      // -1: the library's choice, 0: a release flag per state row, 1: one per head
};
Knobs knobs();

// fp32 SIMT kernel (ssd_simt.cu)
size_t simt_smem_bytes(int64_t P, int64_t N);
cudaError_t launch_simt(const Params &p, int io_dtype, int state_dtype, int sms, cudaStream_t stream);

// variable-length batches (ssd_varlen.cu): chunk table from cu_seqlens, final = initial for empty sequences
cudaError_t launch_varlen_plan(const Params &p, uint32_t *scratch, size_t state_bytes, cudaStream_t stream);

// causal depthwise convolution in front of the SSD (ssd_conv.cu)
cudaError_t launch_conv(const ConvParams &c, int io_dtype, int sms, cudaStream_t stream);

// single-token step (ssd_step.cu)
cudaError_t launch_step(const Params &p, int io_dtype, int state_dtype, int sms, cudaStream_t stream);

// tcgen05 / TMA kernel (ssd_tc.cu)
bool tc_supports(int64_t P, int64_t N, int64_t Q, int io_dtype);
int64_t tc_chunk();  // tokens per state-passing step inside the tensor-core kernel
size_t tc_flag_bytes(int64_t chains);
size_t tc_ring_bytes(int64_t chains, int64_t P, int64_t N, int state_dtype);
uint32_t tc_total_units(int64_t batch, int64_t H, int64_t G, int64_t nc, int heads_per_unit);
int tc_heads_per_unit(int64_t batch, int64_t H, int64_t G, int64_t nc, int sms);
bool tc_late_ticket(int64_t units_per_chunk, int sms);  // ticket order = finishing order (chain-bound problems)
bool tc_head_flags(int64_t chains_per_position, bool late_ticket, int sms);  // fp32 states: one release per head
cudaError_t launch_tc(Params p, int io_dtype, int state_dtype, int heads_per_unit, int sms, cudaStream_t stream);

// two-level state passing (ssd_segstate.cu): segment entering states from block aggregates, before launch_tc
struct SegChoice {
    int64_t nseg, seg_chunks;  // segments per sequence (1: off) and chunks per segment
    int64_t blk, nblk;         // chunks per aggregate block, blocks per sequence with an aggregate
    int hs;                    // heads per block-kernel work unit
};
SegChoice choose_segments(int64_t nseq, int64_t nc, int64_t H, int64_t G, int sms, int64_t forced, bool fp32_states);
struct SegPlan {
    int64_t blk, nblk;
    int hs;
    float *blk_s;  // [nseq][nblk][H][P][N] block aggregates
    float *blk_L;  // [nseq][nblk][H] log2 of the block decays
};
cudaError_t launch_segstate(const Params &p, const SegPlan &sp, int io_dtype, int state_dtype, int sms,
                            cudaStream_t stream);

// ---- the operators around the SSD (ssd_layer_api.cu checks their arguments) ----

int device_sms();  // SM count of the current device, 0 when it cannot be read (ssd_api.cu)

// Lets `kernel` take `bytes` of dynamic shared memory on the current device; asked of the driver once per device
// (`done`: a mask of the devices that have it, one per kernel).
template <typename K> cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Packed or regular sequences of T tokens in all; strides in elements.
struct ScanParams {
    const void *x, *dt, *z, *B, *C;
    void *y;
    const float *A, *dt_bias, *D;
    const void *init;
    void *fin;
    const int32_t *cu;  // packed: [nseq + 1]; null for a regular batch
    WsHeader *hdr;
    int64_t nseq, L, T, D_, N, G, cpg;  // L: tokens of a sequence (packed: T); cpg: channels per group
    int64_t x_seq, x_tok, dt_seq, dt_tok, z_seq, z_tok, b_seq, b_tok, c_seq, c_tok, y_seq, y_tok;
    int softplus, state_f16;
    int unit;                // bytes that x, dt, z and y are copied by: 16, 8, 4, or 0 (single elements)
    int vec_bc, vec_state;   // 4-state vectors of B and C, and of states are aligned
    int64_t rows;                // leading dimension of the token tensors (packed: 1)
    // segments of seg_len tokens: nseg per sequence, packed: of the packed axis; the leaving states [seg_items, D, N] and
    // summed dt [seg_items, D] of all but each last one
    int64_t nseg, seg_len, seg_items;
    float *seg_state, *seg_dt;
};
// Channels and threads of a scan CTA, and the CTAs that an SM holds by their registers (of them where rows are copied by
// single elements), by the number of states (the shapes in ssd_selscan.cuh). Shared memory holds fewer in one case: fp32
// rows with up to 4 states have 20 KB a CTA and 11 of them, so the planner's wave of 16 is 1.45 there.
struct ScanCta {
    int channels, threads, resident, resident_single;
};
inline ScanCta scan_cta(int64_t N) {
    if (N <= 4) return {128, 32, 16, 12};
    if (N <= 8) return {128, 64, 8, 7};
    if (N <= 16) return {128, 128, 5, 4};
    if (N <= 24) return {128, 128, 4, 3};
    if (N <= 32) return {128, 256, 2, 1};
    return {N <= 64 ? 64 : N <= 128 ? 32 : 16, 256, 2, 1};
}
// ssd_selscan.cuh, one translation unit per type
cudaError_t launch_scan_f32(const ScanParams &p, cudaStream_t stream);
cudaError_t launch_scan_bf16(const ScanParams &p, cudaStream_t stream);
cudaError_t launch_scan_f16(const ScanParams &p, cudaStream_t stream);

struct RowConvParams {
    const void *x;
    void *out;
    const float *w, *bias;
    const void *state;
    void *state_out;
    const int32_t *cu;
    WsHeader *hdr;  // may be null
    int64_t nseq, L, T, D;
    int64_t x_seq, x_tok, out_seq, out_tok;
    int k, silu;
    int unit;              // bytes that rows of x and out are copied by: 16, 4, or 0 (single elements)
    int vec_state, vec_w;  // the cache left behind, and the taps lie on 16-byte boundaries
    int64_t rows;          // leading dimension of x and out (packed: 1)
};
cudaError_t launch_row_conv(const RowConvParams &p, int io_dtype, int sms, cudaStream_t stream);

struct NormParams {
    const void *x, *z;
    void *y;
    float *scales;
    const float *w, *bias;
    WsHeader *hdr;  // may be null
    int64_t rows, D, G, x_row, z_row, y_row;
    int center, gate_first, silu;
    int unit;  // bytes of the aligned pieces that every group of x, z and y is made of: 16, 4 (16-bit types), or 0
    float eps;
};
// ssd_norm.cuh, one translation unit per type
cudaError_t launch_norm_f32(const NormParams &p, int sms, cudaStream_t stream);
cudaError_t launch_norm_bf16(const NormParams &p, int sms, cudaStream_t stream);
cudaError_t launch_norm_f16(const NormParams &p, int sms, cudaStream_t stream);

struct QuantParams {
    const void *x;
    uint8_t *q;
    float *scales;
    WsHeader *hdr;  // may be null
    int64_t rows, cols, x_row;
    int block_rows;
    int vec;  // 8-element pieces of x and q are aligned
};
cudaError_t launch_quantize(const QuantParams &p, int io_dtype, int sms, cudaStream_t stream);

struct MatmulParams {
    const uint8_t *a, *b;
    const float *sa, *sb, *bias;
    void *out;
    WsHeader *hdr;
    int64_t m, n, k, out_row;
};
// cudaErrorNotSupported: the forced kernel and split (ssd_debug_product) do not run this problem
cudaError_t launch_matmul(const MatmulParams &p, int out_dtype, int sms, cudaStream_t stream);
bool force_product(int token_tile, int splits);  // false: no such kernel

}  // namespace ssd
