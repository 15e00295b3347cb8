// The C ABI of the operators around the SSD (declared in include/ssd.h):
// argument checks and launches of the selective scan, the depthwise
// convolution by itself, the group norm and the e4m3 projections. Host code only.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/ssd.h"
#include "ssd_internal.h"

namespace {

using ssd::WsHeader;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t elem_size(int dt) { return dt == SSD_F32 ? 4 : 2; }
bool io_ok(int dt) { return dt == SSD_F32 || dt == SSD_BF16 || dt == SSD_F16; }

// A product of sizes that an int64 index must hold with room for strides.
bool fits(double a, double b, double c = 1.0) { return a * b * c <= 4e18; }

// Strides of a [nseq, L, ...] tensor with rows of `width`: non-negative, and far from overflowing an index.
bool strides_ok(int64_t seq, int64_t tok, int64_t nseq, int64_t L, int64_t width) {
    return seq >= 0 && tok >= 0 && (double)seq * (double)nseq + (double)tok * (double)L + (double)width <= 4e18;
}
// An output's rows must not overlap: each sequence's rows behind the one before, or each token's (token-major tensors).
bool rows_apart(int64_t seq, int64_t tok, int64_t nseq, int64_t L, int64_t width) {
    if (L <= 1) return nseq <= 1 || seq >= width;
    if (nseq <= 1) return tok >= width;
    return (tok >= width && seq >= (L - 1) * tok + width) || (seq >= width && tok >= (nseq - 1) * seq + width);
}

ssd_status_t check_scan(const ssd_scan_problem_t *p) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->batch < 0 || p->seqlen < 0 || p->channels < 1 || p->dstate < 1 || p->ngroups < 1 ||
        p->channels % p->ngroups)
        return SSD_ERR_INVALID_ARG;
    if (!io_ok(p->io_dtype) || (p->state_dtype != SSD_F32 && p->state_dtype != SSD_F16)) return SSD_ERR_INVALID_ARG;
    if ((p->packed != 0 && p->packed != 1) || (p->softplus != 0 && p->softplus != 1)) return SSD_ERR_INVALID_ARG;
    if (!fits((double)p->batch * (double)p->seqlen, (double)p->channels, (double)p->dstate) ||
        !fits((double)p->batch, (double)p->channels, (double)p->dstate))
        return SSD_ERR_INVALID_ARG;
    if (p->packed && (p->batch > INT32_MAX - 1 || p->seqlen > INT32_MAX)) return SSD_ERR_INVALID_ARG;
    if (p->packed && p->batch == 0 && p->seqlen > 0) return SSD_ERR_INVALID_ARG;  // tokens of no sequence
    if (p->dstate > 256) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// Segments of a scan and where their buffers lie in the workspace.
struct ScanPlan {
    int64_t nseg = 1, seg_len = 0, items = 0;  // items: segments whose leaving state is kept
    size_t state_off = 0, dt_off = 0, copy_off = 0, bytes = sizeof(WsHeader);
};
// single: rows are copied by single elements (fewer CTAs are resident, and a plan never takes more workspace than without)
ScanPlan plan_scan(const ssd_scan_problem_t &p, int sms, bool segments, bool single) {
    ScanPlan pl;
    const int64_t chains = p.packed ? 1 : p.batch;
    pl.seg_len = std::max<int64_t>(p.seqlen, 1);
    if (!segments || p.batch == 0 || (!p.packed && p.seqlen <= 1)) return pl;
    // Without segments the work of a chain runs once, with them its states' part twice. So segments are cut only where
    // the CTAs leave the SMs short of warps (under about 1.3 CTAs of 128 threads each: 4 x 4096 x 1536 x 16, 48 CTAs,
    // 0.84 ms in one chain and 0.24 segmented; 32 x 4096 x 1536 x 16, 384 CTAs, 1.28 and 1.57 ms when both were
    // measured in one build), and then so many that the resident CTAs are full about once, or twice where segments are
    // long: a part of a wave leaves SMs idle (8192 x 5120 x 16: 0.5, 1, 1.5 and 2 waves 0.70, 0.378, 0.416 and 0.379 ms;
    // 16384 x 5120 x 16: 1 and 2 waves 0.736 and 0.728), and more segments pay their entry more often (4000 x 1536 x 16,
    // packed: 1 and 2 waves 75 and 85 us). The segments of one wave are rounded down and then doubled, so the waves are
    // whole only where a segment has few CTAs: 16 x 4096 x 1536 x 16 has 192, 6 segments and 1.52 waves (908 us; 12
    // sequences 671, 24 1289).
    const ssd::ScanCta cta = ssd::scan_cta(p.dstate);
    const int64_t per_group = (p.channels / p.ngroups + cta.channels - 1) / cta.channels;
    const int64_t ctas = chains * p.ngroups * per_group, threads = ctas * cta.threads;
    if (threads * 10 >= 13 * 128 * (int64_t)sms) return pl;
    const int64_t waves = p.seqlen >= 2 * 400 * (cta.resident * (int64_t)sms / ctas) ? 2 : 1;  // the same for single
    const int64_t wave = (int64_t)(single ? cta.resident_single : cta.resident) * sms / ctas;
    const int64_t want = std::min<int64_t>(waves * wave, p.seqlen / 16);
    if (want < 2) return pl;
    int64_t len = (p.seqlen + want - 1) / want;
    len = (len + 7) / 8 * 8;  // whole tiles
    pl.nseg = (p.seqlen + len - 1) / len;
    pl.seg_len = len;
    if (pl.nseg < 2) return pl;
    pl.items = chains * (pl.nseg - 1);
    const size_t dn = (size_t)(p.channels * p.dstate);
    pl.state_off = sizeof(WsHeader);
    pl.dt_off = align_up(pl.state_off + (size_t)pl.items * dn * 4, 256);
    pl.copy_off = align_up(pl.dt_off + (size_t)(pl.items * p.channels) * 4, 256);
    pl.bytes = align_up(pl.copy_off + (size_t)p.batch * dn * elem_size(p.state_dtype), 256);
    return pl;
}

}  // namespace

extern "C" {

SSD_API ssd_status_t ssd_selective_scan_workspace_size(const ssd_scan_problem_t *prob, size_t *bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    const ssd_status_t st = check_scan(prob);
    if (st != SSD_OK) return st;
    *bytes = plan_scan(*prob, std::max(1, ssd::device_sms()), true, false).bytes;
    return SSD_OK;
}

SSD_API ssd_status_t ssd_selective_scan(const ssd_scan_problem_t *prob, const ssd_scan_tensors_t *t, void *workspace,
                                        size_t workspace_bytes, void *stream) {
    const ssd_status_t st = check_scan(prob);
    if (st != SSD_OK) return st;
    if (!t || !t->A) return SSD_ERR_INVALID_ARG;
    const ssd_scan_problem_t &pr = *prob;
    const size_t es = elem_size(pr.io_dtype), ses = elem_size(pr.state_dtype);
    const int64_t rows_seq = pr.packed ? 1 : pr.batch;  // leading dimension of the token tensors
    const bool tokens = pr.seqlen > 0 && rows_seq > 0;
    if (!aligned(t->A, 4) || !aligned(t->dt_bias, 4) || !aligned(t->D, 4) || !aligned(t->init_states, ses) ||
        !aligned(t->final_states, ses))
        return SSD_ERR_INVALID_ARG;
    if (pr.packed && pr.batch > 0 && (!t->cu_seqlens || !aligned(t->cu_seqlens, 4))) return SSD_ERR_INVALID_ARG;
    if (!pr.packed && t->cu_seqlens) return SSD_ERR_INVALID_ARG;
    if (tokens) {
        if (!t->x || !t->dt_raw || !t->B || !t->C || !t->y) return SSD_ERR_INVALID_ARG;
        if (!aligned(t->x, es) || !aligned(t->dt_raw, es) || !aligned(t->z, es) || !aligned(t->B, es) ||
            !aligned(t->C, es) || !aligned(t->y, es))
            return SSD_ERR_INVALID_ARG;
        const int64_t gn = pr.ngroups * pr.dstate;
        if (!strides_ok(t->x_seq, t->x_tok, rows_seq, pr.seqlen, pr.channels) ||
            !strides_ok(t->dt_seq, t->dt_tok, rows_seq, pr.seqlen, pr.channels) ||
            (t->z && !strides_ok(t->z_seq, t->z_tok, rows_seq, pr.seqlen, pr.channels)) ||
            !strides_ok(t->b_seq, t->b_tok, rows_seq, pr.seqlen, gn) ||
            !strides_ok(t->c_seq, t->c_tok, rows_seq, pr.seqlen, gn) ||
            !strides_ok(t->y_seq, t->y_tok, rows_seq, pr.seqlen, pr.channels) ||
            !rows_apart(t->y_seq, t->y_tok, rows_seq, pr.seqlen, pr.channels))
            return SSD_ERR_INVALID_ARG;
    }
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < sizeof(WsHeader)) return SSD_ERR_WORKSPACE;
    if (pr.batch == 0) return SSD_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!tokens) {  // nothing to scan: every final state is the initial one
        if (!t->final_states || t->final_states == t->init_states) return SSD_OK;
        const size_t n = (size_t)(pr.batch * pr.channels * pr.dstate) * ses;
        const cudaError_t e = t->init_states
                                  ? cudaMemcpyAsync(t->final_states, t->init_states, n, cudaMemcpyDeviceToDevice, s)
                                  : cudaMemsetAsync(t->final_states, 0, n, s);
        return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    }
    const int sms = ssd::device_sms();
    if (sms <= 0) return SSD_ERR_CUDA;
    ssd::ScanParams p;
    memset(&p, 0, sizeof(p));
    p.x = t->x;
    p.dt = t->dt_raw;
    p.z = t->z;
    p.B = t->B;
    p.C = t->C;
    p.y = t->y;
    p.A = t->A;
    p.dt_bias = t->dt_bias;
    p.D = t->D;
    p.init = t->init_states;
    p.fin = t->final_states;
    p.cu = pr.packed ? t->cu_seqlens : nullptr;
    p.hdr = static_cast<WsHeader *>(workspace);
    p.nseq = pr.batch;
    p.L = pr.seqlen;
    p.T = pr.packed ? pr.seqlen : pr.batch * pr.seqlen;
    p.D_ = pr.channels;
    p.N = pr.dstate;
    p.G = pr.ngroups;
    p.cpg = pr.channels / pr.ngroups;
    p.x_seq = t->x_seq;
    p.x_tok = t->x_tok;
    p.dt_seq = t->dt_seq;
    p.dt_tok = t->dt_tok;
    p.z_seq = t->z_seq;
    p.z_tok = t->z_tok;
    p.b_seq = t->b_seq;
    p.b_tok = t->b_tok;
    p.c_seq = t->c_seq;
    p.c_tok = t->c_tok;
    p.y_seq = t->y_seq;
    p.y_tok = t->y_tok;
    p.softplus = pr.softplus;
    p.state_f16 = pr.state_dtype == SSD_F16;
    p.rows = rows_seq;
    const int64_t cpg_bytes = p.cpg * (int64_t)es;
    auto rows_of = [&](const void *q, int64_t seq, int64_t tok, int64_t unit) {  // by whole units
        return !q || (aligned(q, (size_t)unit) && (rows_seq <= 1 || seq * (int64_t)es % unit == 0) &&
                      (pr.seqlen <= 1 || tok * (int64_t)es % unit == 0));
    };
    for (const int unit : {16, 8, 4})
        if (!p.unit && rows_of(p.x, p.x_seq, p.x_tok, unit) && rows_of(p.dt, p.dt_seq, p.dt_tok, unit) &&
            rows_of(p.z, p.z_seq, p.z_tok, unit) && rows_of(p.y, p.y_seq, p.y_tok, unit) &&
            (pr.ngroups == 1 || cpg_bytes % unit == 0))
            p.unit = unit;
    ScanPlan pl = plan_scan(pr, sms, true, p.unit == 0);
    if (workspace_bytes < pl.bytes) pl = plan_scan(pr, sms, false, false);  // too small for segments: one chain a sequence
    char *ws = static_cast<char *>(workspace);
    p.nseg = pl.nseg;
    p.seg_len = pl.seg_len;
    p.seg_items = pl.items;
    p.seg_state = reinterpret_cast<float *>(ws + pl.state_off);
    p.seg_dt = reinterpret_cast<float *>(ws + pl.dt_off);
    auto states4 = [&](const void *q, int64_t seq, int64_t tok) {  // four states of B and C, or of a whole R of a step
        const size_t a = pr.dstate > 128 ? 8 * es : 4 * es;
        return aligned(q, a) && (rows_seq <= 1 || seq * es % a == 0) && (pr.seqlen <= 1 || tok * es % a == 0) &&
               pr.dstate * es % a == 0;
    };
    p.vec_bc = states4(p.B, p.b_seq, p.b_tok) && states4(p.C, p.c_seq, p.c_tok);
    const size_t sa = (pr.dstate > 128 ? 8 : 4) * ses;
    p.vec_state = aligned(p.init, std::min<size_t>(sa, 16)) && aligned(p.fin, std::min<size_t>(sa, 16)) &&
                  aligned(p.A, 16) && pr.dstate * ses % sa == 0;
    // a segment's CTA may read a sequence's initial state after another one wrote its final state: where the two
    // share memory the initial states are copied first
    if (pl.nseg > 1 && p.init && p.fin) {
        const size_t n = (size_t)(pr.batch * pr.channels * pr.dstate) * ses;
        const char *a = static_cast<const char *>(p.init), *b = static_cast<const char *>(p.fin);
        if (a < b + n && b < a + n) {
            if (cudaMemcpyAsync(ws + pl.copy_off, p.init, n, cudaMemcpyDeviceToDevice, s) != cudaSuccess)
                return SSD_ERR_CUDA;
            p.init = ws + pl.copy_off;
        }
    }
    const cudaError_t e = pr.io_dtype == SSD_F32    ? ssd::launch_scan_f32(p, s)
                          : pr.io_dtype == SSD_BF16 ? ssd::launch_scan_bf16(p, s)
                                                    : ssd::launch_scan_f16(p, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

SSD_API ssd_status_t ssd_conv(const ssd_conv_problem_t *prob, const ssd_conv_tensors_t *t, void *workspace,
                              void *stream) {
    if (!prob || !t) return SSD_ERR_INVALID_ARG;
    const ssd_conv_problem_t &pr = *prob;
    if (pr.batch < 0 || pr.seqlen < 0 || pr.channels < 1 || pr.width < 1 || pr.width > 8 || !io_ok(pr.io_dtype))
        return SSD_ERR_INVALID_ARG;
    if ((pr.packed != 0 && pr.packed != 1) || (pr.activation != SSD_ACT_NONE && pr.activation != SSD_ACT_SILU))
        return SSD_ERR_INVALID_ARG;
    if (pr.packed && (pr.batch > INT32_MAX - 1 || pr.seqlen > INT32_MAX)) return SSD_ERR_INVALID_ARG;
    if (pr.packed && pr.batch == 0 && pr.seqlen > 0) return SSD_ERR_INVALID_ARG;  // tokens of no sequence
    if (!fits((double)pr.batch * (double)pr.seqlen, (double)pr.channels) ||
        !fits((double)pr.batch, (double)pr.channels, 8.0))
        return SSD_ERR_INVALID_ARG;
    const size_t es = elem_size(pr.io_dtype);
    const int64_t rows_seq = pr.packed ? 1 : pr.batch;
    const bool tokens = pr.seqlen > 0 && rows_seq > 0;
    if (!t->weight || !aligned(t->weight, 4) || !aligned(t->bias, 4) || !aligned(t->conv_state, es) ||
        !aligned(t->conv_state_out, es))
        return SSD_ERR_INVALID_ARG;
    if (pr.packed && pr.batch > 0 && (!t->cu_seqlens || !aligned(t->cu_seqlens, 4))) return SSD_ERR_INVALID_ARG;
    if (!pr.packed && t->cu_seqlens) return SSD_ERR_INVALID_ARG;
    if (tokens && (!t->x || !t->out || t->x == t->out || !aligned(t->x, es) || !aligned(t->out, es) ||
                   !strides_ok(t->x_seq, t->x_tok, rows_seq, pr.seqlen, pr.channels) ||
                   !strides_ok(t->out_seq, t->out_tok, rows_seq, pr.seqlen, pr.channels) ||
                   !rows_apart(t->out_seq, t->out_tok, rows_seq, pr.seqlen, pr.channels)))
        return SSD_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256)) return SSD_ERR_WORKSPACE;
    if (pr.batch == 0) return SSD_OK;
    const int sms = ssd::device_sms();
    if (sms <= 0) return SSD_ERR_CUDA;
    ssd::RowConvParams p;
    memset(&p, 0, sizeof(p));
    p.x = t->x;
    p.out = t->out;
    p.w = t->weight;
    p.bias = t->bias;
    p.state = t->conv_state;
    p.state_out = t->conv_state_out;
    p.cu = pr.packed ? t->cu_seqlens : nullptr;
    p.hdr = static_cast<WsHeader *>(workspace);
    p.nseq = pr.batch;
    p.L = pr.seqlen;
    p.T = pr.packed ? pr.seqlen : pr.batch * pr.seqlen;
    p.D = pr.channels;
    p.x_seq = t->x_seq;
    p.x_tok = t->x_tok;
    p.out_seq = t->out_seq;
    p.out_tok = t->out_tok;
    p.k = pr.width;
    p.silu = pr.activation == SSD_ACT_SILU;
    p.rows = rows_seq;
    auto rows_of = [&](const void *q, int64_t seq, int64_t tok, int64_t unit) {  // by whole units
        return aligned(q, (size_t)unit) && (rows_seq <= 1 || seq * (int64_t)es % unit == 0) &&
               (pr.seqlen <= 1 || tok * (int64_t)es % unit == 0);
    };
    for (const int unit : {16, 4})
        if (!p.unit && pr.channels * (int64_t)es % unit == 0 && rows_of(p.x, p.x_seq, p.x_tok, unit) &&
            rows_of(p.out, p.out_seq, p.out_tok, unit))
            p.unit = unit;
    p.vec_state = aligned(p.state_out, 16) && aligned(p.state, 16);
    p.vec_w = aligned(p.w, 16);
    return ssd::launch_row_conv(p, pr.io_dtype, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SSD_OK
                                                                                                      : SSD_ERR_CUDA;
}

SSD_API ssd_status_t ssd_group_norm(const ssd_norm_problem_t *prob, const ssd_norm_tensors_t *t, void *workspace,
                                    void *stream) {
    if (!prob || !t) return SSD_ERR_INVALID_ARG;
    const ssd_norm_problem_t &pr = *prob;
    if (pr.rows < 0 || pr.channels < 1 || pr.ngroups < 1 || pr.channels % pr.ngroups || !io_ok(pr.io_dtype) ||
        pr.reserved != 0)
        return SSD_ERR_INVALID_ARG;
    if ((pr.activation != SSD_ACT_NONE && pr.activation != SSD_ACT_SILU) || (pr.center != 0 && pr.center != 1) ||
        (pr.gate_first != 0 && pr.gate_first != 1) || !(pr.eps >= 0.f) || (pr.gate_first && !t->z))
        return SSD_ERR_INVALID_ARG;
    const size_t es = elem_size(pr.io_dtype);
    if (!aligned(t->weight, 4) || !aligned(t->bias, 4) || !aligned(t->scales, 4)) return SSD_ERR_INVALID_ARG;
    if (t->scales && pr.ngroups > 1 && (pr.channels / pr.ngroups) % 128) return SSD_ERR_UNSUPPORTED;
    if (pr.rows > 0 && (!t->x || !t->y || !aligned(t->x, es) || !aligned(t->z, es) ||
                        !aligned(t->y, t->scales ? 1 : es) || !strides_ok(0, t->x_row, 1, pr.rows, pr.channels) ||
                        (t->z && !strides_ok(0, t->z_row, 1, pr.rows, pr.channels)) ||
                        !strides_ok(0, t->y_row, 1, pr.rows, pr.channels) ||
                        !rows_apart(0, t->y_row, 1, pr.rows, pr.channels)))
        return SSD_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256)) return SSD_ERR_WORKSPACE;
    if (pr.rows == 0) return SSD_OK;
    const int sms = ssd::device_sms();
    if (sms <= 0) return SSD_ERR_CUDA;
    ssd::NormParams p;
    memset(&p, 0, sizeof(p));
    p.x = t->x;
    p.z = t->z;
    p.y = t->y;
    p.scales = t->scales;
    p.w = t->weight;
    p.bias = t->bias;
    p.hdr = static_cast<WsHeader *>(workspace);
    p.rows = pr.rows;
    p.D = pr.channels;
    p.G = pr.ngroups;
    p.x_row = t->x_row;
    p.z_row = t->z_row;
    p.y_row = t->y_row;
    p.center = pr.center;
    p.gate_first = pr.gate_first;
    p.silu = pr.activation == SSD_ACT_SILU;
    p.eps = pr.eps;
    const int64_t vec = 16 / (int64_t)es, gs = pr.channels / pr.ngroups;
    auto by = [&](int64_t n, size_t unit, size_t weights) {  // every group is made of pieces of n elements
        return gs % n == 0 && aligned(p.x, unit) && aligned(p.z, unit) && aligned(p.y, unit) && aligned(p.w, weights) &&
               aligned(p.bias, weights) && (pr.rows == 1 || (p.x_row % n == 0 && p.z_row % n == 0 && p.y_row % n == 0));
    };
    p.unit = by(vec, 16, 16) ? 16 : es == 2 && by(2, 4, 8) ? 4 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = pr.io_dtype == SSD_F32    ? ssd::launch_norm_f32(p, sms, s)
                          : pr.io_dtype == SSD_BF16 ? ssd::launch_norm_bf16(p, sms, s)
                                                    : ssd::launch_norm_f16(p, sms, s);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

SSD_API ssd_status_t ssd_fp8_quantize(int64_t rows, int64_t cols, int32_t block_rows, int32_t io_dtype, const void *x,
                                      int64_t x_row, void *q, float *scales, void *workspace, void *stream) {
    if (rows < 0 || cols < 0 || (block_rows != 1 && block_rows != 128) || !io_ok(io_dtype) ||
        !fits((double)rows, (double)cols))
        return SSD_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 256)) return SSD_ERR_WORKSPACE;
    if (rows == 0 || cols == 0) return SSD_OK;
    if (!x || !q || !scales || !aligned(x, elem_size(io_dtype)) || !aligned(scales, 4) ||
        !strides_ok(0, x_row, 1, rows, cols))
        return SSD_ERR_INVALID_ARG;
    const int sms = ssd::device_sms();
    if (sms <= 0) return SSD_ERR_CUDA;
    ssd::QuantParams p;
    memset(&p, 0, sizeof(p));
    p.x = x;
    p.q = static_cast<uint8_t *>(q);
    p.scales = scales;
    p.hdr = static_cast<WsHeader *>(workspace);
    p.rows = rows;
    p.cols = cols;
    p.x_row = x_row;
    p.block_rows = block_rows;
    p.vec = aligned(x, 16) && aligned(q, 8) && cols % 8 == 0 && (rows == 1 || x_row * elem_size(io_dtype) % 16 == 0);
    return ssd::launch_quantize(p, io_dtype, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SSD_OK
                                                                                                   : SSD_ERR_CUDA;
}

SSD_API ssd_status_t ssd_fp8_matmul(const ssd_matmul_problem_t *prob, const void *a, const float *a_scales,
                                    const void *b, const float *b_scales, const float *bias, void *out,
                                    int64_t out_row, void *workspace, size_t workspace_bytes, void *stream) {
    if (!prob) return SSD_ERR_INVALID_ARG;
    const ssd_matmul_problem_t &pr = *prob;
    if (pr.m < 0 || pr.n < 0 || pr.k < 0 || !io_ok(pr.out_dtype) || pr.reserved != 0 ||
        !fits((double)pr.m, (double)pr.n) || !fits((double)pr.m, (double)pr.k) || !fits((double)pr.n, (double)pr.k))
        return SSD_ERR_INVALID_ARG;
    if (pr.m > INT32_MAX - 512 || pr.n > INT32_MAX - 512 || pr.k > INT32_MAX - 512 || pr.k % 16)
        return SSD_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < sizeof(WsHeader)) return SSD_ERR_WORKSPACE;
    if (pr.m == 0 || pr.n == 0) return SSD_OK;
    if (!out || !aligned(out, elem_size(pr.out_dtype)) || !aligned(bias, 4) ||
        !strides_ok(0, out_row, 1, pr.m, pr.n) || !rows_apart(0, out_row, 1, pr.m, pr.n))
        return SSD_ERR_INVALID_ARG;
    if (pr.k > 0 && (!a || !b || !a_scales || !b_scales || !aligned(a, 16) || !aligned(b, 16) ||
                     !aligned(a_scales, 4) || !aligned(b_scales, 4)))
        return SSD_ERR_INVALID_ARG;
    const int sms = ssd::device_sms();
    if (sms <= 0) return SSD_ERR_CUDA;
    ssd::MatmulParams p;
    memset(&p, 0, sizeof(p));
    p.a = static_cast<const uint8_t *>(a);
    p.b = static_cast<const uint8_t *>(b);
    p.sa = a_scales;
    p.sb = b_scales;
    p.bias = bias;
    p.out = out;
    p.hdr = static_cast<WsHeader *>(workspace);
    p.m = pr.m;
    p.n = pr.n;
    p.k = pr.k;
    p.out_row = out_row;
    const cudaError_t e = ssd::launch_matmul(p, pr.out_dtype, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : e == cudaErrorNotSupported ? SSD_ERR_UNSUPPORTED : SSD_ERR_CUDA;
}

SSD_API ssd_status_t ssd_debug_product(int32_t token_tile, int32_t splits) {
    return ssd::force_product(token_tile, splits) ? SSD_OK : SSD_ERR_INVALID_ARG;
}

}  // extern "C"
