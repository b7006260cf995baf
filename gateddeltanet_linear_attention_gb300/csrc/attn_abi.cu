// attn_abi.cu -- the extern "C" entry points of the attention layers (include/gdn.h): argument validation before any
// launch, workspace carving and dispatch.
#include <climits>
#include <cmath>

#include "attn_common.cuh"

namespace {

constexpr int kMaxRows = 65535;
constexpr int kMaxPages = 1 << 24;
constexpr int kMaxLength = 1 << 30;

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
gdn_status launch_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// Head vectors of `heads` heads of `rows` tokens, whose 16-byte pieces can be loaded whole.
bool valid_heads(const void *p, long long ld, long long hs, long long rows, long long heads, long long D) {
    return p && aligned16(p) && ld % 8 == 0 && hs % 8 == 0 && (ld >= D || rows <= 1) && (hs >= D || heads <= 1);
}
// The same where they are written: no two of them overlap.
bool valid_out_heads(const void *p, long long ld, long long hs, long long rows, long long heads, long long D) {
    return valid_heads(p, ld, hs, rows, heads, D) &&
           (rows <= 1 || heads <= 1 || ld >= (heads - 1) * hs + D || hs >= (rows - 1) * ld + D);
}
// `to` in the place of a contiguous `from`: each vector in its own, for others are still to be read.
bool in_place(const void *to, long long ld, long long hs, const void *from, long long rows, long long heads, long long D) {
    return to != from || ((rows <= 1 || ld == heads * D) && (heads <= 1 || hs == D));
}

gdn_status check_cfg(const gdn_attn_config *c, gdn::AttnDims *d) {
    if (!c) return GDN_ERR_INVALID_ARG;
    if (c->q_heads <= 0 || c->kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0 || c->n_pages < 0 || c->n_rows < 0 ||
        c->max_pages < 0 || (c->act != GDN_BF16 && c->act != GDN_FP32) || c->q_heads % c->kv_heads != 0)
        return GDN_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return GDN_ERR_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return GDN_ERR_UNSUPPORTED;
    if (c->q_heads / c->kv_heads > gdn::kAttnMaxGroup || c->q_heads > 4096 || c->n_rows > kMaxRows || c->n_pages > kMaxPages)
        return GDN_ERR_UNSUPPORTED;
    // lengths with a tile behind them, and the rows of a pool (one token of one key head each), are 32-bit numbers
    if ((long long)c->max_pages * c->page_size > kMaxLength || (long long)c->n_pages * c->kv_heads * c->page_size > INT_MAX)
        return GDN_ERR_UNSUPPORTED;
    d->hq = c->q_heads; d->hkv = c->kv_heads; d->grp = c->q_heads / c->kv_heads; d->D = c->head_dim;
    d->page = c->page_size;
    d->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
    d->n_pages = c->n_pages; d->n_rows = c->n_rows; d->max_pages = c->max_pages;
    return GDN_OK;
}

// What both directions of the norm and rotation share.
gdn_status check_prep(const gdn_attn_config *cfg, const gdn_attn_prep_io *io, gdn::AttnPrepArgs *a) {
    gdn_status st = check_cfg(cfg, &a->d);
    if (st != GDN_OK) return st;
    if (!io || io->T < 0 || io->n_seqs < 0) return GDN_ERR_INVALID_ARG;
    const gdn::AttnDims &d = a->d;
    const long long T = io->T, D = d.D;
    if (T > INT_MAX) return GDN_ERR_UNSUPPORTED;
    if (!std::isfinite(io->weight_offset) || !std::isfinite(io->eps) || io->eps < 0.f || io->rotary_dim < 0 ||
        io->rotary_dim > D || io->rotary_dim % 2 != 0 || (io->interleaved != 0 && io->interleaved != 1) ||
        (io->rotary_dim > 0 && !io->inv_freq) || !aligned4(io->inv_freq) || !aligned4(io->positions) ||
        !aligned4(io->cu_seqlens) || !aligned16(io->w_q) || !aligned16(io->w_k))
        return GDN_ERR_INVALID_ARG;
    // the batch: tokens belong to sequences, as many to each where no bounds say otherwise
    if (T > 0 && (io->n_seqs == 0 || (!io->cu_seqlens && T % io->n_seqs != 0))) return GDN_ERR_INVALID_ARG;
    if (io->cu_seqlens && io->n_seqs > (1 << 24)) return GDN_ERR_UNSUPPORTED;
    if (T > 0) {
        if (!valid_heads(io->q, io->ld_q, io->hs_q, T, d.hq, D) || (io->k && !valid_heads(io->k, io->ld_k, io->hs_k, T, d.hkv, D)))
            return GDN_ERR_INVALID_ARG;
    }
    if (io->w_k && !io->k && T > 0) return GDN_ERR_INVALID_ARG;
    a->q = io->q; a->ld_q = io->ld_q; a->hs_q = io->hs_q;
    a->k = io->k; a->ld_k = io->ld_k; a->hs_k = io->hs_k;
    a->T = T; a->w_q = io->w_q; a->w_k = io->w_k; a->inv_freq = io->inv_freq;
    a->offset = io->weight_offset; a->eps = io->eps; a->half = io->rotary_dim / 2; a->interleaved = io->interleaved != 0;
    a->positions = io->positions; a->cu = io->cu_seqlens; a->n_seqs = io->n_seqs;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_attn_prep(const gdn_attn_config *cfg, const gdn_attn_prep_io *io, void *stream) {
    gdn::AttnPrepArgs a{};
    gdn_status st = check_prep(cfg, io, &a);
    if (st != GDN_OK) return st;
    const gdn::AttnDims &d = a.d;
    const bool pools = io->k_pages != nullptr;
    if ((io->v_pages != nullptr) != pools || (io->T > 0 && (io->v != nullptr) != pools) || !aligned16(io->k_pages) ||
        !aligned16(io->v_pages) || !aligned4(io->rows) || !aligned4(io->lens) || !aligned4(io->page_table) ||
        !aligned16(io->q_out) || !aligned16(io->k_out))
        return GDN_ERR_INVALID_ARG;
    if (pools && (!io->lens || !io->page_table || d.n_pages == 0 || d.max_pages == 0)) return GDN_ERR_INVALID_ARG;
    if ((io->lens || io->rows) && d.n_rows == 0) return GDN_ERR_INVALID_ARG;
    if (io->T == 0) return GDN_OK;
    if (!io->q_out || (pools && (!io->k || !valid_heads(io->v, io->ld_v, io->hs_v, io->T, d.hkv, d.D))) ||
        (io->k_out && !io->k) || (io->k && !io->k_out && !pools))
        return GDN_ERR_INVALID_ARG;
    if ((st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.v = io->v; a.ld_v = io->ld_v; a.hs_v = io->hs_v;
    a.rows = io->rows; a.lens = io->lens; a.table = io->page_table;
    a.k_pages = io->k_pages; a.v_pages = io->v_pages; a.q_out = io->q_out; a.k_out = io->k_out;
    return launch_status(gdn::launch_attn_prep(a, cfg->act == GDN_BF16, (cudaStream_t)stream));
}

size_t gdn_attn_prep_workspace_size(const gdn_attn_config *cfg, int64_t max_tokens) {
    gdn::AttnDims d;
    if (check_cfg(cfg, &d) != GDN_OK || max_tokens < 0 || max_tokens > INT_MAX) return 0;
    return gdn::attn_prep_ws_floats(d, max_tokens) * 4 + 256;
}

gdn_status gdn_attn_prep_backward(const gdn_attn_config *cfg, const gdn_attn_prep_io *io, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    gdn::AttnPrepArgs a{};
    gdn_status st = check_prep(cfg, io, &a);
    if (st != GDN_OK) return st;
    const gdn::AttnDims &d = a.d;
    if (!aligned16(io->dq_out) || !aligned16(io->dk_out) || !aligned4(io->dw_q) || !aligned4(io->dw_k) ||
        (io->dw_q && !io->w_q) || (io->dw_k && !io->w_k))
        return GDN_ERR_INVALID_ARG;
    if (io->T > 0 && (!io->dq_out || (io->dq && !valid_out_heads(io->dq, io->ld_dq, io->hs_dq, io->T, d.hq, d.D)) ||
                      (io->k != nullptr) != (io->dk_out != nullptr) || (io->dk && !io->k) ||
                      (io->dk && !valid_out_heads(io->dk, io->ld_dk, io->hs_dk, io->T, d.hkv, d.D)) ||
                      (io->dq && !in_place(io->dq, io->ld_dq, io->hs_dq, io->dq_out, io->T, d.hq, d.D)) ||
                      (io->dk && !in_place(io->dk, io->ld_dk, io->hs_dk, io->dk_out, io->T, d.hkv, d.D))))
        return GDN_ERR_INVALID_ARG;
    const bool weights = io->dw_q || io->dw_k;
    if (weights) {
        if (!workspace || !aligned16(workspace) || workspace_bytes < gdn::attn_prep_ws_floats(d, io->T) * 4)
            return GDN_ERR_WORKSPACE;
        a.ws = (float *)workspace;
    }
    if (io->T == 0 && !weights) return GDN_OK;
    if ((st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.dq_out = io->dq_out; a.dk_out = io->dk_out;
    a.dq = io->dq; a.ld_dq = io->ld_dq; a.hs_dq = io->hs_dq;
    a.dk = io->dk; a.ld_dk = io->ld_dk; a.hs_dk = io->hs_dk;
    a.dw_q = io->dw_q; a.dw_k = io->dw_k;
    return launch_status(gdn::launch_attn_prep_backward(a, cfg->act == GDN_BF16, (cudaStream_t)stream));
}

size_t gdn_attn_workspace_size(const gdn_attn_config *cfg, int32_t max_seqs, int32_t tokens) {
    gdn::AttnDims d;
    if (check_cfg(cfg, &d) != GDN_OK || max_seqs < 0 || max_seqs > kMaxRows || tokens < 1 || tokens > gdn::kAttnMaxTokens) return 0;
    return gdn::attn_decode_ws_bytes(d, d.grp * tokens) + 256;
}

gdn_status gdn_attn_decode(const gdn_attn_config *cfg, const gdn_attn_decode_io *io, void *workspace, size_t workspace_bytes,
                           void *stream) {
    gdn::AttnDecodeArgs a{};
    gdn_status st = check_cfg(cfg, &a.d);
    if (st != GDN_OK) return st;
    if (!io || io->n_seqs < 0 || io->tokens < 1 || io->window < 0 || !std::isfinite(io->scale * gdn::kLog2e) || !(io->scale > 0.f))
        return GDN_ERR_INVALID_ARG;
    if (io->tokens > gdn::kAttnMaxTokens || io->n_seqs > kMaxRows) return GDN_ERR_UNSUPPORTED;
    if (io->n_seqs == 0) return GDN_OK;
    const gdn::AttnDims &d = a.d;
    if (d.n_pages == 0 || d.n_rows == 0 || d.max_pages == 0 || !io->k_pages || !io->v_pages || !aligned16(io->k_pages) ||
        !aligned16(io->v_pages) || !io->page_table || !aligned4(io->page_table) || !io->lens || !aligned4(io->lens) ||
        !aligned4(io->rows) || !io->out || !aligned16(io->out) || !aligned4(io->lse) ||
        !valid_heads(io->q, io->ld_q, io->hs_q, (long long)io->n_seqs * io->tokens, d.hq, d.D))
        return GDN_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < gdn::attn_decode_ws_bytes(d, d.grp * io->tokens))
        return GDN_ERR_WORKSPACE;
    if ((st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.q = io->q; a.ld_q = io->ld_q; a.hs_q = io->hs_q; a.k_pages = io->k_pages; a.v_pages = io->v_pages;
    a.table = io->page_table; a.lens = io->lens; a.rows = io->rows;
    a.n_seqs = io->n_seqs; a.tokens = io->tokens;
    // a window that no length reaches is none, and no difference of a length and a window leaves 32 bits
    a.window = io->window < d.max_pages * d.page ? io->window : 0;
    a.scale_log2 = io->scale * gdn::kLog2e;
    a.out = io->out; a.lse = io->lse; a.wait_ns = gdn::wait_limit_ns();
    a.lose = gdn::lost_copies();
    gdn::attn_decode_carve(a, workspace);
    return launch_status(gdn::launch_attn_decode(a, cfg->act == GDN_BF16, (cudaStream_t)stream));
}

// ------------------------------------------------------------------- pages
size_t gdn_page_workspace_size(const gdn_attn_config *cfg, int32_t max_lanes) {
    gdn::AttnDims d;
    if (check_cfg(cfg, &d) != GDN_OK || max_lanes < 0) return 0;
    return gdn::page_ws_ints(d, max_lanes) * 4 + 256;
}

namespace {
// A configuration with a cache, and lanes to work on.
gdn_status check_pages(const gdn_attn_config *cfg, int32_t n, gdn::PageArgs *a) {
    const gdn_status st = check_cfg(cfg, &a->d);
    if (st != GDN_OK) return st;
    if (n < 0 || a->d.n_pages == 0 || a->d.n_rows == 0 || a->d.max_pages == 0) return GDN_ERR_INVALID_ARG;
    a->n = n;
    return GDN_OK;
}
bool good(const void *p) { return p && aligned4(p); }
gdn_status check_ws(const gdn::PageArgs &a, const void *ws, size_t bytes) {
    return ws && aligned16(ws) && bytes >= gdn::page_ws_ints(a.d, a.n) * 4 ? GDN_OK : GDN_ERR_WORKSPACE;
}
}  // namespace

gdn_status gdn_page_resize(const gdn_attn_config *cfg, int32_t *page_table, int32_t *lens, int32_t *refs, const int32_t *rows,
                           const int32_t *new_lens, int32_t n, int32_t *granted, int32_t *src_idx, int32_t *dst_idx,
                           void *workspace, size_t workspace_bytes, void *stream) {
    gdn::PageArgs a{};
    gdn_status st = check_pages(cfg, n, &a);
    if (st != GDN_OK || n == 0) return st;
    if (n > kMaxRows) return GDN_ERR_UNSUPPORTED;
    if (!good(page_table) || !good(lens) || !good(refs) || !good(rows) || !good(new_lens) || !good(granted) || !good(src_idx) ||
        !good(dst_idx))
        return GDN_ERR_INVALID_ARG;
    if ((st = check_ws(a, workspace, workspace_bytes)) != GDN_OK || (st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.table = page_table; a.lens = lens; a.refs = refs; a.rows = rows; a.new_lens = new_lens;
    a.granted = granted; a.src = src_idx; a.dst = dst_idx; a.ws = (int32_t *)workspace;
    return launch_status(gdn::launch_page_resize(a, (cudaStream_t)stream));
}

gdn_status gdn_page_fork(const gdn_attn_config *cfg, int32_t *page_table, int32_t *lens, int32_t *refs, const int32_t *src_rows,
                         const int32_t *dst_rows, int32_t n, void *stream) {
    gdn::PageArgs a{};
    gdn_status st = check_pages(cfg, n, &a);
    if (st != GDN_OK || n == 0) return st;
    if (n > kMaxRows) return GDN_ERR_UNSUPPORTED;
    if (!good(page_table) || !good(lens) || !good(refs) || !good(src_rows) || !good(dst_rows)) return GDN_ERR_INVALID_ARG;
    if ((st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.table = page_table; a.lens = lens; a.refs = refs; a.rows = dst_rows; a.new_lens = src_rows;
    return launch_status(gdn::launch_page_fork(a, (cudaStream_t)stream));
}

gdn_status gdn_page_compact(const gdn_attn_config *cfg, const int32_t *page_table, const int32_t *lens, const int32_t *refs,
                            int32_t *table_out, int32_t *refs_out, int32_t *src_idx, int32_t *dst_idx, int32_t n, void *workspace,
                            size_t workspace_bytes, void *stream) {
    gdn::PageArgs a{};
    gdn_status st = check_pages(cfg, n, &a);
    if (st != GDN_OK) return st;
    if (!good(page_table) || !good(lens) || !good(refs) || !good(table_out) || !good(refs_out) ||
        (n > 0 && (!good(src_idx) || !good(dst_idx))))
        return GDN_ERR_INVALID_ARG;
    if ((st = check_ws(a, workspace, workspace_bytes)) != GDN_OK || (st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.table = const_cast<int32_t *>(page_table); a.lens = const_cast<int32_t *>(lens); a.refs = const_cast<int32_t *>(refs);
    a.table_out = table_out; a.refs_out = refs_out; a.src = src_idx; a.dst = dst_idx; a.ws = (int32_t *)workspace;
    return launch_status(gdn::launch_page_compact(a, (cudaStream_t)stream));
}

gdn_status gdn_page_copy(const gdn_attn_config *cfg, const void *src_k, const void *src_v, int32_t n_src, void *dst_k, void *dst_v,
                         int32_t n_dst, const int32_t *src_idx, const int32_t *dst_idx, int32_t n, void *stream) {
    gdn::AttnDims d;
    gdn_status st = check_cfg(cfg, &d);
    if (st != GDN_OK) return st;
    if (n < 0 || n_src < 0 || n_dst < 0) return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    if ((!dst_k && !dst_v) || !aligned16(src_k) || !aligned16(src_v) || !aligned16(dst_k) || !aligned16(dst_v) || !good(src_idx) ||
        !good(dst_idx))
        return GDN_ERR_INVALID_ARG;
    unsigned *err;
    if ((st = gdn::device_error_word(&err)) != GDN_OK) return st;
    const long long bytes = (long long)d.hkv * d.page * d.D * (cfg->act == GDN_BF16 ? 2 : 4);
    return launch_status(gdn::launch_page_copy(src_k, src_v, n_src, dst_k, dst_v, n_dst, src_idx, dst_idx, n, bytes, err,
                                               (cudaStream_t)stream));
}

}  // extern "C"
