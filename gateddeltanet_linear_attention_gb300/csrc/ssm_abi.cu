// ssm_abi.cu -- the extern "C" entry points of the selective state space mixer
// and of the block norms (include/gdn.h): argument validation before any
// launch, workspace carving and dispatch.
#include <climits>
#include <cmath>

#include "ssm_common.cuh"

namespace {

constexpr int kMaxSeqs = 65535;       // one grid dimension per sequence
constexpr int kMaxNormDim = 16384;

bool valid_dtype(gdn_dtype t) { return t == GDN_BF16 || t == GDN_FP32; }
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
gdn_status launch_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// A wide view: 16-byte aligned rows of at least `width` elements.
bool valid_view(const void *p, long long ld, long long width) {
    return p && aligned16(p) && ld >= width && ld % 8 == 0;
}

gdn_status check_cfg(const gdn_ssm_config *c, gdn::SsmDims *d) {
    if (!c) return GDN_ERR_INVALID_ARG;
    if (c->groups <= 0 || c->heads <= 0 || c->d_state <= 0 || c->head_dim <= 0 || c->n_slots < 0 ||
        !valid_dtype(c->act))
        return GDN_ERR_INVALID_ARG;
    // written so that a NaN fails
    if (!(c->dt_min >= 0.f && c->dt_max >= c->dt_min) || std::isinf(c->dt_min)) return GDN_ERR_INVALID_ARG;
    if (c->heads % c->groups != 0) return GDN_ERR_INVALID_ARG;
    if (c->d_state != 16 && c->d_state != 32 && c->d_state != 64 && c->d_state != 128)
        return GDN_ERR_UNSUPPORTED;
    if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return GDN_ERR_UNSUPPORTED;
    const long long ch = (long long)c->heads * c->head_dim + 2LL * c->groups * c->d_state;
    if (c->heads > 4096 || ch > (1LL << 22)) return GDN_ERR_UNSUPPORTED;
    d->groups = c->groups; d->heads = c->heads; d->N = c->d_state; d->P = c->head_dim;
    d->per = c->heads / c->groups; d->ch = (int)ch; d->n_slots = c->n_slots;
    d->dt_min = c->dt_min; d->dt_max = c->dt_max;
    return GDN_OK;
}

// Packed-batch arguments shared by the prompt calls.
gdn_status check_batch(int64_t T, int32_t n_seqs, const int32_t *cu) {
    if (T < 0 || n_seqs < 0) return GDN_ERR_INVALID_ARG;
    if (n_seqs > kMaxSeqs || T > INT_MAX) return GDN_ERR_UNSUPPORTED;
    if (n_seqs == 0) return T == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
    if (!cu || !aligned4(cu)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

size_t elem(bool bf16) { return bf16 ? 2 : 4; }

}  // namespace

extern "C" {

size_t gdn_ssm_workspace_size(const gdn_ssm_config *cfg, int64_t max_tokens, int32_t max_seqs) {
    gdn::SsmDims d;
    if (check_cfg(cfg, &d) != GDN_OK || max_tokens < 0 || max_seqs < 0) return 0;
    if (max_tokens > INT_MAX || max_seqs > kMaxSeqs) return 0;
    const size_t scan = gdn::ssm_scan_ws_bytes(d, cfg->act == GDN_BF16, max_tokens, max_seqs),
                 step = gdn::ssm_step_ws_bytes(d, max_seqs);
    return (scan > step ? scan : step) + 256;
}

gdn_status gdn_ssm_conv_prefill(const gdn_ssm_config *cfg, const void *x, int64_t ld_x,
                                const int32_t *cu_seqlens, int32_t n_seqs, int64_t T, const void *w,
                                const void *bias, void *conv_state, const int32_t *state_idx, void *out,
                                void *stream) {
    gdn::SsmConvArgs a{};
    gdn_status st = check_cfg(cfg, &a.d);
    if (st != GDN_OK || (st = check_batch(T, n_seqs, cu_seqlens)) != GDN_OK) return st;
    if (T == 0 || n_seqs == 0) return GDN_OK;
    if (!valid_view(x, ld_x, a.d.ch) || !w || !aligned16(w) || !aligned16(bias) || !out || !aligned16(out) ||
        !aligned16(conv_state) || !aligned4(state_idx) || (conv_state && cfg->n_slots == 0))
        return GDN_ERR_INVALID_ARG;
    if (!conv_state) a.d.n_slots = INT_MAX;      // no pool to bound the slots by
    if ((st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.x = x; a.ld_x = ld_x; a.cu = cu_seqlens; a.n_seqs = n_seqs; a.T = T; a.w = w; a.bias = bias;
    a.conv_state = conv_state; a.state_idx = state_idx; a.out = out;
    return launch_status(gdn::launch_ssm_conv(a, cfg->act == GDN_BF16, (cudaStream_t)stream));
}

gdn_status gdn_ssm_prefill(const gdn_ssm_config *cfg, const gdn_ssm_io *io, void *workspace,
                           size_t workspace_bytes, void *stream) {
    gdn::SsmScanArgs a{};
    gdn_status st = check_cfg(cfg, &a.d);
    if (st != GDN_OK) return st;
    if (!io) return GDN_ERR_INVALID_ARG;
    if ((st = check_batch(io->T, io->n_seqs, io->cu_seqlens)) != GDN_OK) return st;
    if (io->n_seqs == 0) return GDN_OK;
    const gdn::SsmDims &d = a.d;
    const long long hp = (long long)d.heads * d.P, gn = (long long)d.groups * d.N;
    if (io->T > 0 && (!valid_view(io->x, io->ld_x, hp) || !valid_view(io->b, io->ld_bc, gn) ||
                      !valid_view(io->c, io->ld_bc, gn) || !io->dt || io->ld_dt < d.heads ||
                      ((uintptr_t)io->dt & (elem(cfg->act == GDN_BF16) - 1)) != 0 ||
                      (io->z && !valid_view(io->z, io->ld_z, hp)) || !io->y || !aligned16(io->y)))
        return GDN_ERR_INVALID_ARG;
    if (!io->A_log || !aligned4(io->A_log) || !aligned4(io->dt_bias) || !aligned4(io->D) ||
        !aligned16(io->state_in) || !aligned16(io->state_out) || !aligned4(io->state_idx) ||
        ((io->state_in || io->state_out) && cfg->n_slots == 0))
        return GDN_ERR_INVALID_ARG;
    const bool bf16 = cfg->act == GDN_BF16;
    a.T = io->T; a.n_seqs = io->n_seqs;
    const size_t need = gdn::ssm_scan_carve(a, bf16, workspace);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if ((st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.x = io->x; a.ld_x = io->ld_x; a.b = io->b; a.c = io->c; a.ld_bc = io->ld_bc;
    a.dt = io->dt; a.ld_dt = io->ld_dt; a.z = io->z; a.ld_z = io->ld_z;
    a.A_log = io->A_log; a.dt_bias = io->dt_bias; a.D = io->D;
    a.cu = io->cu_seqlens; a.state_idx = io->state_idx;
    a.state_in = io->state_in; a.state_out = io->state_out; a.y = io->y;
    a.wait_ns = gdn::wait_limit_ns();
    a.lose = gdn::lost_copies();
    if (!io->state_in && !io->state_out) a.d.n_slots = INT_MAX;
    return launch_status(gdn::launch_ssm_scan(a, bf16, (cudaStream_t)stream));
}

gdn_status gdn_ssm_decode(const gdn_ssm_config *cfg, const gdn_ssm_io *io, void *workspace,
                          size_t workspace_bytes, void *stream) {
    gdn::SsmStepArgs a{};
    gdn_status st = check_cfg(cfg, &a.d);
    if (st != GDN_OK) return st;
    if (!io || io->n_seqs < 0 || io->T != io->n_seqs) return GDN_ERR_INVALID_ARG;
    if (io->n_seqs > kMaxSeqs) return GDN_ERR_UNSUPPORTED;
    if (io->n_seqs == 0) return GDN_OK;
    const gdn::SsmDims &d = a.d;
    const long long hp = (long long)d.heads * d.P;
    const bool bf16 = cfg->act == GDN_BF16;
    if (!valid_view(io->x, io->ld_x, d.ch) || io->b || io->c || !io->dt || io->ld_dt < d.heads ||
        ((uintptr_t)io->dt & (elem(bf16) - 1)) != 0 || (io->z && !valid_view(io->z, io->ld_z, hp)) ||
        !io->conv_w || !aligned16(io->conv_w) || !aligned16(io->conv_bias) || !io->A_log ||
        !aligned4(io->A_log) || !aligned4(io->dt_bias) || !aligned4(io->D) || !io->state_in ||
        io->state_out != io->state_in || !aligned16(io->state_in) || !io->conv_state ||
        !aligned16(io->conv_state) || !aligned4(io->state_idx) || !io->y || !aligned16(io->y) ||
        cfg->n_slots == 0)
        return GDN_ERR_INVALID_ARG;
    const size_t need = gdn::ssm_step_ws_bytes(d, io->n_seqs);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if ((st = gdn::device_error_word(&a.err)) != GDN_OK) return st;
    a.x = io->x; a.ld_x = io->ld_x; a.dt = io->dt; a.ld_dt = io->ld_dt; a.z = io->z; a.ld_z = io->ld_z;
    a.w = io->conv_w; a.bias = io->conv_bias; a.conv_state = io->conv_state;
    a.A_log = io->A_log; a.dt_bias = io->dt_bias; a.D = io->D; a.n = io->n_seqs;
    a.state_idx = io->state_idx; a.state = io->state_out; a.y = io->y; a.ws = (float *)workspace;
    return launch_status(gdn::launch_ssm_step(a, bf16, (cudaStream_t)stream));
}

// ------------------------------------------------------------- block norms
namespace {

gdn_status check_norm(const gdn_block_norm_io *io, bool backward, gdn::NormArgs *a) {
    if (!io || io->rows < 0 || io->dim <= 0 || !valid_dtype(io->act) || !valid_dtype(io->res)) return GDN_ERR_INVALID_ARG;
    if (io->dim > kMaxNormDim || io->rows > (1LL << 40) || (io->act == GDN_FP32 && io->res == GDN_BF16))
        return GDN_ERR_UNSUPPORTED;
    if (!std::isfinite(io->eps) || io->eps < 0.f || !std::isfinite(io->weight_offset) || !std::isfinite(io->res_scale))
        return GDN_ERR_INVALID_ARG;
    const size_t ea = elem(io->act == GDN_BF16), er = elem(io->res == GDN_BF16);
    const int64_t dim = io->dim;
    bool vec = dim % 8 == 0, ok = true;
    // a row-strided view of `cols` columns; `wide` ones decide on vector access
    auto view = [&](const void *p, int64_t ld, size_t e, int64_t cols, bool wide) {
        if (!p) return;
        if (((uintptr_t)p & (e - 1)) != 0 || ld < cols) ok = false;
        if (wide && (!aligned16(p) || (ld * (int64_t)e) % 16 != 0)) vec = false;
    };
    auto vector = [&](const float *p) {
        if (!aligned4(p)) ok = false;
        if (!aligned16(p)) vec = false;
    };
    const bool channel = io->gate && io->gate_cols != 1;
    if (io->gate && io->gate_cols != 1 && io->gate_cols != io->dim) return GDN_ERR_INVALID_ARG;
    view(io->block, io->ld_block, ea, dim, true);
    view(io->gate, io->ld_gate, ea, io->gate_cols, channel);
    view(io->residual, io->ld_residual, er, dim, true);
    vector(io->w_post);
    vector(io->w_pre);
    if (!aligned4(io->rstd_post) || !aligned4(io->rstd_pre)) ok = false;
    if (!backward) {
        view(io->res_out, io->ld_res_out, er, dim, true);
        view(io->h, io->ld_h, ea, dim, true);
    } else {
        view(io->dh, io->ld_dh, ea, dim, true);
        view(io->d_res_out, io->ld_d_res_out, er, dim, true);
        view(io->d_residual, io->ld_d_residual, er, dim, true);
        view(io->d_block, io->ld_d_block, ea, dim, true);
        view(io->d_gate, io->ld_d_gate, ea, io->gate_cols, channel);
        vector(io->dw_post);
        vector(io->dw_pre);
    }
    // which operands go together; without rows, views may be null
    if (io->rows > 0) {
        if (!io->block && (io->gate || io->w_post)) ok = false;
        if (!backward) {
            if (!io->residual || (!io->h && !io->res_out) || (io->w_pre == nullptr) != (io->h == nullptr) ||
                (io->res_out && !io->block) || (io->rstd_post && !io->w_post) || (io->rstd_pre && !io->w_pre))
                ok = false;
        } else {
            if ((io->w_pre == nullptr) != (io->dh == nullptr) || (!io->dh && !io->d_res_out) ||
                (io->dh && (!io->residual || !io->rstd_pre)) || (io->w_post && !io->rstd_post) ||
                (io->d_block && !io->block) || (io->d_gate && !io->gate) || (io->dw_post && !io->w_post) ||
                (io->dw_pre && !io->w_pre))
                ok = false;
        }
    }
    if (!ok) return GDN_ERR_INVALID_ARG;
    a->rows = io->rows; a->dim = io->dim; a->act_bf16 = io->act == GDN_BF16; a->res_bf16 = io->res == GDN_BF16;
    a->eps = io->eps; a->offset = io->weight_offset; a->scale = io->res_scale;
    a->block = io->block; a->ld_block = io->ld_block; a->gate = io->gate; a->ld_gate = io->ld_gate;
    a->gate_cols = channel ? io->dim : 1;
    a->residual = io->residual; a->ld_res = io->ld_residual;
    a->w_post = io->w_post; a->w_pre = io->w_pre;
    a->vec = vec;
    return GDN_OK;
}

}  // namespace

gdn_status gdn_block_norm(const gdn_block_norm_io *io, void *stream) {
    gdn::NormArgs a{};
    const gdn_status st = check_norm(io, false, &a);
    if (st != GDN_OK || io->rows == 0) return st;
    a.res_out = io->res_out; a.ld_out = io->ld_res_out; a.h = io->h; a.ld_h = io->ld_h;
    a.rstd_post = io->rstd_post; a.rstd_pre = io->rstd_pre;
    return launch_status(gdn::launch_block_norm(a, (cudaStream_t)stream));
}

size_t gdn_block_norm_workspace_size(int64_t rows, int32_t dim) {
    if (rows < 0 || dim <= 0 || dim > kMaxNormDim) return 0;
    return gdn::norm_bwd_ws_bytes(rows, dim) + 256;
}

gdn_status gdn_block_norm_backward(const gdn_block_norm_io *io, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    gdn::NormArgs a{};
    const gdn_status st = check_norm(io, true, &a);
    if (st != GDN_OK) return st;
    a.k_post = io->rstd_post; a.k_pre = io->rstd_pre;
    a.dh = io->dh; a.ld_dh = io->ld_dh; a.d_res_out = io->d_res_out; a.ld_dout = io->ld_d_res_out;
    a.d_res = io->d_residual; a.ld_dres = io->ld_d_residual;
    a.d_block = io->d_block; a.ld_dblock = io->ld_d_block; a.d_gate = io->d_gate; a.ld_dgate = io->ld_d_gate;
    a.dw_post = io->dw_post; a.dw_pre = io->dw_pre;
    if ((a.dw_post || a.dw_pre) && io->rows > 0) {
        if (!workspace || !aligned16(workspace) || workspace_bytes < gdn::norm_bwd_ws_bytes(io->rows, io->dim))
            return GDN_ERR_WORKSPACE;
        a.ws = (float *)workspace;
    }
    return launch_status(gdn::launch_block_norm_backward(a, (cudaStream_t)stream));
}

}  // extern "C"
