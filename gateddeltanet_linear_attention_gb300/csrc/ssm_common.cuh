// ssm_common.cuh -- arguments and device helpers of the selective state space
// mixer's kernels (gdn_ssm_* in gdn.h).
#pragma once

#include "gdn_common.cuh"

namespace gdn {

struct SsmDims {
    int groups, heads, N, P, per;   // N = d_state, P = head_dim, per = heads / groups
    int ch;                         // heads*P + 2*groups*N, channels [x | B | C]
    int n_slots;
    float dt_min, dt_max;
};

struct SsmScanArgs {
    const void *x, *b, *c, *dt, *z;   // activation dtype; z may be null
    long long ld_x, ld_bc, ld_dt, ld_z;
    const float *A_log, *dt_bias, *D; // dt_bias, D may be null
    const int32_t *cu;
    int n_seqs;
    long long T;
    const int32_t *state_idx;
    const float *state_in;
    float *state_out;
    void *y;                          // [T][heads*P] activation dtype
    SsmDims d;
    unsigned *err;
    unsigned long long wait_ns;
    // Long sequences are cut into segments of seg_len tokens (seg_len >= T: no cut, and the
    // arrays below are unused).
    long long seg_len;
    int max_enter;                    // entries of `enter`
    int *seg_base;                    // [n_seqs + 1]: segments before sequence n
    int *enter_base;                  // [n_seqs + 1]: entries of `enter` before sequence n
    float *enter;                     // [max_enter][heads][N][P]: state entering each segment of
                                      // a sequence of two segments or more
    float *seg_log;                   // [max_enter][heads]: a segment's summed log-decay
};

// Step size and log-decay of one (token, head).
__device__ __forceinline__ float ssm_dt(float raw, float bias, const SsmDims &d) {
    return fminf(fmaxf(softplus_f(raw + bias), d.dt_min), d.dt_max);
}

// Segment `b` of the batch: its sequence, tokens [t0, t1), whether it is the sequence's first or
// last one, the state slot (-1: padding lane) and the entry of `enter` that holds the state it
// starts from (-1: it starts from state_in).  False: nothing to do.
struct SsmSegment {
    int seq, slot, entry;
    long long t0, t1;
    bool first, last;
};
__device__ __forceinline__ bool ssm_segment(const SsmScanArgs &a, int b, SsmSegment &g) {
    long long s, e;
    if (a.seg_len >= a.T) {
        g.seq = b;
        seq_bounds(a.cu, b, a.T, a.err, s, e);
        g.t0 = s; g.t1 = e; g.first = g.last = true; g.entry = -1;
    } else {
        if (b >= a.seg_base[a.n_seqs]) return false;
        int lo = 0, hi = a.n_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.seg_base[mid] <= b) lo = mid; else hi = mid - 1;
        }
        g.seq = lo;
        seq_bounds(a.cu, lo, a.T, a.err, s, e);
        const int k = b - a.seg_base[lo], count = a.seg_base[lo + 1] - a.seg_base[lo];
        // malformed lengths (already reported): what has no room is not run
        if (count > 1 && a.enter_base[lo] + count > a.max_enter) return false;
        g.t0 = s + (long long)k * a.seg_len;
        g.t1 = g.t0 + a.seg_len < e ? g.t0 + a.seg_len : e;
        g.first = k == 0;
        g.last = k == count - 1;
        g.entry = count > 1 ? a.enter_base[lo] + k : -1;
    }
    g.slot = slot_of(a.state_idx, g.seq, a.d.n_slots, a.err);
    return true;
}

// Sigmoid and SiLU of values that end in the type T: through the approximate exp and quotient
// (relative error below 2e-6 where the result matters) for 16-bit results, whose half step is
// 4e-3; through the accurate ones for 32-bit results.
template <typename T> __device__ __forceinline__ float sigmoid_for(float x) { return sigmoid_f(x); }
template <> __device__ __forceinline__ float sigmoid_for<__nv_bfloat16>(float x) {
    return __fdividef(1.0f, 1.0f + __expf(-x));
}
template <typename T> __device__ __forceinline__ float silu_for(float x) { return silu_f(x); }
template <> __device__ __forceinline__ float silu_for<__nv_bfloat16>(float x) { return silu_fast(x); }

// Row vectors of four elements.
__device__ __forceinline__ float4 load4f(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 bf16x4_f32(uint2 v) {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4f(const __nv_bfloat16 *p) {
    return bf16x4_f32(*reinterpret_cast<const uint2 *>(p));
}
__device__ __forceinline__ void store4f(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4f(__nv_bfloat16 *p, float4 v) {
    __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(h);
}

struct SsmConvArgs {
    const void *x;
    long long ld_x;
    const int32_t *cu;
    int n_seqs;
    long long T;
    const void *w, *bias;             // [CH][4], [CH] activation dtype; bias may be null
    void *conv_state;                 // may be null (zero history, not written)
    const int32_t *state_idx;
    void *out;                        // [T][CH]
    SsmDims d;
    unsigned *err;
};

struct SsmStepArgs {
    const void *x, *dt, *z;           // raw channels [n][ld_x]; z may be null
    long long ld_x, ld_dt, ld_z;
    const void *w, *bias;
    void *conv_state;
    const float *A_log, *dt_bias, *D;
    int n;
    const int32_t *state_idx;
    float *state;
    void *y;
    float *ws;                        // [n][CH]: channels after the convolution
    SsmDims d;
    unsigned *err;
};

// Workspace for up to T tokens and n_seqs sequences; and the cut of a batch, its arrays laid out
// in ws (unless null), with the bytes that this batch needs.
size_t ssm_scan_ws_bytes(const SsmDims &d, bool act_bf16, long long T, long long n_seqs);
size_t ssm_scan_carve(SsmScanArgs &a, bool act_bf16, void *ws);
cudaError_t launch_ssm_scan(const SsmScanArgs &a, bool act_bf16, cudaStream_t s);
// The tensor-core form (bf16 activations): a unit is 128 value columns of a group's heads.
bool ssm_tc_supported(const SsmDims &d);
int ssm_tc_units(const SsmDims &d);
cudaError_t launch_ssm_scan_tc(const SsmScanArgs &a, bool states, unsigned segments, cudaStream_t s);
cudaError_t launch_ssm_conv(const SsmConvArgs &a, bool act_bf16, cudaStream_t s);
size_t ssm_step_ws_bytes(const SsmDims &d, long long n);
cudaError_t launch_ssm_step(const SsmStepArgs &a, bool act_bf16, cudaStream_t s);

// A gated post-norm, residual add and pre-norm over rows (gdn_block_norm and its backward).
struct NormArgs {
    long long rows;
    int dim;
    bool act_bf16, res_bf16;
    float eps, offset, scale;
    const void *block, *gate, *residual;
    long long ld_block, ld_gate, ld_res, ld_out, ld_h;
    int gate_cols;
    const float *w_post, *w_pre;
    void *res_out, *h;
    float *rstd_post, *rstd_pre;
    // backward
    const float *k_post, *k_pre;      // the forward's rstd values
    const void *dh, *d_res_out;
    long long ld_dh, ld_dout, ld_dres, ld_dblock, ld_dgate;
    void *d_res, *d_block, *d_gate;
    float *dw_post, *dw_pre;
    float *ws;
    bool vec;                         // every row starts on 16 bytes and dim % 8 == 0
};
size_t norm_bwd_ws_bytes(long long rows, int dim);
cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s);
cudaError_t launch_block_norm_backward(const NormArgs &a, cudaStream_t s);

// The device error word of the current device, and the limit of bounded waits.
gdn_status device_error_word(unsigned **out);
unsigned long long wait_limit_ns();
}  // namespace gdn
