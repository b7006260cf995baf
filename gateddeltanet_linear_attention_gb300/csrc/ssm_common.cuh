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
    unsigned long long wait_ns;       // limit of bounded waits, and the copies a test drops
    unsigned lose;
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

// Step size of one (token, head); NaN stays NaN.
__device__ __forceinline__ float ssm_dt(float raw, float bias, const SsmDims &d) {
    const float dt = softplus_f(raw + bias);
    return dt < d.dt_min ? d.dt_min : dt > d.dt_max ? d.dt_max : dt;
}

// How a batch is cut: every sequence has one segment or more (one of an empty sequence), and a
// sequence of two or more keeps the states that enter them, side by side in `enter`.  Batches of
// up to kWarpSeqs sequences are laid out by every warp for itself, longest sequence first so that
// the last CTAs to start are short ones; larger ones in order, by ssm_segment_map_kernel if cut.
constexpr int kWarpSeqs = 32;
struct SsmCut {
    int seg0, segs, entry0;           // first segment, segments; first entry of `enter`, -1: none
    int front0;                       // segments before it that are not their sequence's last
};
// The cut of sequence `lane` (n_seqs <= kWarpSeqs; a whole warp calls it).
__device__ __forceinline__ SsmCut ssm_warp_cut(const SsmScanArgs &a, int lane) {
    long long len = -1;
    if (lane < a.n_seqs) {
        long long s, e;
        seq_bounds(a.cu, lane, a.T, a.err, s, e);
        len = e - s;
    }
    const int segs = lane >= a.n_seqs ? 0 : len <= a.seg_len ? 1 : (int)((len + a.seg_len - 1) / a.seg_len);
    SsmCut c{0, segs, 0, 0};
    for (int m = 0; m < a.n_seqs; ++m) {
        const long long other = __shfl_sync(0xffffffffu, len, m);
        const int count = __shfl_sync(0xffffffffu, segs, m);
        if (other > len || (other == len && m < lane)) {
            c.seg0 += count;
            c.entry0 += count > 1 ? count : 0;
            c.front0 += count - 1;
        }
    }
    if (segs < 2) c.entry0 = -1;
    return c;
}

// Segment `b` of the batch, or (FRONT) of its segments that are not their sequence's last: its
// sequence, tokens [t0, t1), its index there and whether it is the last one, the state slot (-1:
// padding lane) and the entry of `enter` that holds the state it starts from (-1: it starts from
// state_in).  False: nothing to do.  Whole warps call it.
struct SsmSegment {
    int seq, slot, entry, index;
    long long t0, t1;
    bool last;
};
template <bool FRONT> __device__ __forceinline__ bool ssm_segment(const SsmScanArgs &a, int b, SsmSegment &g) {
    SsmCut c{b, 1, -1, 0};
    g.seq = b;
    int k = 0;
    if (a.n_seqs <= kWarpSeqs) {
        c = ssm_warp_cut(a, threadIdx.x & 31);
        k = FRONT ? b - c.front0 : b - c.seg0;
        const unsigned mine = __ballot_sync(0xffffffffu, k >= 0 && k < (FRONT ? c.segs - 1 : c.segs));
        if (mine == 0) return false;
        g.seq = __ffs(mine) - 1;
        k = __shfl_sync(0xffffffffu, k, g.seq);
        c.segs = __shfl_sync(0xffffffffu, c.segs, g.seq);
        c.entry0 = __shfl_sync(0xffffffffu, c.entry0, g.seq);
    } else if (a.seg_len < a.T) {
        // seg_base[n], less n for the front segments: every sequence has one last segment
        if (b >= a.seg_base[a.n_seqs] - (FRONT ? a.n_seqs : 0)) return false;
        // the last sequence whose base is not beyond b: 32 places at a time, so that the loads in
        // turn are few (one in turn per halving: 200 sequences of 8 tokens took 57 us more)
        int lo = 0;
        for (int count = a.n_seqs; count > 1;) {
            const int step = (count + 31) >> 5, at = lo + (int)(threadIdx.x & 31) * step;
            const bool le = at < lo + count && a.seg_base[at] - (FRONT ? at : 0) <= b;
            const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
            lo += k * step;
            count = min(step, count - k * step);
        }
        g.seq = lo;
        k = b - (a.seg_base[lo] - (FRONT ? lo : 0));
        c.segs = a.seg_base[lo + 1] - a.seg_base[lo];
        if (c.segs > 1) c.entry0 = a.enter_base[lo];
    }
    // malformed lengths (reported below or by the map): what has no room is not run
    if (c.entry0 >= 0 && c.entry0 + c.segs > a.max_enter) {
        set_error(a.err, GDN_DEVERR_CU_SEQLENS);
        return false;
    }
    long long s, e;
    seq_bounds(a.cu, g.seq, a.T, a.err, s, e);
    g.t0 = s + (long long)k * a.seg_len;
    g.t1 = g.t0 + a.seg_len < e ? g.t0 + a.seg_len : e;
    if (g.t0 > g.t1) return false;
    g.index = k;
    g.last = k == c.segs - 1;
    g.entry = c.entry0 >= 0 ? c.entry0 + k : -1;
    g.slot = slot_of(a.state_idx, g.seq, a.d.n_slots, a.err);
    return true;
}

// Two packed fp32 values: one instruction for two multiply-adds.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^x to two units in the last place.  exp(x) through it is off by |x| 2^-24 more.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// Sigmoid and SiLU of values that end in the type T: through the approximate exp and reciprocal
// (relative error below 2e-6 where the result matters) for 16-bit results, whose half step is
// 4e-3; through the accurate ones for 32-bit results.
template <typename T> __device__ __forceinline__ float sigmoid_for(float x) { return sigmoid_f(x); }
template <> __device__ __forceinline__ float sigmoid_for<__nv_bfloat16>(float x) {
    return rcp_fast(1.0f + exp2_fast(-kLog2e * x));
}
template <typename T> __device__ __forceinline__ float silu_for(float x) { return silu_f(x); }
template <> __device__ __forceinline__ float silu_for<__nv_bfloat16>(float x) { return x * sigmoid_for<__nv_bfloat16>(x); }
// sigmoid(x) and 1 - sigmoid(x) without the difference, so that the gradient of a gate that is all but
// open keeps its digits: 1 / (1 + e) and e / (1 + e) with e = exp(-|x|), which is which by x's sign.
// NaN stays NaN.
__device__ __forceinline__ void sigmoid_pair(float x, float &s, float &rest) {
    const float e = expf(-fabsf(x)), most = 1.0f / (1.0f + e), least = e * most;
    s = x < 0.f ? least : most;
    rest = x < 0.f ? most : least;
}
// The same of two gates for 16-bit results, e = exp(-x): fewer instructions.  Below -88, where the sigmoid
// leaves the normal numbers, both are 0 (1 - sigmoid is a factor beside the sigmoid only).  dw_post, 32
// bits, sums terms of it too: each is off by 2 + 1.2 |x| units in the last place.
__device__ __forceinline__ void sigmoid_pairs_fast(float x0, float x1, f32x2 &s, f32x2 &rest) {
    float t0, t1;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(t0) : "f"(-kLog2e * x0), "f"(127.5f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(t1) : "f"(-kLog2e * x1), "f"(127.5f));
    const f32x2 e = pack2(exp2_fast(t0), exp2_fast(t1));
    const float2 q = unpack2(add2(e, pack2(1.0f, 1.0f)));
    s = pack2(rcp_fast(q.x), rcp_fast(q.y));
    rest = mul2(e, s);
}

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

// Launch a kernel that may start before the one in front of it in the stream ends
// (programmatic dependent launch).  It calls await_previous() before it touches what that one
// writes, and at the latest before it ends, so that the order of the stream holds for what follows.
template <typename... A>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t s, const A &...args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
unsigned lost_copies();
}  // namespace gdn
