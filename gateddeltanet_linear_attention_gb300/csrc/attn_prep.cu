// attn_prep.cu -- norms of queries and keys for each head with the position rotation, the new keys' and
// values' way into the paged cache, and the gradients.
//
//   n = x rstd(x) w,   rstd(x) = 1 / sqrt(mean(x^2) + eps)
//   (a', b') = (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i]
//
// Backward, with g the gradient turned back by -t and x^ = x rstd:
//   dw = sum g x^,   dx = rstd (g w - x^ mean(g w x^))
//
// HBM-bound: q, k and v are read once and written once.  D / 8 lanes own a head vector and keep it in registers;
// a block takes a few tokens, whose angles are computed once and shared by all heads.
#include "attn_common.cuh"

namespace gdn {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepTokens = 8;       // most tokens of a block

__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = load4f(p), b = load4f(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const float4 a = bf16x4_f32(make_uint2(u.x, u.y)), b = bf16x4_f32(make_uint2(u.z, u.w));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    store4f(p, make_float4(v[0], v[1], v[2], v[3]));
    store4f(p + 4, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    __nv_bfloat162 h[4] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3]),
                           __floats2bfloat162_rn(v[4], v[5]), __floats2bfloat162_rn(v[6], v[7])};
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(h);
}

// a + b = sum + rest exactly.
__device__ __forceinline__ float two_sum(float a, float b, float &rest) {
    const float sum = a + b, back = sum - a;
    rest = (a - (sum - back)) + (b - back);
    return sum;
}

// cos and sin of p f, p a whole number below 2^24.  The product is taken exactly (p f = hi + lo; lo is as large as hi's
// last place, 2 at the far end), whole turns are taken off hi by Cody and Waite's method (2 pi in three parts, the first
// two of 24 bits; hi - k C1 is exact: both are multiples of C1's last place, and they are near each other), the rest is
// added up with its rounding errors, and these go in by the angle sum to first order.  So far positions are as exact as
// near ones: 1e-7.
__device__ __forceinline__ float2 cos_sin(float p, float f) {
    constexpr double kTurn = 6.283185307179586476925;
    constexpr float C1 = (float)kTurn, C2 = (float)(kTurn - (double)C1), C3 = (float)(kTurn - (double)C1 - (double)C2);
    const float hi = p * f, lo = fmaf(p, f, -hi);
    const float k = rintf(hi * (float)(1.0 / kTurn));
    const float t = -k * C2, t_lo = fmaf(-k, C2, -t);
    float e0, e1;
    const float s = two_sum(two_sum(fmaf(-k, C1, hi), lo, e0), t, e1);
    const float rest = (e0 + e1) + fmaf(-k, C3, t_lo);
    float sn, cs;
    sincosf(s, &sn, &cs);
    return make_float2(fmaf(-rest, sn, cs), fmaf(rest, cs, sn));
}

// What a token is: its kind, position, and where its key and value go (in rows of D elements of the pools, for key
// head 0; -1: nowhere).
enum { kBehind = 0, kPadding = 1, kLive = 2 };
struct PrepToken {
    int kind;
    float pos;
    long long place;
};
__device__ PrepToken prep_token(const AttnPrepArgs &a, long long t, bool pools) {
    PrepToken o{kBehind, 0.f, -1};
    if (t >= a.T) return o;
    int n = 0;
    long long j = t, L = a.T;
    if (a.cu) {
        // the last sequence that begins at or before t
        int lo = 0, hi = a.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        n = lo;
        long long s, e;
        seq_bounds(a.cu, n, a.T, a.err, s, e);
        if (t < s || t >= e) return o;
        j = t - s;
        L = e - s;
    } else {
        L = a.T / a.n_seqs;
        n = (int)(t / L);
        j = t - n * L;
    }
    o.kind = kPadding;
    long long at = j;
    int row = n;
    if (a.lens) {
        row = attn_row(a.rows, n, a.d, a.err);
        if (row < 0) return o;
        const int len = a.lens[row];
        at = (long long)len - L + j;
        if (at < 0 || (pools && len > a.d.max_pages * a.d.page)) {
            set_error(a.err, GDN_DEVERR_PAGE);
            return o;
        }
    } else if (a.rows && attn_row(a.rows, n, a.d, a.err) < 0) {
        return o;
    }
    const long long pos = a.positions ? a.positions[t] : at;
    if (pos < 0) return o;
    if (pos >= kMaxPosition) {
        set_error(a.err, GDN_DEVERR_PAGE);
        return o;
    }
    o.kind = kLive;
    o.pos = (float)(int)pos;
    if (pools) {
        const int page = a.table[(long long)row * a.d.max_pages + (at >> a.d.page_shift)];
        if (page < 0 || page >= a.d.n_pages) set_error(a.err, GDN_DEVERR_PAGE);
        else o.place = (long long)page * a.d.hkv * a.d.page + (at & (a.d.page - 1));
    }
    return o;
}

// Reports malformed cu_seqlens wherever they are, not only where a token meets them (one block).
__device__ void check_bounds(const AttnPrepArgs &a) {
    if (!a.cu) return;
    for (int n = threadIdx.x; n < a.n_seqs; n += blockDim.x) {
        long long s, e;
        seq_bounds(a.cu, n, a.T, a.err, s, e);
        if (n == 0 && a.cu[0] != 0) set_error(a.err, GDN_DEVERR_CU_SEQLENS);
    }
}

// The partner of each of a lane's 8 columns under the rotation, and its cos and sign * sin: out = v cos + partner sin.
// Columns that are not rotated get cos 1 and sin 0.  `turn` +1 forward, -1 backward.
struct Rotation {
    int half;
    bool interleaved, lanes;          // lanes: partners 8 neighbours in one other lane
    int c0;                           // the lane's first column
    __device__ __forceinline__ Rotation(const AttnPrepArgs &a, int l) : half(a.half), interleaved(a.interleaved), c0(l * 8) {
        lanes = !interleaved && (half & 7) == 0;
    }
    // lane that holds the partners (relative to the head's first lane)
    __device__ __forceinline__ int partner_lane(int l) const {
        return c0 < half ? l + (half >> 3) : c0 < 2 * half ? l - (half >> 3) : l;
    }
    __device__ __forceinline__ bool rotated(int e) const { return c0 + e < 2 * half; }
    __device__ __forceinline__ int partner(int e) const {
        const int c = c0 + e;
        return interleaved ? c ^ 1 : c < half ? c + half : c - half;
    }
    __device__ __forceinline__ bool lower(int e) const { return interleaved ? !((c0 + e) & 1) : c0 + e < half; }
    __device__ __forceinline__ int pair(int e) const {
        const int c = c0 + e;
        return interleaved ? c >> 1 : c < half ? c : c - half;
    }
    // v: own values, u: the partners'; cs: cos and sin of the token's pairs
    __device__ __forceinline__ void turn(float (&v)[8], const float (&u)[8], const float2 *cs, float sign) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (rotated(e)) {
                const float2 t = cs[pair(e)];
                const float sn = lower(e) ? -sign * t.y : sign * t.y;
                v[e] = fmaf(v[e], t.x, u[e] * sn);
            }
        }
    }
};

template <int LPR> __device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The values of a head's partner columns: from the partner lane, from the lane itself (neighbouring pairs), or,
// where pairs of 8 do not fall together, from memory (`at(column)`).
template <int LPR, typename F>
__device__ __forceinline__ void partners(const Rotation &rot, const float (&v)[8], float (&u)[8], int l, F at) {
    if (rot.lanes) {
        const int from = (threadIdx.x & 31 & ~(LPR - 1)) + rot.partner_lane(l);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = __shfl_sync(0xffffffffu, v[e], from);
    } else if (rot.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = v[e ^ 1];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = rot.rotated(e) ? at(rot.partner(e)) : 0.f;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrepThreads) attn_prep_kernel(const AttnPrepArgs a, const int per_block) {
    constexpr int LPR = D / 8, GROUPS = kPrepThreads / LPR;
    extern __shared__ float2 turns[];                       // [per_block][half]
    __shared__ PrepToken tokens[kPrepTokens];
    const int tid = threadIdx.x, group = tid / LPR, l = tid % LPR;
    const long long t0 = (long long)blockIdx.x * per_block;
    const bool pools = a.k_pages != nullptr;
    if (blockIdx.x == 0) check_bounds(a);
    if (tid < per_block) tokens[tid] = prep_token(a, t0 + tid, pools);
    __syncthreads();
    for (int i = tid; i < per_block * a.half; i += kPrepThreads) {
        const int k = i / a.half;
        if (tokens[k].kind == kLive) turns[i] = cos_sin(tokens[k].pos, a.inv_freq[i - k * a.half]);
    }
    __syncthreads();
    const Rotation rot(a, l);
    const int heads = a.d.hq + (a.k ? a.d.hkv : 0) + (pools ? a.d.hkv : 0);
    const int items = per_block * heads;
    // whole warps walk together: a group without an item repeats the last one's loads and stores nothing
    for (int i0 = 0; i0 < items; i0 += GROUPS) {
        const bool mine = i0 + group < items;
        const int i = mine ? i0 + group : items - 1, k = i / heads;
        int h = i - k * heads;
        const long long t = t0 + k;
        const PrepToken tok = tokens[k];
        const bool live = mine && tok.kind == kLive;
        const int what = h < a.d.hq ? 0 : h < a.d.hq + a.d.hkv ? 1 : 2;      // q, k, v
        h -= what == 0 ? 0 : what == 1 ? a.d.hq : a.d.hq + a.d.hkv;
        const T *src = what == 0 ? (const T *)a.q + t * a.ld_q + h * a.hs_q
                     : what == 1 ? (const T *)a.k + t * a.ld_k + h * a.hs_k : (const T *)a.v + t * a.ld_v + h * a.hs_v;
        float v[8] = {};
        if (live) load8(src + l * 8, v);
        const float *w = what == 0 ? a.w_q : what == 1 ? a.w_k : nullptr;
        float sq = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(v[e], v[e], sq);
        const float mean = head_sum<LPR>(sq) * (1.f / D), rstd = live ? rsqrtf(mean + a.eps) : 0.f;
        if (w) {
            float wv[8];
            load8(w + l * 8, wv);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * (a.offset + wv[e]);
        }
        float u[8];
        partners<LPR>(rot, v, u, l, [&](int c) {
            const float x = live ? to_f32(src[c]) : 0.f;
            return w ? x * rstd * (a.offset + w[c]) : x;
        });
        if (what != 2 && live) rot.turn(v, u, turns + k * a.half, 1.f);
        if (!mine || tok.kind == kBehind) continue;
        if (what == 0) store8((T *)a.q_out + (t * a.d.hq + h) * D + l * 8, v);
        if (what == 1 && a.k_out) store8((T *)a.k_out + (t * a.d.hkv + h) * D + l * 8, v);
        if (what != 0 && pools && tok.place >= 0)
            store8((T *)(what == 1 ? a.k_pages : a.v_pages) + (tok.place + (long long)h * a.d.page) * D + l * 8, v);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrepThreads) attn_prep_backward_kernel(const AttnPrepArgs a, const int per_block) {
    constexpr int LPR = D / 8, GROUPS = kPrepThreads / LPR;
    extern __shared__ float2 turns[];                       // [per_block][half]; at the end sums[GROUPS][D]
    __shared__ PrepToken tokens[kPrepTokens];
    const int tid = threadIdx.x, group = tid / LPR, l = tid % LPR;
    if (blockIdx.x == 0) check_bounds(a);
    const Rotation rot(a, l);
    const int heads = a.d.hq + (a.k ? a.d.hkv : 0), items = per_block * heads;
    float sum[2][8] = {};
    for (long long t0 = (long long)blockIdx.x * per_block; t0 < a.T; t0 += (long long)gridDim.x * per_block) {
        __syncthreads();
        if (tid < per_block) tokens[tid] = prep_token(a, t0 + tid, false);
        __syncthreads();
        for (int i = tid; i < per_block * a.half; i += kPrepThreads) {
            const int k = i / a.half;
            if (tokens[k].kind == kLive) turns[i] = cos_sin(tokens[k].pos, a.inv_freq[i - k * a.half]);
        }
        __syncthreads();
        for (int i0 = 0; i0 < items; i0 += GROUPS) {
            const bool mine = i0 + group < items;
            const int i = mine ? i0 + group : items - 1, k = i / heads;
            const bool key = i - k * heads >= a.d.hq;
            const int h = i - k * heads - (key ? a.d.hq : 0);
            const long long t = t0 + k;
            const PrepToken tok = tokens[k];
            const bool live = mine && tok.kind == kLive;
            const T *src = key ? (const T *)a.k + t * a.ld_k + h * a.hs_k : (const T *)a.q + t * a.ld_q + h * a.hs_q;
            const T *grad = (key ? (const T *)a.dk_out + (t * a.d.hkv + h) * D : (const T *)a.dq_out + (t * a.d.hq + h) * D);
            float x[8] = {}, g[8] = {}, u[8];
            const float *w = key ? a.w_k : a.w_q;
            if (live) {
                load8(grad + l * 8, g);
                if (w) load8(src + l * 8, x);
            }
            partners<LPR>(rot, g, u, l, [&](int c) { return live ? to_f32(grad[c]) : 0.f; });
            if (live) rot.turn(g, u, turns + k * a.half, -1.f);
            // heads of q and of k may stand in one warp, so all take the sums, with weights or not
            float gw[8], sq = 0.f, dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
            sq = head_sum<LPR>(sq) * (1.f / D);
            const float rstd = live ? rsqrtf(sq + a.eps) : 0.f;
            if (w) load8(w + l * 8, gw);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] *= rstd;
                if (live) sum[key][e] = fmaf(g[e], x[e], sum[key][e]);
                gw[e] = w ? g[e] * (a.offset + gw[e]) : 0.f;
                dot = fmaf(gw[e], x[e], dot);
            }
            dot = head_sum<LPR>(dot) * (1.f / D);
            if (w) {
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = rstd * (gw[e] - x[e] * dot);
            }
            T *to = key ? (T *)a.dk : (T *)a.dq;
            __syncwarp();         // the partners' gradients have been read: `to` may be where they stand
            if (mine && tok.kind != kBehind && to)
                store8(to + t * (key ? a.ld_dk : a.ld_dq) + h * (key ? a.hs_dk : a.hs_dq) + l * 8, g);
        }
    }
    if (!a.ws) return;
    // sums over the block's groups in order, q's weights then k's
    float *sums = reinterpret_cast<float *>(turns);
    for (int key = 0; key < 2; ++key) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[group * D + l * 8 + e] = sum[key][e];
        __syncthreads();
        if (tid < D) {
            float s = 0.f;
            for (int g = 0; g < GROUPS; ++g) s += sums[g * D + tid];
            a.ws[((long long)blockIdx.x * 2 + key) * D + tid] = s;
        }
    }
}

// Weight gradients: the blocks' sums in a fixed order.  A warp takes a column: lane i adds blocks i, i + 32, ...
__global__ void __launch_bounds__(256) attn_prep_weights_kernel(const AttnPrepArgs a, const int blocks) {
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31, key = i / a.d.D, col = i % a.d.D;
    await_previous();
    if (key > 1) return;
    float *to = key ? a.dw_k : a.dw_q;
    if (!to) return;
    float s = 0.f;
    for (int b = lane; b < blocks; b += 32) s += a.ws[((long long)b * 2 + key) * a.d.D + col];
    s = warp_sum(s);
    if (lane == 0) to[col] = s;
}

// Blocks of a backward call: as many as run at once, each over several tokens.
int backward_blocks(long long T) {
    const long long most = (long long)sm_count() * 4;
    return (int)(T < most ? (T > 0 ? T : 1) : most);
}

int tokens_per_block(long long T) {
    long long k = T / ((long long)sm_count() * 8);
    return (int)(k < 1 ? 1 : k > kPrepTokens ? kPrepTokens : k);
}

template <typename T, int D> cudaError_t run_prep(const AttnPrepArgs &a, cudaStream_t s) {
    const int per = tokens_per_block(a.T);
    attn_prep_kernel<T, D><<<(unsigned)((a.T + per - 1) / per), kPrepThreads, per * a.half * 8, s>>>(a, per);
    return cudaGetLastError();
}
template <typename T, int D> cudaError_t run_backward(const AttnPrepArgs &a, cudaStream_t s) {
    constexpr int sums = kPrepThreads / (D / 8) * D * 4;
    const int blocks = backward_blocks(a.T);
    int per = (int)((a.T + blocks - 1) / blocks);
    per = per > kPrepTokens ? kPrepTokens : per < 1 ? 1 : per;
    const int angles = per * a.half * 8;
    attn_prep_backward_kernel<T, D><<<blocks, kPrepThreads, angles > sums ? angles : sums, s>>>(a, per);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.ws) return e;
    return launch_early(attn_prep_weights_kernel, dim3((2 * D + 7) / 8), 256, 0, s, a, blocks);
}

}  // namespace

size_t attn_prep_ws_floats(const AttnDims &d, long long T) { return (size_t)backward_blocks(T) * 2 * d.D; }

cudaError_t launch_attn_prep(const AttnPrepArgs &a, bool act_bf16, cudaStream_t s) {
    if (act_bf16)
        return a.d.D == 64 ? run_prep<__nv_bfloat16, 64>(a, s) : a.d.D == 128 ? run_prep<__nv_bfloat16, 128>(a, s)
                                                                              : run_prep<__nv_bfloat16, 256>(a, s);
    return a.d.D == 64 ? run_prep<float, 64>(a, s) : a.d.D == 128 ? run_prep<float, 128>(a, s) : run_prep<float, 256>(a, s);
}

cudaError_t launch_attn_prep_backward(const AttnPrepArgs &a, bool act_bf16, cudaStream_t s) {
    if (act_bf16)
        return a.d.D == 64 ? run_backward<__nv_bfloat16, 64>(a, s) : a.d.D == 128 ? run_backward<__nv_bfloat16, 128>(a, s)
                                                                                  : run_backward<__nv_bfloat16, 256>(a, s);
    return a.d.D == 64 ? run_backward<float, 64>(a, s) : a.d.D == 128 ? run_backward<float, 128>(a, s) : run_backward<float, 256>(a, s);
}

}  // namespace gdn
