// attn_prep.cu -- norms of queries and keys for each head with the position rotation, the new keys' and
// values' way into the paged cache, and the gradients.
//
//   n = x rstd(x) w,   rstd(x) = 1 / sqrt(mean(x^2) + eps)
//   (a', b') = (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i]
//
// Backward, with g the gradient turned back by -t and x^ = x rstd:
//   dw = sum g x^,   dx = rstd (g w - x^ mean(g w x^))
//
// HBM-bound: q, k and v are read once and written once.  A warp takes a token (in small batches a part of its heads);
// D / 8 lanes own a head vector and keep it in registers.  The token's angles are computed once, a pair or a few a
// lane, and kept in registers for all its heads; the loads of the next heads are issued before a batch of them is
// worked on.
#include "attn_common.cuh"

namespace gdn {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;

// Eight neighbouring values of a head as the memory holds them.
template <typename T> struct Raw;
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) { a = load4f(p); b = load4f(p + 4); }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ __forceinline__ Raw from(int lane) const {
        Raw r;
        r.a = make_float4(__shfl_sync(0xffffffffu, a.x, lane), __shfl_sync(0xffffffffu, a.y, lane), __shfl_sync(0xffffffffu, a.z, lane),
                          __shfl_sync(0xffffffffu, a.w, lane));
        r.b = make_float4(__shfl_sync(0xffffffffu, b.x, lane), __shfl_sync(0xffffffffu, b.y, lane), __shfl_sync(0xffffffffu, b.z, lane),
                          __shfl_sync(0xffffffffu, b.w, lane));
        return r;
    }
};
template <> struct Raw<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void clear() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const float4 a = bf16x4_f32(make_uint2(u.x, u.y)), b = bf16x4_f32(make_uint2(u.z, u.w));
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ __forceinline__ Raw from(int lane) const {
        Raw r;
        r.u = make_uint4(__shfl_sync(0xffffffffu, u.x, lane), __shfl_sync(0xffffffffu, u.y, lane), __shfl_sync(0xffffffffu, u.z, lane),
                         __shfl_sync(0xffffffffu, u.w, lane));
        return r;
    }
};
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
// head 0; -1: nowhere).  Whole warps call it.
enum { kBehind = 0, kPadding = 1, kLive = 2 };
struct PrepToken {
    int kind;
    float pos;
    long long place;
};
__device__ __forceinline__ PrepToken prep_token(const AttnPrepArgs &a, long long t, bool pools) {
    PrepToken o{kBehind, 0.f, -1};
    int n = 0;
    long long j = t, L = a.T;
    if (a.cu) {
        // the last sequence that begins at or before t: 32 places at a time, so that the loads in turn are few
        int lo = 0;
        for (int count = a.n_seqs; count > 1;) {
            const int step = (count + 31) >> 5, at = lo + (int)(threadIdx.x & 31) * step;
            const bool le = at < lo + count && a.cu[at] <= t;
            const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
            lo += k * step;
            count = min(step, count - k * step);
        }
        n = lo;
        long long s, e;
        seq_bounds(a.cu, n, a.T, a.err, s, e);
        if (t < s || t >= e) return o;
        j = t - s;
        L = e - s;
    } else if (a.n_seqs > 1) {
        L = a.T / a.n_seqs;
        n = (int)t / (int)L;
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

template <int LPR> __device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// How the rotation meets a lane's 8 columns: their partners are 8 neighbours in one other lane (kLanes; most
// models), the columns next to them (kPairs), or, where half the rotated width is no multiple of 8, scattered (kAny):
// then partners come from memory, one by one.
enum { kLanes = 0, kPairs = 1, kAny = 2 };
template <int MODE, int LPR> struct Turn {
    int c0, half, from;               // the lane's first column; the partners' lane
    __device__ __forceinline__ Turn(int half_) : c0((threadIdx.x & 31) % LPR * 8), half(half_) {
        const int lane = threadIdx.x & 31;
        from = MODE != kLanes || c0 >= 2 * half ? lane : c0 < half ? lane + (half >> 3) : lane - (half >> 3);
    }
    __device__ __forceinline__ bool rotated(int e) const { return c0 + e < 2 * half; }
    __device__ __forceinline__ bool lower(int e) const { return MODE == kPairs ? !(e & 1) : MODE == kLanes ? c0 < half : c0 + e < half; }
    // the column that column e meets (itself, if it is not rotated)
    __device__ __forceinline__ int partner(int e) const {
        const int c = c0 + e;
        return !rotated(e) ? c : MODE == kPairs ? c ^ 1 : lower(e) ? c + half : c - half;
    }
    // v' = v x own + u x other with the angles of a token's pairs, `sign` -1 to turn back
    __device__ __forceinline__ void angles(const float2 *turns, float sign, float (&own)[8], float (&other)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float2 t = make_float2(1.f, 0.f);
            if (rotated(e)) t = turns[MODE == kPairs ? (c0 + e) >> 1 : lower(e) ? c0 + e : c0 + e - half];
            own[e] = t.x;
            other[e] = lower(e) ? -sign * t.y : sign * t.y;
        }
    }
    // The partners' values of a head; `p`: the head in memory, for kAny.
    template <typename T> __device__ __forceinline__ void partners(const Raw<T> &raw, const float (&v)[8], const T *p, float (&u)[8]) const {
        if (MODE == kLanes) {
            raw.from(from).get(u);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = !rotated(e) ? v[e] : MODE == kPairs ? v[e ^ 1] : to_f32(p[partner(e)]);
        }
    }
};

// A token's cosines and sines into the warp's part of shared memory.
__device__ __forceinline__ void make_turns(const AttnPrepArgs &a, float2 *turns, float pos) {
    __syncwarp();                     // the token before has been read
    for (int i = threadIdx.x & 31; i < a.half; i += 32) turns[i] = cos_sin(pos, a.inv_freq[i]);
    __syncwarp();
}

// A token's heads as a warp walks over them, HPW at a time: q's, then k's, then v's.
template <int HPW> struct Walk {
    int hq, hk, nq, nk, all;
    __device__ __forceinline__ Walk(int hq_, int hk_, int hv) : hq(hq_), hk(hk_) {
        nq = (hq + HPW - 1) / HPW;
        nk = nq + (hk + HPW - 1) / HPW;
        all = nk + (hv + HPW - 1) / HPW;
    }
    __device__ __forceinline__ int kind(int i) const { return i < nq ? 0 : i < nk ? 1 : 2; }
    __device__ __forceinline__ int head(int i, int kind, int sub) const { return (i - (kind == 0 ? 0 : kind == 1 ? nq : nk)) * HPW + sub; }
    __device__ __forceinline__ bool in(int head, int kind) const { return head < (kind == 0 ? hq : hk); }
};

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kPrepThreads, 3) attn_prep_kernel(const AttnPrepArgs a, const int split) {
    constexpr int LPR = D / 8, HPW = 32 / LPR, UN = sizeof(T) == 2 ? 4 : 2;
    extern __shared__ float2 all_turns[];                   // [warps][half]
    const int warp = threadIdx.x >> 5, sub = (threadIdx.x & 31) / LPR;
    if (blockIdx.x == 0) check_bounds(a);
    const long long id = (long long)blockIdx.x * kPrepWarps + warp, t = split == 1 ? id : id / split;
    const int part = (int)(id - t * split);
    if (t >= a.T) return;
    const bool pools = a.k_pages != nullptr;
    const Turn<MODE, LPR> rot(a.half);
    const Walk<HPW> walk(a.d.hq, a.k ? a.d.hkv : 0, pools ? a.d.hkv : 0);
    const T *q = (const T *)a.q + t * a.ld_q, *k = (const T *)a.k + t * a.ld_k, *v = (const T *)a.v + t * a.ld_v;
    auto head_at = [&](int kind, int h) { return kind == 0 ? q + h * a.hs_q : kind == 1 ? k + h * a.hs_k : v + h * a.hs_v; };
    Raw<T> next[UN];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            const int i = i0 + j * split, kind = walk.kind(i), h = walk.head(i, kind, sub);
            if (i < walk.all && walk.in(h, kind)) next[j].load(head_at(kind, h) + rot.c0);
            else next[j].clear();
        }
    };
    fetch(part);                                            // whatever the token turns out to be
    const PrepToken tok = prep_token(a, t, pools);
    if (tok.kind == kBehind) return;
    const bool live = tok.kind == kLive;
    float2 *turns = all_turns + warp * a.half;
    if (live) make_turns(a, turns, tok.pos);
    // the columns' factors: angles with the weights, of q's heads or of k's
    float own[8], other[8];
    int factors = -1;
    for (int i0 = part; i0 < walk.all; i0 += UN * split) {
        Raw<T> raw[UN];
#pragma unroll
        for (int j = 0; j < UN; ++j) raw[j] = next[j];
        if (i0 + UN * split < walk.all) fetch(i0 + UN * split);
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            const int i = i0 + j * split;
            if (i >= walk.all) break;
            const int kind = walk.kind(i), h = walk.head(i, kind, sub);
            const bool in = walk.in(h, kind);
            float x[8];
            raw[j].get(x);
            if (kind < 2) {
                const float *w = kind ? a.w_k : a.w_q;
                if (kind != factors && live) {
                    rot.angles(turns, 1.f, own, other);
                    if (w) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            own[e] *= a.offset + w[rot.c0 + e];
                            other[e] *= a.offset + w[rot.partner(e)];
                        }
                    }
                    factors = kind;
                }
                float u[8], sq = 0.f;
                rot.partners(raw[j], x, in ? head_at(kind, h) : q, u);
                float rstd = 1.f;
                if (w) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
                    rstd = rsqrtf(head_sum<LPR>(sq) * (1.f / D) + a.eps);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = live ? fmaf(x[e] * rstd, own[e], u[e] * rstd * other[e]) : 0.f;
            }
            if (in) {
                if (kind == 0) store8((T *)a.q_out + (t * a.d.hq + h) * D + rot.c0, x);
                if (kind == 1 && a.k_out) store8((T *)a.k_out + (t * a.d.hkv + h) * D + rot.c0, x);
                if (kind > 0 && tok.place >= 0)
                    store8((T *)(kind == 1 ? a.k_pages : a.v_pages) + (tok.place + (long long)h * a.d.page) * D + rot.c0, x);
            }
        }
    }
}

// A warp walks over tokens; the weights' gradients gather in registers over a token's heads of one kind, in shared
// memory over the tokens, each lane for itself, and at the end over the block in a fixed order.
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kPrepThreads, 2) attn_prep_backward_kernel(const AttnPrepArgs a) {
    constexpr int LPR = D / 8, HPW = 32 / LPR, UN = sizeof(T) == 2 ? 4 : 2;
    extern __shared__ float2 all_turns[];                   // [warps][half], then sums[2][warps][lanes][8]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR;
    float2 *turns = all_turns + warp * a.half;
    float *sums = reinterpret_cast<float *>(all_turns + kPrepWarps * a.half) + (warp * 32 + lane) * 8;
    constexpr int kKind = kPrepWarps * 32 * 8;
    if (blockIdx.x == 0) check_bounds(a);
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[e] = sums[kKind + e] = 0.f;
    const Turn<MODE, LPR> rot(a.half);
    const Walk<HPW> walk(a.d.hq, a.k ? a.d.hkv : 0, 0);
    const long long step = (long long)gridDim.x * kPrepWarps;
    for (long long t = (long long)blockIdx.x * kPrepWarps + warp; t < a.T; t += step) {
        const T *q = (const T *)a.q + t * a.ld_q, *k = (const T *)a.k + t * a.ld_k;
        const T *gq = (const T *)a.dq_out + t * a.d.hq * D, *gk = (const T *)a.dk_out + t * a.d.hkv * D;
        Raw<T> next_x[UN], next_g[UN];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                const int i = i0 + j, kind = walk.kind(i), h = walk.head(i, kind, sub);
                next_x[j].clear();
                next_g[j].clear();
                if (i < walk.all && walk.in(h, kind)) {
                    if (kind ? a.w_k : a.w_q) next_x[j].load((kind ? k + h * a.hs_k : q + h * a.hs_q) + rot.c0);
                    next_g[j].load((kind ? gk : gq) + h * D + rot.c0);
                }
            }
        };
        fetch(0);
        const PrepToken tok = prep_token(a, t, false);
        if (tok.kind == kBehind) continue;
        const bool live = tok.kind == kLive;
        if (live) make_turns(a, turns, tok.pos);
        float own[8], other[8], acc[8];
        rot.angles(turns, -1.f, own, other);
        int at = 0;                                         // whose sums are in acc
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        for (int i0 = 0; i0 < walk.all; i0 += UN) {
            Raw<T> raw_x[UN], raw_g[UN];
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                raw_x[j] = next_x[j];
                raw_g[j] = next_g[j];
            }
            if (i0 + UN < walk.all) fetch(i0 + UN);
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                const int i = i0 + j;
                if (i >= walk.all) break;
                const int kind = walk.kind(i), h = walk.head(i, kind, sub);
                const bool in = walk.in(h, kind);
                const float *w = kind ? a.w_k : a.w_q;
                if (kind != at) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sums[e] += acc[e];
                        acc[e] = 0.f;
                    }
                    at = kind;
                }
                float g[8], u[8];
                raw_g[j].get(g);
                rot.partners(raw_g[j], g, (kind ? gk : gq) + (in ? h : 0) * D, u);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = live ? fmaf(g[e], own[e], u[e] * other[e]) : 0.f;
                if (w) {
                    float x[8], sq = 0.f, dot = 0.f;
                    raw_x[j].get(x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
                    const float mean = head_sum<LPR>(sq) * (1.f / D), rstd = live && in ? rsqrtf(mean + a.eps) : 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = live ? x[e] * rstd : 0.f;
                        acc[e] = fmaf(g[e], x[e], acc[e]);
                        g[e] *= a.offset + w[rot.c0 + e];
                        dot = fmaf(g[e], x[e], dot);
                    }
                    dot = head_sum<LPR>(dot) * (1.f / D);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = rstd * (g[e] - x[e] * dot);
                }
                __syncwarp();         // the partners' gradients have been read: dq may be dq_out
                T *to = kind ? (T *)a.dk : (T *)a.dq;
                if (in && to) store8(to + t * (kind ? a.ld_dk : a.ld_dq) + h * (kind ? a.hs_dk : a.hs_dq) + rot.c0, g);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[(at ? kKind : 0) + e] += acc[e];
    }
    if (!a.ws) return;
    __syncthreads();
    const float *all = reinterpret_cast<const float *>(all_turns + kPrepWarps * a.half);
    for (int i = threadIdx.x; i < 2 * D; i += kPrepThreads) {
        const int kind = i / D, c = i - kind * D;
        float s = 0.f;
        for (int w = 0; w < kPrepWarps * HPW; ++w) s += all[kind * kKind + ((w / HPW) * 32 + (w % HPW) * LPR) * 8 + c];
        a.ws[((long long)blockIdx.x * 2 + kind) * D + c] = s;
    }
}

// Weight gradients: the blocks' sums in a fixed order.  A warp takes a column: lane i adds blocks i, i + 32, ...
__global__ void __launch_bounds__(256) attn_prep_weights_kernel(const AttnPrepArgs a, const int blocks) {
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31, kind = i / a.d.D, c = i % a.d.D;
    await_previous();
    if (kind > 1) return;
    float *to = kind ? a.dw_k : a.dw_q;
    if (!to) return;
    float s = 0.f;
    for (int b = lane; b < blocks; b += 32) s += a.ws[((long long)b * 2 + kind) * a.d.D + c];
    s = warp_sum(s);
    if (lane == 0) to[c] = s;
}

// Blocks of a backward call: as many as run at once, each over several tokens.
int backward_blocks(long long T) {
    const long long most = (long long)sm_count() * 2, all = (T + kPrepWarps - 1) / kPrepWarps;
    return (int)(all < 1 ? 1 : all < most ? all : most);
}

// Warps of a token: one, or in batches too small to fill the GPU so many that each has a head or a few.
int warps_per_token(const AttnPrepArgs &a) {
    const int heads = a.d.hq + (a.k ? a.d.hkv : 0) + (a.k_pages ? a.d.hkv : 0), hpw = 256 / a.d.D;
    const long long want = (long long)sm_count() * 24 / a.T, most = (heads + hpw - 1) / hpw;
    return (int)(want < 1 ? 1 : want < most ? want : most);
}

template <typename T, int D, int MODE> cudaError_t run_prep(const AttnPrepArgs &a, cudaStream_t s) {
    const int split = warps_per_token(a);
    const long long blocks = (a.T * split + kPrepWarps - 1) / kPrepWarps;
    attn_prep_kernel<T, D, MODE><<<(unsigned)blocks, kPrepThreads, kPrepWarps * a.half * 8, s>>>(a, split);
    return cudaGetLastError();
}
template <typename T, int D, int MODE> cudaError_t run_backward(const AttnPrepArgs &a, cudaStream_t s) {
    const int blocks = backward_blocks(a.T);
    attn_prep_backward_kernel<T, D, MODE><<<blocks, kPrepThreads, kPrepWarps * (a.half * 8 + 2 * 32 * 8 * 4), s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.ws) return e;
    return launch_early(attn_prep_weights_kernel, dim3((2 * D + 7) / 8), 256, 0, s, a, blocks);
}

int mode_of(const AttnPrepArgs &a) { return a.interleaved ? kPairs : a.half % 8 == 0 ? kLanes : kAny; }

#define GDN_PREP_MODES(RUN, T, D)                                                                    \
    return mode_of(a) == kLanes ? RUN<T, D, kLanes>(a, s) : mode_of(a) == kPairs ? RUN<T, D, kPairs>(a, s) : RUN<T, D, kAny>(a, s)
#define GDN_PREP_DIMS(RUN, T)                \
    if (a.d.D == 64) GDN_PREP_MODES(RUN, T, 64);   \
    if (a.d.D == 128) GDN_PREP_MODES(RUN, T, 128); \
    GDN_PREP_MODES(RUN, T, 256)

}  // namespace

size_t attn_prep_ws_floats(const AttnDims &d, long long T) { return (size_t)backward_blocks(T) * 2 * d.D; }

cudaError_t launch_attn_prep(const AttnPrepArgs &a, bool act_bf16, cudaStream_t s) {
    if (act_bf16) {
        GDN_PREP_DIMS(run_prep, __nv_bfloat16);
    }
    GDN_PREP_DIMS(run_prep, float);
}

cudaError_t launch_attn_prep_backward(const AttnPrepArgs &a, bool act_bf16, cudaStream_t s) {
    if (act_bf16) {
        GDN_PREP_DIMS(run_backward, __nv_bfloat16);
    }
    GDN_PREP_DIMS(run_backward, float);
}

}  // namespace gdn
