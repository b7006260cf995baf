// attn_prep.cu -- norms of queries and keys for each head with the position rotation, the new keys' and
// values' way into the paged cache, and the gradients.
//
//   n = x rstd(x) w,   rstd(x) = 1 / sqrt(mean(x^2) + eps)
//   (a', b') = (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i]
//
// Backward, with g the gradient turned back by -t and x^ = x rstd:
//   dw = sum g x^,   dx = rstd (g w - x^ mean(g w x^))
//
// HBM-bound: q, k and v are read once and written once.  D / 8 lanes own a head vector and keep it in registers.  A
// warp takes a few tokens at a time: what they are and their angles come first, a lane a token, then a lane an angle;
// then it goes through their heads in batches, the next batches (of the next kind of heads, of the next token) under way:
// forward four, by asynchronous copies of each lane's pieces to shared memory, backward one, in registers.  No warp waits for
// another.  Tokens that share a block's angles instead took 70 us where this takes 36.
//
// Measured in bf16: 9,600 prompt tokens into the cache (16 + 2 + 2 heads of 256, 64 columns rotated) 36 us, 0.81 of the copy
// rate, issue used by 0.55 (one batch of four heads ahead in registers 40, two to four of them in shared memory 36 to 38; three
// blocks an SM 47 to 53: spills); the backward of 8,192
// tokens (32 + 8 heads of 128) 56 us, 0.66, issue used by 0.57; 64 tokens of a decode step 5.2 us.  Of 32 + 8 heads of 128, all
// columns rotated, 6,905 tokens forward (floor 21, fp32 42) and 8,192 backward (floor 37, fp32 74), in us: halves 27 and 56 (fp32 49
// and 87), neighbouring pairs 30 and 62 (70 and 96), half of 50 columns 74 and 128 (97 and 150): its partners come from memory one by
// one.  The backward kernels of the pairs and of the free width spill 64 to 144 bytes.
#include <type_traits>

#include "attn_common.cuh"

namespace gdn {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepWarps = kPrepThreads / 32;
constexpr int kPrepBlocks = 2;       // of the forward kernel on an SM

// A lane's eight values of a head, two pieces of four, as the memory holds them and as pairs for the packed
// multiply-adds.
template <typename T> struct Raw;
template <> struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p, const float *q) { a = load4f(p); b = load4f(q); }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(f32x2 (&v)[4]) const {
        v[0] = pack2(a.x, a.y); v[1] = pack2(a.z, a.w); v[2] = pack2(b.x, b.y); v[3] = pack2(b.z, b.w);
    }
    __device__ __forceinline__ void store(float *p, float *q) const { store4f(p, a); store4f(q, b); }
};
template <> struct Raw<__nv_bfloat16> {
    uint2 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, const __nv_bfloat16 *q) {
        a = *reinterpret_cast<const uint2 *>(p);
        b = *reinterpret_cast<const uint2 *>(q);
    }
    __device__ __forceinline__ void clear() { a = b = make_uint2(0u, 0u); }
    static __device__ __forceinline__ f32x2 pair(uint32_t x) { return pack2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)); }
    __device__ __forceinline__ void get(f32x2 (&v)[4]) const { v[0] = pair(a.x); v[1] = pair(a.y); v[2] = pair(b.x); v[3] = pair(b.y); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p, __nv_bfloat16 *q) const {
        *reinterpret_cast<uint2 *>(p) = a;
        *reinterpret_cast<uint2 *>(q) = b;
    }
};
__device__ __forceinline__ void store8(float *p, float *q, const f32x2 (&v)[4]) {
    const float2 a = unpack2(v[0]), b = unpack2(v[1]), c = unpack2(v[2]), d = unpack2(v[3]);
    store4f(p, make_float4(a.x, a.y, b.x, b.y));
    store4f(q, make_float4(c.x, c.y, d.x, d.y));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, __nv_bfloat16 *q, const f32x2 (&v)[4]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __float22bfloat162_rn(unpack2(v[j]));
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(h);
    *reinterpret_cast<uint2 *>(q) = *reinterpret_cast<const uint2 *>(h + 2);
}
__device__ __forceinline__ f32x2 both(float x) { return pack2(x, x); }
// Sum of the products of two rows of eight.
__device__ __forceinline__ float dot8(const f32x2 (&a)[4], const f32x2 (&b)[4]) {
    f32x2 s = mul2(a[0], b[0]), t = mul2(a[1], b[1]);
    s = fma2(a[2], b[2], s);
    t = fma2(a[3], b[3], t);
    const float2 r = unpack2(add2(s, t));
    return r.x + r.y;
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
    // in half turns, whose sine and cosine need no further reduction
    constexpr double kInv = 1.0 / 3.14159265358979323846;
    constexpr float I1 = (float)kInv, I2 = (float)(kInv - (double)I1);
    const float y = s * I1, y_lo = fmaf(s, I1, -y) + fmaf(s, I2, rest * I1);
    float sn, cs;
    sincospif(y, &sn, &cs);
    const float d = y_lo * (float)(kTurn / 2);
    return make_float2(fmaf(-d, sn, cs), fmaf(d, cs, sn));
}

// What a token is: its kind and position, and where its key and value go (in rows of D elements of the pools, for key
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
    long long at = t, L = a.T;
    if (a.cu) {
        // the last sequence that begins at or before t
        for (int count = a.n_seqs; count > 1;) {
            const int half = count >> 1;
            if (a.cu[n + half] <= t) {
                n += half;
                count -= half;
            } else {
                count = half;
            }
        }
        long long s, e;
        seq_bounds(a.cu, n, a.T, a.err, s, e);
        if (t < s || t >= e) return o;
        at = t - s;
        L = e - s;
    } else if (a.n_seqs > 1) {
        L = a.T / a.n_seqs;
        n = (int)t / (int)L;
        at = t - n * L;
    }
    o.kind = kPadding;
    int row = n;
    if (a.lens) {
        row = attn_row(a.rows, n, a.d, a.err);
        if (row < 0) return o;
        const int len = a.lens[row];
        at += (long long)len - L;
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

// Which 8 columns of a head a lane has, and where their partners under the rotation are.
//   kHalves  most models: four columns and the four that they are turned with, from the other half; behind the
//            rotated columns 8 neighbours
//   kPairs   8 neighbours, each turned with the one beside it
//   kAny     half the rotated width is no multiple of 4: 8 neighbours, partners from memory one by one
enum { kHalves = 0, kPairs = 1, kAny = 2 };
template <int MODE, int LPR> struct Turn {
    int half, ca, cb;                 // columns ca .. ca + 3 and cb .. cb + 3
    __device__ __forceinline__ Turn(int half_) : half(half_) {
        const int l = (threadIdx.x & 31) % LPR;
        const bool turned = MODE == kHalves && 4 * l < half;
        ca = turned ? 4 * l : 8 * l;
        cb = turned ? 4 * l + half : 8 * l + 4;
    }
    __device__ __forceinline__ int column(int e) const { return e < 4 ? ca + e : cb + e - 4; }
    __device__ __forceinline__ bool rotated(int e) const { return MODE == kHalves ? ca < half : column(e) < 2 * half; }
    __device__ __forceinline__ int partner(int e) const {     // of a rotated column
        const int c = column(e);
        return MODE == kPairs ? c ^ 1 : c < half ? c + half : c - half;
    }
    // The factors of a token's heads of one kind, v' = v x own + u x other with u the partners' values: its angles,
    // `sign` -1 to turn back, times the weights that the columns and their partners have (`w` null: none).
    __device__ __forceinline__ void factors(const float2 *turns, float sign, const float *w, float offset, f32x2 (&own)[4], f32x2 (&other)[4]) const {
        f32x2 x[4], y[4];
        if (w) {
            Raw<float> r;
            r.load(w + ca, w + cb);
            r.get(x);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = add2(x[j], both(offset));
        }
        if (MODE == kHalves) {
            const bool turned = ca < half;
            const float4 *t = reinterpret_cast<const float4 *>(turns + (turned ? ca : 0));      // two pairs each
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 p = turned ? t[j] : make_float4(1.f, 0.f, 1.f, 0.f);
                own[j] = own[j + 2] = pack2(p.x, p.z);
                other[j] = pack2(-sign * p.y, -sign * p.w);
                other[j + 2] = pack2(sign * p.y, sign * p.w);
                y[j] = x[j + 2];
                y[j + 2] = x[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float c[2], s[2], p[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = 2 * j + k;
                    const bool low = MODE == kPairs ? k == 0 : column(e) < half;
                    const float2 t = rotated(e) ? turns[MODE == kPairs ? column(e) >> 1 : low ? column(e) : column(e) - half] : make_float2(1.f, 0.f);
                    c[k] = t.x;
                    s[k] = low ? -sign * t.y : sign * t.y;
                    p[k] = w && rotated(e) ? w[partner(e)] + offset : 0.f;
                }
                own[j] = pack2(c[0], c[1]);
                other[j] = pack2(s[0], s[1]);
                y[j] = pack2(p[0], p[1]);
            }
        }
        if (!w) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            own[j] = mul2(own[j], x[j]);
            other[j] = mul2(other[j], y[j]);
        }
    }
    // v turned.  What is not rotated stays as it is, whatever stands beside it.  `p`: the head in memory (null: none), for kAny.
    template <typename T> __device__ __forceinline__ void turn(f32x2 (&v)[4], const f32x2 (&own)[4], const f32x2 (&other)[4], const T *p) const {
        f32x2 r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = mul2(v[j], own[j]);
            if (MODE == kHalves) {
                if (ca < half) r[j] = fma2(v[j ^ 2], other[j], r[j]);
            } else if (MODE == kPairs) {
                const float2 x = unpack2(v[j]);
                if (rotated(2 * j)) r[j] = fma2(pack2(x.y, x.x), other[j], r[j]);
            } else if (p) {
                float2 x = unpack2(r[j]);
                const float2 o = unpack2(other[j]);
                if (rotated(2 * j)) x.x = fmaf(to_f32(p[partner(2 * j)]), o.x, x.x);
                if (rotated(2 * j + 1)) x.y = fmaf(to_f32(p[partner(2 * j + 1)]), o.y, x.y);
                r[j] = pack2(x.x, x.y);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = r[j];
    }
};

// What a warp keeps of its next kPrepTokens tokens, `step` apart: lane i the i-th one's kind and place, shared memory their
// cosines and sines [token][half].
constexpr int kPrepTokens = 4;
__device__ __forceinline__ PrepToken prep_tokens(const AttnPrepArgs &a, long long t, long long step, bool pools, float2 *turns) {
    const int lane = threadIdx.x & 31;
    PrepToken mine{kBehind, 0.f, -1};
    if (lane < kPrepTokens) mine = prep_token(a, t + lane * step, pools);
    __syncwarp();                     // the angles before have been read
    for (int k = 0; k < kPrepTokens; ++k) {
        const float pos = __shfl_sync(0xffffffffu, mine.pos, k);
        if (__shfl_sync(0xffffffffu, mine.kind, k) == kLive)
            for (int i = lane; i < a.half; i += 32) turns[k * a.half + i] = cos_sin(pos, a.inv_freq[i]);
    }
    __syncwarp();
    return mine;
}

// A lane's share of a token's heads of one kind, `by` apart: its own, those that every lane of the warp has, and those that
// any lane has.
struct Share {
    int mine, full, any;
    __device__ __forceinline__ Share(int heads, int first, int hpw, int by, int sub)
        : mine(max(0, (heads - first - sub + by - 1) / by)), full(max(0, (heads - first - hpw + by) / by)), any(max(0, (heads - first + by - 1) / by)) {}
};

// What a lane has asked for lies in shared memory, a batch of UN heads a stage: each lane copies and reads its own pieces.
template <typename T, int UN> struct Stage {
    uint4 v[UN][sizeof(T) / 2][32];
    __device__ __forceinline__ void ask(int j, int lane, const T *p, const T *q) {
        if (sizeof(T) == 2) {
            const uint32_t to = smem_addr(&v[j][0][lane]);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" :: "r"(to), "l"(p) : "memory");
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" :: "r"(to + 8), "l"(q) : "memory");
        } else {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_addr(&v[j][0][lane])), "l"(p) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_addr(&v[j][sizeof(T) / 2 - 1][lane])), "l"(q) : "memory");
        }
    }
    __device__ __forceinline__ Raw<T> get(int j, int lane) const {
        Raw<T> r;
        if constexpr (sizeof(T) == 2) r = *reinterpret_cast<const Raw<T> *>(&v[j][0][lane]);
        else r.load(reinterpret_cast<const T *>(&v[j][0][lane]), reinterpret_cast<const T *>(&v[j][1][lane]));
        return r;
    }
    static __device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
};

// PLAIN: heads stand one after another in q, k and v, and a warp has all of a token's: the distances from one to the next
// are constants of the code.  (Address arithmetic was half of the instructions, and the kernels issue half of the time.)
constexpr int kStages = 5, kBatch = 2;       // stages: one that is worked on, four under way
template <typename T, int D, int MODE, bool PLAIN>
__global__ void __launch_bounds__(kPrepThreads, kPrepBlocks) attn_prep_kernel(const AttnPrepArgs a) {
    constexpr int LPR = D / 8, HPW = 32 / LPR, UN = kBatch;
    extern __shared__ float4 smem4[];                       // stages [warps][kStages], cosines and sines [warps][kPrepTokens][half]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR;
    Stage<T, UN> *stages = reinterpret_cast<Stage<T, UN> *>(smem4) + warp * kStages;
    float2 *turns = reinterpret_cast<float2 *>(reinterpret_cast<Stage<T, UN> *>(smem4) + kPrepWarps * kStages) + warp * kPrepTokens * a.half;
    const long long tokens = (long long)gridDim.x * kPrepWarps;      // side by side
    long long t = (long long)blockIdx.x * kPrepWarps + warp;
    await_previous();
    let_next_start();
    if (blockIdx.x == 0 && blockIdx.y == 0) check_bounds(a);
    if (t >= a.T) return;
    const bool pools = a.k_pages != nullptr;
    const Turn<MODE, LPR> rot(a.half);
    const int ca = rot.ca, cb = rot.cb, by = PLAIN ? HPW : HPW * gridDim.y, first = PLAIN ? 0 : (int)blockIdx.y * HPW;
    const Share nq(a.d.hq, first, HPW, by, sub), nk(a.k ? a.d.hkv : 0, first, HPW, by, sub), nv(pools ? a.d.hkv : 0, first, HPW, by, sub);
    const long long sq = PLAIN ? HPW * D : by * a.hs_q, sk = PLAIN ? HPW * D : by * a.hs_k, sv = PLAIN ? HPW * D : by * a.hs_v;
    const T *qp = (const T *)a.q + t * a.ld_q + (first + sub) * (PLAIN ? D : a.hs_q);
    const T *kp = (const T *)a.k + t * a.ld_k + (first + sub) * (PLAIN ? D : a.hs_k);
    const T *vp = (const T *)a.v + t * a.ld_v + (first + sub) * (PLAIN ? D : a.hs_v);
    // the next batch to ask for: of token t_ask, of q, k or v (kind_ask), heads from p_ask on
    long long t_ask = t;
    const T *p_ask = qp, *q_ask = qp, *k_ask = kp, *v_ask = vp;
    int kind_ask = 0, left_ask = nq.any, mine_ask = nq.mine, in_stage = 0, out_stage = 0;
    auto ask = [&]() {
        if (t_ask < a.T) {
            const long long step = PLAIN || kind_ask == 0 ? sq : kind_ask == 1 ? sk : sv;
#pragma unroll
            for (int j = 0; j < UN; ++j)
                if (j < mine_ask) stages[in_stage].ask(j, lane, p_ask + j * step + ca, p_ask + j * step + cb);
            p_ask += UN * step;
            left_ask -= UN;
            mine_ask -= UN;
            if (left_ask <= 0) {
                if (kind_ask == 0 && nk.any) {
                    kind_ask = 1;
                    p_ask = k_ask;
                    left_ask = nk.any;
                    mine_ask = nk.mine;
                } else if (kind_ask == 1 && nv.any) {
                    kind_ask = 2;
                    p_ask = v_ask;
                    left_ask = nv.any;
                    mine_ask = nv.mine;
                } else {
                    t_ask += tokens;
                    q_ask += tokens * a.ld_q;
                    k_ask += tokens * a.ld_k;
                    v_ask += tokens * a.ld_v;
                    kind_ask = 0;
                    p_ask = q_ask;
                    left_ask = nq.any;
                    mine_ask = nq.mine;
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        in_stage = (in_stage + 1) % kStages;
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) ask();            // whatever the tokens turn out to be
    f32x2 own[4], other[4];
    // The heads of one kind of a token, a batch of UN at a time, while the next ones are under way.
    auto run = [&](auto kind_of, const Share &n, const T *p, long long step, int state, T *out, T *cache) {
        constexpr int kind = decltype(kind_of)::value;
        const float *w = kind == 0 ? a.w_q : kind == 1 ? a.w_k : nullptr;
        const int cache_step = kind == 0 ? 0 : by * a.d.page * D;
        for (int i = 0; i < n.any; i += UN) {
            asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 2) : "memory");
            Raw<T> held[UN];
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                held[j].clear();
                if (i + j < n.mine) held[j] = stages[out_stage].get(j, lane);
            }
            out_stage = (out_stage + 1) % kStages;
            ask();                                          // into the stage that was read before this one
            auto work = [&](int j, bool in) {
                f32x2 x[4];
                held[j].get(x);
                float rstd = 1.f;
                if (w) rstd = rsqrtf(fmaf(head_sum<LPR>(dot8(x, x)), 1.f / D, a.eps));
                rot.turn(x, own, other, in ? p + j * step : nullptr);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], both(rstd));
                if (in) {
                    if (kind == 0 || out) store8(out + j * by * D + ca, out + j * by * D + cb, x);
                    if (kind == 1 && cache) store8(cache + j * cache_step + ca, cache + j * cache_step + cb, x);
                }
            };
            if (kind == 2 || state != kLive) {
                // values as they are; zeros for a padding token, nothing for one behind the last sequence
#pragma unroll
                for (int j = 0; j < UN; ++j) {
                    Raw<T> raw = held[j];
                    if (i + j >= n.mine) continue;
                    if (kind == 2 && cache) raw.store(cache + j * cache_step + ca, cache + j * cache_step + cb);
                    raw.clear();
                    if (kind < 2 && out && state == kPadding) raw.store(out + j * by * D + ca, out + j * by * D + cb);
                }
            } else if (i + UN <= n.full) {
#pragma unroll
                for (int j = 0; j < UN; ++j) work(j, true);
            } else {
#pragma unroll
                for (int j = 0; j < UN; ++j) work(j, i + j < n.mine);
            }
            p += UN * step;
            if (kind < 2 && out) out += UN * by * D;
            if (kind > 0 && cache) cache += UN * cache_step;
        }
    };
    PrepToken mine;
    for (int k = 0; t < a.T; t += tokens, k = (k + 1) % kPrepTokens) {
        if (k == 0) mine = prep_tokens(a, t, tokens, pools, turns);
        const int state = __shfl_sync(0xffffffffu, mine.kind, k);
        const float2 *angles = turns + k * a.half;
        T *k_out = a.k_out ? (T *)a.k_out + (t * a.d.hkv + first + sub) * D : nullptr, *k_cache = nullptr, *v_cache = nullptr;
        if (pools) {
            long long place = __shfl_sync(0xffffffffu, mine.place, k);
            if (place >= 0) {
                place = (place + (long long)(first + sub) * a.d.page) * D;
                k_cache = (T *)a.k_pages + place;
                v_cache = (T *)a.v_pages + place;
            }
        }
        if (state == kLive) rot.factors(angles, 1.f, a.w_q, a.offset, own, other);
        run(std::integral_constant<int, 0>(), nq, qp, sq, state, (T *)a.q_out + (t * a.d.hq + first + sub) * D, nullptr);
        if (nk.any) {
            if (state == kLive) rot.factors(angles, 1.f, a.w_k, a.offset, own, other);
            run(std::integral_constant<int, 1>(), nk, kp, sk, state, k_out, k_cache);
            if (nv.any) run(std::integral_constant<int, 2>(), nv, vp, sv, state, nullptr, v_cache);
        }
        qp += tokens * a.ld_q;
        kp += tokens * a.ld_k;
        vp += tokens * a.ld_v;
    }
}

// The weights' gradients gather in registers over a token's heads of one kind, then in shared memory over the tokens, each
// lane for itself, and at the end over the block in a fixed order.
template <typename T, int D, int MODE, bool PLAIN>
__global__ void __launch_bounds__(kPrepThreads, 2) attn_prep_backward_kernel(const AttnPrepArgs a) {
    constexpr int LPR = D / 8, HPW = 32 / LPR, UN = sizeof(T) == 2 ? 4 : 2;
    extern __shared__ float4 smem4[];                       // sums[2][warps][lanes][8], cosines and sines [warps][kPrepTokens][half]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / LPR;
    constexpr int kKind = kPrepWarps * 32 * 8;
    float *all = reinterpret_cast<float *>(smem4), *sums = all + (warp * 32 + lane) * 8;
    float2 *turns = reinterpret_cast<float2 *>(all + 2 * kKind) + warp * kPrepTokens * a.half;
    await_previous();
    let_next_start();
    if (blockIdx.x == 0) check_bounds(a);
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[e] = sums[kKind + e] = 0.f;
    const Turn<MODE, LPR> rot(a.half);
    const int ca = rot.ca, cb = rot.cb;
    const Share nq(a.d.hq, 0, HPW, HPW, sub), nk(a.k ? a.d.hkv : 0, 0, HPW, HPW, sub);
    const long long sq = PLAIN ? HPW * D : HPW * a.hs_q, sk = PLAIN ? HPW * D : HPW * a.hs_k;
    const long long tokens = (long long)gridDim.x * kPrepWarps;      // side by side
    long long t = (long long)blockIdx.x * kPrepWarps + warp;
    if (t < a.T) {
        const T *qp = (const T *)a.q + t * a.ld_q + sub * (PLAIN ? D : a.hs_q);
        const T *kp = (const T *)a.k + t * a.ld_k + sub * (PLAIN ? D : a.hs_k);
        const T *gqp = (const T *)a.dq_out + (t * a.d.hq + sub) * D, *gkp = (const T *)a.dk_out + (t * a.d.hkv + sub) * D;
        Raw<T> held_x[UN], held_g[UN];
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            held_x[j].clear();
            held_g[j].clear();
            if (j < nq.mine) {
                held_g[j].load(gqp + j * HPW * D + ca, gqp + j * HPW * D + cb);
                held_x[j].load(qp + j * sq + ca, qp + j * sq + cb);
            }
        }
        f32x2 own[4], other[4];
        // The heads of one kind of a token, a batch of UN loads ahead: of its next ones or, at the end, of those at `then`.
        auto run = [&](auto kind_of, const Share &n, const T *p, long long step, const T *grad, const T *then, long long then_step,
                       const T *then_grad, int then_mine, int state, T *to, long long to_step) {
            constexpr int kind = decltype(kind_of)::value;
            const float *w = kind == 0 ? a.w_q : a.w_k;
            f32x2 acc[4] = {}, wv[4] = {};
            if (w) {
                Raw<float> r;
                r.load(w + ca, w + cb);
                r.get(wv);
#pragma unroll
                for (int e = 0; e < 4; ++e) wv[e] = add2(wv[e], both(a.offset));
            }
            for (int i = 0; i < n.any; i += UN) {
                const bool more = i + UN < n.any;
                const T *next = more ? p + UN * step : then, *next_grad = more ? grad + UN * HPW * D : then_grad;
                const long long next_step = PLAIN ? step : more ? step : then_step;
                const int next_mine = more ? n.mine - i - UN : then_mine;
                auto refill = [&](int j) {
                    if (j < next_mine) {
                        held_g[j].load(next_grad + j * HPW * D + ca, next_grad + j * HPW * D + cb);
                        held_x[j].load(next + j * next_step + ca, next + j * next_step + cb);
                    }
                };
                auto work = [&](int j, bool in) {
                    f32x2 g[4], x[4];
                    held_g[j].get(g);
                    held_x[j].get(x);
                    refill(j);
                    rot.turn(g, own, other, in ? grad + j * HPW * D : nullptr);
                    if (w) {
                        const float mean_sq = head_sum<LPR>(dot8(x, x)) * (1.f / D);
                        const f32x2 rstd = both(rsqrtf(mean_sq + a.eps));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] = mul2(x[e], rstd);
                            if (in) acc[e] = fma2(g[e], x[e], acc[e]);
                            g[e] = mul2(g[e], wv[e]);
                        }
                        const f32x2 mean = both(head_sum<LPR>(dot8(g, x)) * (-1.f / D));
#pragma unroll
                        for (int e = 0; e < 4; ++e) g[e] = mul2(fma2(x[e], mean, g[e]), rstd);
                    }
                    if (MODE == kAny) __syncwarp();     // the partners' gradients have been read: dq may be dq_out
                    if (in && to) store8(to + j * to_step + ca, to + j * to_step + cb, g);
                };
                if (state != kLive) {
                    const f32x2 zero[4] = {};
#pragma unroll
                    for (int j = 0; j < UN; ++j) {
                        refill(j);
                        if (i + j < n.mine && to && state == kPadding) store8(to + j * to_step + ca, to + j * to_step + cb, zero);
                    }
                } else if (i + UN <= n.full) {
#pragma unroll
                    for (int j = 0; j < UN; ++j) work(j, true);
                } else {
#pragma unroll
                    for (int j = 0; j < UN; ++j) work(j, i + j < n.mine);
                }
                p = next;
                grad = next_grad;
                if (to) to += UN * to_step;
            }
            if (w) {
                float *sum = sums + kind * kKind;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = unpack2(acc[e]);
                    sum[2 * e] += v.x;
                    sum[2 * e + 1] += v.y;
                }
            }
        };
        PrepToken mine;
        for (int k = 0; t < a.T; t += tokens, k = (k + 1) % kPrepTokens) {
            if (k == 0) mine = prep_tokens(a, t, tokens, false, turns);
            const int state = __shfl_sync(0xffffffffu, mine.kind, k);
            const T *next_q = qp + tokens * a.ld_q, *next_g = gqp + tokens * a.d.hq * D;
            const int next_mine = t + tokens < a.T ? nq.mine : 0;
            if (state == kLive) rot.factors(turns + k * a.half, -1.f, nullptr, 0.f, own, other);
            run(std::integral_constant<int, 0>(), nq, qp, sq, gqp, nk.any ? kp : next_q, nk.any ? sk : sq, nk.any ? gkp : next_g,
                nk.any ? nk.mine : next_mine, state, a.dq ? (T *)a.dq + t * a.ld_dq + sub * a.hs_dq : nullptr, HPW * a.hs_dq);
            if (nk.any)
                run(std::integral_constant<int, 1>(), nk, kp, sk, gkp, next_q, sq, next_g, next_mine, state,
                    a.dk ? (T *)a.dk + t * a.ld_dk + sub * a.hs_dk : nullptr, HPW * a.hs_dk);
            qp = next_q;
            gqp = next_g;
            kp += tokens * a.ld_k;
            gkp += tokens * a.d.hkv * D;
        }
    }
    if (!a.ws) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kPrepThreads) {
        const int kind = i / D, c = i - kind * D;
        // the lane and value that hold column c
        const int at = MODE != kHalves || c >= 2 * a.half ? c : c < a.half ? (c >> 2) * 8 + (c & 3) : ((c - a.half) >> 2) * 8 + 4 + (c & 3);
        float s = 0.f;
        for (int w = 0; w < kPrepWarps * HPW; ++w) s += all[kind * kKind + ((w / HPW) * 32 + (w % HPW) * LPR) * 8 + at];
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

// Blocks of a call: as many as run at once, each warp over several tokens.
int prep_blocks(long long T, int per_sm) {
    const long long most = (long long)sm_count() * per_sm, all = (T + kPrepWarps - 1) / kPrepWarps;
    return (int)(all < 1 ? 1 : all < most ? all : most);
}
int backward_blocks(long long T) { return prep_blocks(T, 2); }

template <typename K> cudaError_t with_smem(K kernel, int bytes) {
    return bytes <= 48 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int D, int MODE> cudaError_t run_prep(const AttnPrepArgs &a, cudaStream_t s) {
    const int hpw = 256 / D, smem = kPrepWarps * (kStages * (int)sizeof(Stage<T, kBatch>) + kPrepTokens * a.half * 8), blocks = prep_blocks(a.T, kPrepBlocks);
    // a token's heads over several warps where there are few tokens
    const long long most = (a.d.hq + hpw - 1) / hpw, want = (long long)sm_count() * 24 / a.T;
    const unsigned split = (unsigned)(want < 1 ? 1 : want < most ? want : most);
    const bool plain = MODE != kAny && split == 1 && a.hs_q == D && (!a.k || a.hs_k == D) && (!a.k_pages || a.hs_v == D);
    const auto kernel = plain ? attn_prep_kernel<T, D, MODE, MODE != kAny> : attn_prep_kernel<T, D, MODE, false>;
    const cudaError_t e = with_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    return launch_early(kernel, dim3((unsigned)blocks, split), kPrepThreads, smem, s, a);
}
template <typename T, int D, int MODE> cudaError_t run_backward(const AttnPrepArgs &a, cudaStream_t s) {
    const int blocks = backward_blocks(a.T), smem = 2 * kPrepThreads * 8 * 4 + kPrepWarps * kPrepTokens * a.half * 8;
    const bool plain = MODE != kAny && a.hs_q == D && (!a.k || a.hs_k == D);
    const auto kernel = plain ? attn_prep_backward_kernel<T, D, MODE, MODE != kAny> : attn_prep_backward_kernel<T, D, MODE, false>;
    cudaError_t e = with_smem(kernel, smem);
    if (e != cudaSuccess) return e;
    e = launch_early(kernel, dim3(blocks), kPrepThreads, smem, s, a);
    if (e != cudaSuccess || !a.ws) return e;
    return launch_early(attn_prep_weights_kernel, dim3((2 * D + 7) / 8), 256, 0, s, a, blocks);
}

int mode_of(const AttnPrepArgs &a) { return a.interleaved ? kPairs : a.half % 4 == 0 ? kHalves : kAny; }

#define GDN_PREP_MODES(RUN, T, D)                                                                    \
    return mode_of(a) == kHalves ? RUN<T, D, kHalves>(a, s) : mode_of(a) == kPairs ? RUN<T, D, kPairs>(a, s) : RUN<T, D, kAny>(a, s)
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
