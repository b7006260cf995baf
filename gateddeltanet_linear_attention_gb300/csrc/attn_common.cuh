// attn_common.cuh -- arguments and device helpers of the attention layers' kernels
// (gdn_attn_* and gdn_page_* in gdn.h).
#pragma once

#include "ssm_common.cuh"

namespace gdn {

struct AttnDims {
    int hq, hkv, grp, D;              // grp = hq / hkv
    int page, page_shift;             // page = 1 << page_shift
    int n_pages, n_rows, max_pages;
};
constexpr int kAttnMaxTokens = 8;     // new tokens of a sequence in one gdn_attn_decode
constexpr int kAttnMaxGroup = 16;
constexpr int kMaxPosition = 1 << 24; // positions below it are exact in 32-bit floats

struct AttnPrepArgs {
    const void *q, *k, *v;            // k may be null; v only with pools
    long long ld_q, hs_q, ld_k, hs_k, ld_v, hs_v, T;
    const float *w_q, *w_k, *inv_freq;
    float offset, eps;
    int half;                         // rotary_dim / 2
    bool interleaved;
    const int32_t *positions, *cu, *rows, *lens, *table;
    int n_seqs;
    void *k_pages, *v_pages, *q_out, *k_out;
    // backward
    const void *dq_out, *dk_out;
    void *dq, *dk;
    long long ld_dq, hs_dq, ld_dk, hs_dk;
    float *dw_q, *dw_k, *ws;
    AttnDims d;
    unsigned *err;
};

struct AttnDecodeArgs {
    const void *q, *k_pages, *v_pages;
    long long ld_q, hs_q;
    const int32_t *table, *lens, *rows;
    int n_seqs, tokens, window;
    float scale_log2;                 // scale * log2(e)
    void *out;
    float *lse;
    AttnDims d;
    unsigned *err;
    unsigned long long wait_ns;       // limit of bounded waits, and the copies that a test drops
    unsigned lose;
    // workspace: what CTA c leaves of a unit that it does not hold whole, in slot 0 where that unit is its
    // first one, else 1: rows x D sums, then rows x (m, l), m in powers of two; and the join kernel's for CTA c
    float *parts;                     // [ctas][2][attn_part_floats]
    int4 *joins;                      // [ctas]: sequence, key head, slot of the first part, parts
    int ctas, lead;                   // lead: see AttnWalk
};
// Most CTAs that share the work of a decode: the workspace is laid out for them.
constexpr int kAttnCtasPerSm = 2, kAttnMaxCtas = 512;

constexpr float kLn2 = 0.6931471805599453f;
__host__ __device__ inline long long attn_part_floats(int rows, int D) { return (long long)rows * D + ((2 * rows + 3) & ~3); }
__device__ __forceinline__ float *attn_part(const AttnDecodeArgs &a, int cta, int slot) {
    return a.parts + ((long long)cta * 2 + slot) * attn_part_floats(a.d.grp * a.tokens, a.d.D);
}

// Row of sequence n in the page table; -1 for a padding lane (or a row that is reported).
__device__ __forceinline__ int attn_row(const int32_t *rows, int n, const AttnDims &d, unsigned *err) {
    const int r = rows ? rows[n] : n;
    if (r >= d.n_rows) {
        set_error(err, GDN_DEVERR_SLOT);
        return -1;
    }
    return r < 0 ? -1 : r;
}

// A sequence as its attention sees it: table row (-1: nothing to see), length, first token in sight of any of its new
// ones, and the tiles that hold what is in sight (one of an empty sequence, so that its rows are written).
struct AttnSeq {
    int row, len, first, tile0, tiles;
};
template <int TILE> __device__ __forceinline__ AttnSeq attn_seq(const AttnDecodeArgs &a, int n) {
    AttnSeq s;
    s.row = attn_row(a.rows, n, a.d, a.err);
    s.len = s.row < 0 ? 0 : a.lens[s.row];
    if (s.len > a.d.max_pages * a.d.page) {       // the product fits in 32 bits: checked on the host
        set_error(a.err, GDN_DEVERR_PAGE);
        s.len = 0;
    }
    if (s.len < 0) s.len = 0;
    s.first = a.window > 0 ? max(0, s.len - a.tokens + 1 - a.window) : 0;
    s.tile0 = s.first / TILE;
    s.tiles = max(1, (s.len + TILE - 1) / TILE - s.tile0);
    return s;
}

// The batch as one line of tiles, sequence after sequence, in each its key heads after another, cut into
// equal shares: CTA c takes places [c * per, (c + 1) * per) whatever sequences they belong to, so that mixed
// lengths and single long ones keep every SM busy alike.  A unit is one key head of one sequence; in front of its
// tiles lie `lead` places without any, as many as its end costs in tiles, so that who gets many short ones is not late.
struct AttnWalk {
    long long per, left;              // places of a CTA; of this one still to do
    int lead;                         // of them in front of the first unit
    int n, h, t;                      // sequence, key head, tile in the unit
    AttnSeq s;
};
// Where CTA c begins (whole block; `sums`: 33 values of shared memory).  False: nothing to do.
template <int TILE, int THREADS>
__device__ __forceinline__ bool attn_begin(const AttnDecodeArgs &a, int c, long long *sums, int *found, AttnWalk &w) {
    constexpr int WARPS = THREADS / 32;
    static_assert(WARPS <= 32, "one warp scans the warps' sums");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (a.n_seqs + THREADS - 1) / THREADS, lo = min(tid * each, a.n_seqs), hi = min(lo + each, a.n_seqs);
    long long mine = 0;
    for (int n = lo; n < hi; ++n) mine += attn_seq<TILE>(a, n).tiles + a.lead;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        long long v = lane < WARPS ? sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        sums[lane] = v;
    }
    __syncthreads();
    const long long total = sums[WARPS - 1] * a.d.hkv;
    upto += warp > 0 ? sums[warp - 1] : 0;
    w.per = (total + a.ctas - 1) / a.ctas;
    const long long at = w.per * c;
    if (at >= total) return false;
    w.left = min(w.per, total - at);
    // the thread whose sequences hold the first tile finds which
    if (at < upto * a.d.hkv && at >= (upto - mine) * a.d.hkv) {
        long long base = (upto - mine) * a.d.hkv;
        for (int n = lo; n < hi; ++n) {
            const int places = attn_seq<TILE>(a, n).tiles + a.lead;
            if (at < base + (long long)places * a.d.hkv) {
                found[0] = n;
                found[1] = (int)((at - base) / places);
                found[2] = (int)((at - base) % places);
                break;
            }
            base += (long long)places * a.d.hkv;
        }
    }
    __syncthreads();
    w.n = found[0];
    w.h = found[1];
    w.lead = max(a.lead - found[2], 0);
    w.t = max(found[2] - a.lead, 0);
    w.s = attn_seq<TILE>(a, w.n);
    return w.left > w.lead;
}
// To the next tile, where units lead with none; true where a new unit begins.
template <int TILE> __device__ __forceinline__ bool attn_next(const AttnDecodeArgs &a, AttnWalk &w) {
    --w.left;
    if (++w.t < w.s.tiles) return false;
    w.t = 0;
    if (++w.h == a.d.hkv) {
        w.h = 0;
        if (++w.n < a.n_seqs && w.left > 0) w.s = attn_seq<TILE>(a, w.n);
    }
    return true;
}

struct PageArgs {
    int32_t *table, *lens, *refs;
    const int32_t *rows, *new_lens;   // resize; fork: destinations and sources
    int n;
    int32_t *granted, *src, *dst;
    int32_t *table_out, *refs_out;    // compact
    int32_t *ws;
    AttnDims d;
    unsigned *err;
};
size_t page_ws_ints(const AttnDims &d, long long lanes);
cudaError_t launch_page_resize(const PageArgs &a, cudaStream_t s);
cudaError_t launch_page_fork(const PageArgs &a, cudaStream_t s);
cudaError_t launch_page_compact(const PageArgs &a, cudaStream_t s);
cudaError_t launch_page_copy(const void *src_k, const void *src_v, int n_src, void *dst_k, void *dst_v, int n_dst,
                             const int32_t *src_idx, const int32_t *dst_idx, int n, long long page_bytes, unsigned *err,
                             cudaStream_t s);

cudaError_t launch_attn_prep(const AttnPrepArgs &a, bool act_bf16, cudaStream_t s);
size_t attn_prep_ws_floats(const AttnDims &d, long long T);
cudaError_t launch_attn_prep_backward(const AttnPrepArgs &a, bool act_bf16, cudaStream_t s);

// Bytes of the workspace for `rows` query rows of a unit; carve lays it out.
size_t attn_decode_ws_bytes(const AttnDims &d, int rows);
void attn_decode_carve(AttnDecodeArgs &a, void *ws);
cudaError_t launch_attn_decode(const AttnDecodeArgs &a, bool act_bf16, cudaStream_t s);
cudaError_t launch_attn_decode_tc(const AttnDecodeArgs &a, cudaStream_t s);
cudaError_t launch_attn_decode_rows(const AttnDecodeArgs &a, cudaStream_t s);
cudaError_t launch_attn_join(const AttnDecodeArgs &a, bool act_bf16, cudaStream_t s);
}  // namespace gdn
