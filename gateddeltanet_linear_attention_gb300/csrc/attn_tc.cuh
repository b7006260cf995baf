// attn_tc.cuh -- what the two tensor-core kernels of the decode attention share: the tiles' way into shared memory, and how a
// unit's tiles are described to the warps that compute.
#pragma once

#include <cuda.h>

#include "attn_common.cuh"
#include "tc_sm103.cuh"

namespace gdn {
namespace attn_tc {

constexpr int kTile = 64;                          // tokens
constexpr int kMaxEntries = 24;                    // of the ring of K and V tiles

// A unit's tiles in this CTA, as the copying warp describes them.
struct Unit {
    int n, h, len, first, i0, count, seq0, slot;   // slot -1: the unit is whole
    bool more;                                     // the CTA has another one
};

struct Maps {
    CUtensorMap k, v, q;                           // q: where the kernel takes query rows by TMA
};

// The maps on their way before the first copy asks for them.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) { asm volatile("prefetch.tensormap [%0];" :: "l"(m) : "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// Either half's exponent all ones.
__device__ __forceinline__ bool not_finite2(uint32_t v) {
    return (v & 0x7f80u) == 0x7f80u || (v & 0x7f800000u) == 0x7f800000u;
}
// Whether all threads of the barrier say so.
__device__ __forceinline__ bool bar_all(int id, int threads, bool mine) {
    int all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}\n"
                 : "=r"(all) : "r"(id), "r"(threads), "r"((int)mine) : "memory");
    return all != 0;
}

// The two copying warps: K (kv 0) and V of the CTA's tiles into a ring of `ring` entries each, as D / 64 blocks of 64 tokens by
// 128 bytes in the 128-byte swizzle.  A warp each: V's entries are needed longer, and K's that are free would wait behind them.
// The first also writes the units into `units` and fetches their query rows (q_bytes of them) by load_q(slot, sequence, key
// head, barrier).  Of the ring: entries, full, empty (barriers), pieces_of (which 16-token pieces of an entry's tile are there;
// what is not there is not copied: the entry holds what it held).  Of the units: ufull, uempty [kUnits].
template <int D, int kUnits, typename LoadQ>
__device__ __forceinline__ void copy_tiles(const AttnDecodeArgs &a, const AttnWalk &w, const Maps &maps, uint32_t kv, uint32_t ring, uint32_t entries, uint32_t full,
                                           uint32_t empty, uint32_t ufull, uint32_t uempty, int *pieces_of, Unit *units, uint32_t q_bytes,
                                           LoadQ load_q) {
    const int lane = threadIdx.x & 31;
    constexpr int NB = D / 64;
    const int piece = min(a.d.page, kTile), shift = min(a.d.page_shift, 6), boxes = (kTile >> shift) * NB;
    const int my_piece = lane / NB, my_col = lane % NB;
    const uint32_t box_bytes = piece * 128u, at = my_col * (kTile * 128u) + my_piece * box_bytes;
    const CUtensorMap *map = kv ? &maps.v : &maps.k;
    uint32_t e = 0, phase = 0, issued = 0;
    int seq = 0, u = 0;
    bool alive = true;
    // the page of this lane's piece of tile t of a sequence; -1: not there
    auto page_of = [&](const AttnSeq &s, int t) {
        const int i = (s.tile0 + t) * kTile + (my_piece << shift);
        if (lane >= boxes || i >= s.len || i + piece <= s.first) return -1;
        const int p = a.table[(long long)s.row * a.d.max_pages + (i >> a.d.page_shift)];
        if (p >= 0 && p < a.d.n_pages) return p;
        set_error(a.err, GDN_DEVERR_PAGE);
        return -1;
    };
    AttnSeq s = w.s;
    int n = w.n, h = w.h, t0 = w.t, page = page_of(s, t0);
    long long left = w.left - w.lead;
    for (bool more = true; more && alive; ++u) {
        const int count = (int)min((long long)(s.tiles - t0), left);
        const bool unit_end = t0 + count == s.tiles;
        left -= count + a.lead;
        more = unit_end && left > 0;                        // (what remains has tiles of the next unit)
        const int slot = t0 == 0 && unit_end ? -1 : u == 0 ? 0 : 1;
        if (kv == 0) {
            const uint32_t us = u % kUnits, uphase = (u / kUnits) & 1;
            if (u >= kUnits) alive = tc::mbar_wait(uempty + 8 * us, uphase ^ 1, a.wait_ns);
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) break;
            if (lane == 0) {
                units[us] = Unit{n, h, s.len, s.first, (s.tile0 + t0) * kTile, count, seq, slot, more};
                tc::mbar_arrive_expect_tx(ufull + 8 * us, q_bytes);
            }
            __syncwarp();
            load_q(us, n, h, ufull + 8 * us);
        }
        // the unit behind this one, and where its first tile lies: known before this one's last tile is asked for
        AttnSeq next_s = s;
        int next_n = n, next_h = h + 1, next_page = -1;
        for (int j = 0; j < count && alive; ++j) {
            const int here = page, i0 = (s.tile0 + t0 + j) * kTile;
            if (j + 1 < count) page = page_of(s, t0 + j + 1);
            const unsigned there = __ballot_sync(0xffffffffu, here >= 0);
            const uint32_t bytes = __popc(there) * box_bytes;
            // the row of the pools where this lane's piece begins
            const int y = (here * a.d.hkv + h) * a.d.page + ((i0 + (my_piece << shift)) & (a.d.page - 1));
            if (issued >= ring) alive = tc::mbar_wait(empty + 8 * e, phase ^ 1, a.wait_ns);
            alive = __all_sync(0xffffffffu, alive);
            if (!alive) break;
            if (lane == 0) {
                int bits = 0;
                for (int p = 0; p < 4; ++p) bits |= (there >> ((p * 16) >> shift) * NB & 1u) << p;
                pieces_of[e] = bits;
                if (bytes) tc::mbar_arrive_expect_tx(full + 8 * e, bytes);
                else tc::mbar_arrive(full + 8 * e);
            }
            __syncwarp();
            const bool drop = (a.lose & LOSE_ATTN_TILE_COPY) && kv == 0 && issued == 0 && lane == 0;
            if (here >= 0 && !drop) tc::tma_load_2d(entries + e * (kTile * D * 2) + at, map, my_col * 64, y, full + 8 * e);
            ++issued;
            if (++e == ring) {
                e = 0;
                phase ^= 1;
            }
            if (j == 0 && more) {
                if (next_h == a.d.hkv) {
                    next_h = 0;
                    next_s = attn_seq<kTile>(a, ++next_n);
                }
                next_page = page_of(next_s, 0);
            }
        }
        seq += count;
        if (!more && kv == 0 && lane == 0) {
            // the CTA that holds a unit's front joins it: the CTAs behind that hold the rest
            int parts = 0;
            if (!unit_end && t0 == 0) parts = 1 + (int)((s.tiles - count + w.per - 1) / w.per);
            a.joins[blockIdx.x] = make_int4(n, h, u == 0 ? 0 : 1, parts);
        }
        s = next_s;
        n = next_n;
        h = next_h;
        t0 = 0;
        page = next_page;
    }
    if (lane == 0) {
        if (!alive) {             // nothing more is copied
            set_error(a.err, GDN_DEVERR_TIMEOUT);
            if (kv == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        }
        // what is under way arrives before the block ends
        for (uint32_t k = 0; k < min(issued, ring); ++k) {
            const uint32_t last = issued - 1 - k;
            tc::mbar_wait(full + 8 * (last % ring), (last / ring) & 1, a.wait_ns);
        }
        for (int k = 0; kv == 0 && k < min(u, kUnits); ++k) {
            const int last = u - 1 - k;
            tc::mbar_wait(ufull + 8 * (last % kUnits), (last / kUnits) & 1, a.wait_ns);
        }
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// A pool as rows of D columns (one token of one key head each), in boxes of a piece of a page by 64 columns.
inline bool encode_pool(CUtensorMap *m, const void *pool, const AttnDims &d) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d.D, (cuuint64_t)d.n_pages * d.hkv * d.page}, strides[1] = {(cuuint64_t)d.D * 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)(d.page < kTile ? d.page : kTile)}, estr[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Query rows in boxes of `rows` of one sequence and key head by 64 columns: columns, heads, tokens.
inline bool encode_queries(CUtensorMap *m, const AttnDecodeArgs &a) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.d.D, (cuuint64_t)a.d.hq, (cuuint64_t)a.n_seqs * a.tokens};
    // (the distance of a single token to the next may be anything)
    const cuuint64_t strides[2] = {(cuuint64_t)a.hs_q * 2, dims[2] > 1 ? (cuuint64_t)a.ld_q * 2 : dims[0] * dims[1] * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)a.d.grp, (cuuint32_t)a.tokens}, estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn_tc
}  // namespace gdn
