// attn_decode_rows.cu -- attention of new tokens over a paged bf16 cache where a key head has many query rows (17 to 128:
// verification rounds, many query heads a key head), on tcgen05.
//
// The shares, parts and join of attn_decode.cu, tiles of 64 tokens copied as for the kernel of few rows.  With the query rows
// as the 128 rows of the products, both accumulators in TMEM:
//   S = Q K^T     rows x 64 tokens; K from shared memory as TMA left it
//   P = exp(S - m) a thread a row: maximum and sum need no other lane; P, in two bf16 parts, in the place of S
//   O += P V      P from TMEM, V from shared memory as TMA left it
// Two groups of four warps (one at 256 columns) take turns with the tiles, each with its own S, O, m and l; O of both lies in
// the same lanes, so the first group adds the second one's to its own where a unit ends.
//
// m is the maximum of a row's first tile and is raised only where a score passes it by 8 powers of two: P stays below 256,
// which changes no rounding, and O is seldom scaled again.
//
// HBM-bound by design; what stands in the way is the chain of a tile, about 2,000 cycles (scores, 64 exponentials a thread,
// products), two of which overlap.
#include "attn_tc.cuh"

namespace gdn {

namespace {

using namespace attn_tc;

constexpr float kSlack = 8.f;                      // powers of two that a score may pass m by

// NG groups; room for RB query rows (products read 128: behind them whatever follows, into lanes that nobody reads).
template <int D, int NG, int RB> struct Shape {
    static constexpr int threads = (5 * NG + 1) * 32;
    static constexpr int units = D == 256 && RB == 128 ? 1 : 2;
    static constexpr int entry = kTile * D * 2, q_block = RB * D * 2;
    static constexpr int fixed = units * q_block + NG * (128 * 8 + D * 4) + 1024;
    static constexpr int limit = 227 * 1024 - 1024;
    static constexpr int fit = (limit - fixed) / entry, turn = 2 * NG;
    // a multiple of the groups' entries: an entry then serves tiles of one group alone
    static constexpr int entries = fit < kMaxEntries ? fit / turn * turn : kMaxEntries;
    static constexpr int bytes = fixed + entries * entry;
    static constexpr uint32_t col_o = 128;         // TMEM: S and P of group g at 64 g, its O at 128 + g D
    static_assert(entries >= turn && entries % turn == 0, "a tile of each group in flight, in entries of its own");
    static_assert(128 + NG * D <= 512, "tensor memory");
    static_assert(q_block + entries * entry >= 128 * 128 * (D / 64), "products read 128 rows of the last block");
};

// One lane (`lead`) of a warp that stays together issues products, commits and arrivals.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t lead;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(lead));
    return lead;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
        :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead) : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t b) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
        :: "r"(b), "r"(lead) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory"); }
enum { kBarGroup = 1, kBarActive = 3 };            // of each group, of its warps that have rows

// 128-byte-swizzled operands, 64-column blocks `block` bytes apart.  K-major: the row index is M or N; MN-major: it is K.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) { return tc::smem_desc(saddr, 16, 1024) | (2ull << 61); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t block) { return tc::smem_desc(saddr, block, 1024) | (2ull << 61); }
// In 16-byte units of the start address: 16 columns on in a K-major operand, 16 rows on in an MN-major one.
__device__ __forceinline__ uint64_t step_k(int ks, uint32_t block) { return (uint64_t)((ks >> 2) * (block >> 4) + (ks & 3) * 2); }
__device__ __forceinline__ uint64_t step_mn(int ks) { return (uint64_t)(ks * 128); }

template <int D, int NG, int RB>
__global__ void __launch_bounds__((Shape<D, NG, RB>::threads), 1) attn_decode_rows_kernel(const AttnDecodeArgs a, const __grid_constant__ Maps maps) {
    using S = Shape<D, NG, RB>;
    constexpr int KS = D / 16, kUnits = S::units, kThreads = S::threads;
    constexpr uint32_t E = S::entries, kBlock = kTile * 128, kQBlock = RB * 128;
    extern __shared__ unsigned char raw[];
    __shared__ long long sums[33];
    __shared__ int found[3], spoiled[NG];
    __shared__ uint32_t tmem_base;
    __shared__ uint64_t bars[2 * kMaxEntries + 2 * kUnits + 4 * NG + 2];
    __shared__ int pieces_of[kMaxEntries];
    __shared__ Unit units[kUnits];
    unsigned char *base = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    // queries in front of the ring, so that what products read behind them is shared memory of this CTA
    unsigned char *q_mem = base, *ring = base + kUnits * S::q_block;
    float2 *stats = reinterpret_cast<float2 *>(ring + E * S::entry);               // [groups][128]: m and l
    unsigned *spoil = reinterpret_cast<unsigned *>(stats + NG * 128);              // [groups][D]: new tokens whose sum is not finite
    const uint32_t entries = tc::smem_u32(ring), full = tc::smem_u32(bars), empty = full + 8 * kMaxEntries,
                   ufull = empty + 8 * kMaxEntries, uempty = ufull + 8 * kUnits, s_full = uempty + 8 * kUnits, p_ready = s_full + 8 * NG,
                   pv_done = p_ready + 8 * NG, ended = pv_done + 8 * NG, merged = ended + 8 * NG, taken = merged + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rows = a.d.grp * a.tokens, active = (rows + 31) / 32;                // warps of a group that have rows
    if (tid == 0) {
        for (uint32_t e = 0; e < E; ++e) {
            tc::mbar_init(full + 8 * e, 1);
            tc::mbar_init(empty + 8 * e, 1);
        }
        for (int u = 0; u < kUnits; ++u) {
            tc::mbar_init(ufull + 8 * u, 1);
            tc::mbar_init(uempty + 8 * u, 5 * NG);
        }
        for (int g = 0; g < NG; ++g) {
            tc::mbar_init(s_full + 8 * g, 1);
            tc::mbar_init(p_ready + 8 * g, active);
            tc::mbar_init(pv_done + 8 * g, 1);
            tc::mbar_init(ended + 8 * g, 1);
            spoiled[g] = 0;
        }
        tc::mbar_init(merged, active);
        tc::mbar_init(taken, active);
        tc::mbar_fence_init();
    }
    for (int i = tid; i < NG * D; i += kThreads) spoil[i] = 0u;
    // rows that pad the query block stay zero
    for (int i = tid; i < kUnits * S::q_block / 16; i += kThreads) reinterpret_cast<uint4 *>(q_mem)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_async_smem();
    await_previous();
    let_next_start();
    AttnWalk w;
    const bool work = attn_begin<kTile, kThreads>(a, blockIdx.x, sums, found, w);      // synchronises the block
    if (!work) {
        if (tid == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    if (warp == 4 * NG) {
        tc::tmem_alloc(tc::smem_u32(&tmem_base), 512);
        tc::tmem_relinquish();
        tc::fence_before_sync();
    }
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *(volatile uint32_t *)&tmem_base;

    if (warp == 4 * NG) {
        // ------------------------------------------------------------ copies
        copy_tiles<D, E, kUnits>(a, w, maps, entries, full, empty, ufull, uempty, pieces_of, units, (uint32_t)rows * D * 2,
                                 [&](uint32_t us, int n, int h, uint32_t bar) {
            if (lane < D / 64)
                asm volatile(
                    "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                    :: "r"(tc::smem_u32(q_mem) + us * S::q_block + lane * kQBlock), "l"(&maps.q), "r"(lane * 64), "r"(h * a.d.grp),
                       "r"(n * a.tokens), "r"(bar) : "memory");
        });
    } else if (warp > 4 * NG) {
        // ---------------------------------------------------------- products
        constexpr uint32_t id_s = tc::idesc_bf16(128, kTile), id_pv = tc::idesc_bf16(128, D) | tc::kTransB;
        const int g = warp - 4 * NG - 1;
        const uint32_t lead = elect_lane(), t_s = tmem + g * 64, t_o = tmem + S::col_o + g * D;
        uint32_t e = 2 * g, phase = 0, k = 0;               // k: tiles of the group so far
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(b, parity, a.wait_ns)); };
        int u = 0;
        for (long long left = w.left; left > 0 && ok; ++u) {
            const uint32_t us = u % kUnits;
            wait(ufull + 8 * us, (u / kUnits) & 1);
            if (!ok) break;
            const int count = units[us].count, seq0 = units[us].seq0;
            left -= count;
            const uint64_t q_desc = desc_k(tc::smem_u32(q_mem) + us * S::q_block);
            uint32_t sum = 0;                               // whether O holds this unit's sums
            for (int j = (g - seq0) & (NG - 1); j < count && ok; j += NG) {
                wait(full + 8 * e, phase);
                if (k > 0) wait(pv_done + 8 * g, (k - 1) & 1);      // P of the tile before has been read
                if (!ok) break;
                tc::fence_after_sync();
                const uint64_t k_desc = desc_k(entries + e * S::entry);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) mma_ss(lead, t_s, q_desc + step_k(ks, kQBlock), k_desc + step_k(ks, kBlock), id_s, ks > 0);
                commit(lead, s_full + 8 * g);
                commit(lead, empty + 8 * e);
                wait(full + 8 * (e + 1), phase);
                wait(p_ready + 8 * g, k & 1);
                if (!ok) break;
                tc::fence_after_sync();
                const uint64_t v_desc = desc_mn(entries + (e + 1) * S::entry, kBlock);
#pragma unroll
                for (int ks = 0; ks < 2 * kTile / 16; ++ks) {       // the leading parts of P, then the rest
                    mma_ts(lead, t_o, t_s + ks * 8, v_desc + step_mn(ks & (kTile / 16 - 1)), id_pv, sum);
                    sum = 1;
                }
                commit(lead, pv_done + 8 * g);
                commit(lead, empty + 8 * (e + 1));
                ++k;
                e += 2 * NG;
                if (e >= E) {
                    e -= E;
                    phase ^= 1;
                }
            }
            if (ok) commit(lead, uempty + 8 * us);
        }
        if (!ok && lane == 0) set_error(a.err, GDN_DEVERR_TIMEOUT);
        // products under way end before tensor memory is given back
        commit(lead, ended + 8 * g);
        if (!tc::mbar_wait(ended + 8 * g, 0, a.wait_ns) && lane == 0) set_error(a.err, GDN_DEVERR_TIMEOUT);
    } else {
        // ------------------------------------------------------------ softmax
        const int g = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const bool on = quarter < active;                   // this warp has rows
        const int token = min(row / a.d.grp, a.tokens - 1);
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16, t_s = tmem + lanes + g * 64, t_o = tmem + lanes + S::col_o + g * D;
        unsigned *my_spoil = spoil + g * D;
        uint32_t e = 2 * g, phase = 0, k = 0;
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(b, parity, a.wait_ns)); };
        int u = 0;
        for (long long left = w.left; left > 0; ++u) {
            const uint32_t us = u % kUnits;
            // a group's warps give up together: they meet at its barrier
            if (!bar_all(kBarGroup + g, 128, ok && tc::mbar_wait(ufull + 8 * us, (u / kUnits) & 1, a.wait_ns))) {
                ok = false;
                break;
            }
            const Unit unit = units[us];
            left -= unit.count;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(uempty + 8 * us);
            const int first_j = (g - unit.seq0) & (NG - 1), tiles = unit.count > first_j ? (unit.count - first_j + NG - 1) / NG : 0;
            // the second group's O and statistics are the first one's until it has taken them
            bool mine = g == 0 || u == 0;
            auto take_back = [&]() {
                if (!mine) wait(taken, (u - 1) & 1);
                mine = true;
            };
            if (spoiled[g]) {
                take_back();
                for (int c = tid & 127; c < D; c += 128) my_spoil[c] = 0u;
                bar_sync(kBarGroup + g, 128);
                spoiled[g] = 0;
                bar_sync(kBarGroup + g, 128);
            }
            if (!on) continue;
            float m = -INFINITY, l = 0.f;
            // what all rows see lies below `open`, and not below `wide`
            const int open = unit.len - a.tokens + 1, wide = a.window > 0 ? unit.len - a.window : 0;
            const int end = open + token, begin = a.window > 0 ? end - a.window : 0;
            for (int j = first_j; j < unit.count; j += NG) {
                const int i0 = unit.i0 + j * kTile;
                wait(s_full + 8 * g, k & 1);
                // V's entry stays this tile's until its product is done; K's may be another tile's by now
                wait(full + 8 * (e + 1), phase);
                tc::fence_after_sync();
                const int pieces = pieces_of[e + 1];
                const bool masked = pieces != 15 || i0 + kTile > open || i0 < wide;
                float v[64];
                tc::tmem_ld64(t_s, v);
                if (masked) {
                    // tokens that this row sees
                    unsigned long long seen = 0;
                    for (int p = 0; p < 4; ++p)
                        if (pieces >> p & 1) seen |= 0xffffull << (p * 16);
                    const int lo = min(max(begin - i0, 0), 64), hi = min(max(end - i0, 0), 64);
                    seen &= hi < 64 ? (1ull << hi) - 1 : ~0ull;
                    seen &= lo < 64 ? ~0ull << lo : 0ull;
#pragma unroll
                    for (int i = 0; i < 64; ++i) v[i] = seen >> i & 1 ? v[i] : -INFINITY;
                }
                float top = v[0];
#pragma unroll
                for (int i = 1; i < 64; ++i) top = fmaxf(top, v[i]);
                top *= a.scale_log2;
                if (j == first_j) {
                    m = top;
                } else if (__any_sync(0xffffffffu, top > m + kSlack || (m == -INFINITY && top > m))) {
                    const float nm = top > m + kSlack || m == -INFINITY ? top : m;
                    const float back = nm == m ? 1.f : exp2_fast(m - nm);
                    m = nm;
                    l *= back;
                    wait(pv_done + 8 * g, (k - 1) & 1);     // the sums are whole
                    tc::fence_after_sync();
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        uint32_t x[8], y[8];
                        tc::tmem_ld16(t_o + c, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x[i] = __float_as_uint(o[i] * back);
                            y[i] = __float_as_uint(o[8 + i] * back);
                        }
                        tmem_st8(t_o + c, x);
                        tmem_st8(t_o + c + 8, y);
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float p0 = exp2_fast(fmaf(v[c * 16 + 2 * i], a.scale_log2, -ref)),
                                    p1 = exp2_fast(fmaf(v[c * 16 + 2 * i + 1], a.scale_log2, -ref));
                        part[i & 3] += p0 + p1;
                        hi[i] = pack_bf16(p0, p1);
                        lo[i] = pack_bf16(p0 - __uint_as_float(hi[i] << 16), p1 - __uint_as_float(hi[i] & 0xffff0000u));
                    }
                    tmem_st8(t_s + c * 8, hi);
                    tmem_st8(t_s + 32 + c * 8, lo);
                }
                l += (part[0] + part[1]) + (part[2] + part[3]);
                if (masked) {
                    // Places that no row sees may hold anything: they become zeros.  A value that is not finite in a place that
                    // only some new tokens see becomes zero too, and the sums of its column for those tokens are NaN, as sums
                    // with it are not finite.
                    const uint32_t tile = entries + (e + 1) * S::entry;
                    for (int c = quarter * 32 + lane; c < kTile * (D / 8); c += active * 32) {
                        const int t = c / (D / 8), chunk = c % (D / 8), i = i0 + t;
                        const uint32_t at = tile + (chunk >> 3) * kBlock + t * 128 + (((chunk & 7) ^ (t & 7)) << 4);
                        if (!(pieces >> (t >> 4) & 1) || i >= unit.len || i < unit.first) {
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" :: "r"(at), "r"(0u) : "memory");
                        } else if (i >= open || i < wide) {
                            uint32_t x[4];
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
                            if (not_finite2(x[0]) || not_finite2(x[1]) || not_finite2(x[2]) || not_finite2(x[3])) {
                                unsigned who = 0;
                                for (int n = 0; n < a.tokens; ++n)
                                    if (i < open + n && (a.window == 0 || i >= open + n - a.window)) who |= 1u << n;
#pragma unroll
                                for (int q = 0; q < 8; ++q) {
                                    const uint32_t half = q & 1 ? 0xffff0000u : 0xffffu;
                                    if (not_finite2(x[q >> 1] & half)) {
                                        atomicOr(my_spoil + chunk * 8 + q, who);
                                        x[q >> 1] &= ~half;
                                    }
                                }
                                spoiled[g] = 1;
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
                            }
                        }
                    }
                    tc::fence_async_smem();
                }
                tmem_wait_st();
                tc::fence_before_sync();
                if (j == first_j) take_back();              // O is written anew
                __syncwarp();
                if (ok && lane == 0) tc::mbar_arrive(p_ready + 8 * g);
                ++k;
                e += 2 * NG;
                if (e >= E) {
                    e -= E;
                    phase ^= 1;
                }
            }
            if (tiles > 0) wait(pv_done + 8 * g, (k - 1) & 1);
            tc::fence_after_sync();
            if (g > 0) {
                take_back();
                stats[g * 128 + row] = make_float2(m, l);
                bar_sync(kBarActive + g, active * 32);      // (and what any of its warps spoiled)
                if (ok && lane == 0) tc::mbar_arrive(merged);
                continue;
            }
            bar_sync(kBarActive, active * 32);
            // whether the second group has sums of this unit
            const bool two = NG > 1 && unit.count > ((1 - unit.seq0) & (NG - 1));
            float f0 = 1.f, f1 = 0.f, total = l, nm = m;
            if (NG > 1) {
                wait(merged, u & 1);
                tc::fence_after_sync();
                const float2 other = stats[128 * (NG - 1) + row];
                nm = fmaxf(m, other.x);
                const float ref = nm == -INFINITY ? 0.f : nm;
                f0 = exp2_fast(m - ref);
                f1 = exp2_fast(other.x - ref);
                total = l * f0 + other.y * f1;
            }
            if (ok) {
                const bool bad = spoiled[0] || (NG > 1 && spoiled[NG - 1]);
                const bool whole = unit.slot < 0, there = row < rows;
                const long long orow = ((long long)unit.n * a.tokens + token) * a.d.hq + unit.h * a.d.grp + row - token * a.d.grp;
                float *part = attn_part(a, blockIdx.x, max(unit.slot, 0));
                const float inv = whole ? (total == 0.f ? 0.f : 1.f / total) : 1.f;
                for (int c = 0; c < D; c += 16) {
                    float x[16];
                    if (tiles > 0) {
                        tc::tmem_ld16(t_o + c, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] *= f0;
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = 0.f;
                    }
                    if (two) {
                        float y[16];
                        tc::tmem_ld16(t_o + D + c, y);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = fmaf(y[i], f1, x[i]);
                    }
                    if (bad) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if ((spoil[c + i] | (NG > 1 ? spoil[(NG - 1) * D + c + i] : 0u)) >> token & 1) x[i] = NAN;
                    }
                    if (!there) continue;
                    if (whole) {
                        uint4 *to = reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + orow * D + c);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            to[i] = make_uint4(pack_bf16(x[8 * i] * inv, x[8 * i + 1] * inv), pack_bf16(x[8 * i + 2] * inv, x[8 * i + 3] * inv),
                                               pack_bf16(x[8 * i + 4] * inv, x[8 * i + 5] * inv), pack_bf16(x[8 * i + 6] * inv, x[8 * i + 7] * inv));
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) store4f(part + row * D + c + 4 * i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
                    }
                }
                if (there) {
                    if (!whole) *reinterpret_cast<float2 *>(part + rows * D + 2 * row) = make_float2(nm, total);
                    else if (a.lse) a.lse[orow] = total == 0.f ? -INFINITY : (nm + log2f(total)) * kLn2;
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (NG > 1 && ok && lane == 0) tc::mbar_arrive(taken);
        }
        if (!ok && lane == 0) set_error(a.err, GDN_DEVERR_TIMEOUT);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 4 * NG) tc::tmem_dealloc(tmem, 512);
}

template <int D, int NG, int RB> cudaError_t run(AttnDecodeArgs a, const Maps &maps, cudaStream_t s) {
    using S = Shape<D, NG, RB>;
    const auto kernel = attn_decode_rows_kernel<D, NG, RB>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
    if (e != cudaSuccess) return e;
    a.ctas = sm_count();
    const cudaError_t l = launch_early(kernel, dim3(a.ctas), S::threads, S::bytes, s, a, maps);
    return l != cudaSuccess ? l : launch_attn_join(a, true, s);
}
template <int D> cudaError_t run_rows(const AttnDecodeArgs &a, const Maps &maps, cudaStream_t s) {
    constexpr int NG = D == 256 ? 1 : 2;                   // O of two groups fills tensor memory at 128 columns
    return a.d.grp * a.tokens <= 64 ? run<D, NG, 64>(a, maps, s) : run<D, NG, 128>(a, maps, s);
}

}  // namespace

cudaError_t launch_attn_decode_rows(const AttnDecodeArgs &a, cudaStream_t s) {
    Maps maps;
    if (!encode_pool(&maps.k, a.k_pages, a.d) || !encode_pool(&maps.v, a.v_pages, a.d) || !encode_queries(&maps.q, a)) return cudaErrorInvalidValue;
    return a.d.D == 64 ? run_rows<64>(a, maps, s) : a.d.D == 128 ? run_rows<128>(a, maps, s) : run_rows<256>(a, maps, s);
}

}  // namespace gdn
