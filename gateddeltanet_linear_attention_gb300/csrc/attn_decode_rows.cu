// attn_decode_rows.cu -- attention of new tokens over a paged bf16 cache where a key head has many query rows (17 to 128:
// verification rounds, many query heads a key head), on tcgen05.
//
// The shares, parts and join of attn_decode.cu, tiles of 64 tokens copied as for the kernel of few rows.  With the query rows
// as the 128 rows of the products, both accumulators in TMEM:
//   S = Q K^T     rows x 64 tokens; K from shared memory as TMA left it
//   P = exp(S - m) a thread a row: maximum and sum need no other lane; P, in two bf16 parts (16 bits), in the place of S
//   O += P V      P from TMEM, V from shared memory as TMA left it
// Two groups of four warps (one at 256 columns) take turns with the tiles, each with its own S, O, m and l; O of both lies in
// the same lanes, so where a unit ends each group adds both, in half of the columns.
//
// m is the maximum of a row's first tile and is raised only where a score passes it by 8 powers of two: P stays below 256,
// which changes no rounding, and O is seldom scaled again.
//
// Each group has S twice, so that the next tile's scores are there when its warps are done with one.  With 32 sequences of up to
// 8,192 tokens, 8 new ones each, 4 key heads of 128 columns, 8 query heads each (278 MB): 57 us with the join kernel, 0.72 of the
// copy rate.  A tile takes a group's warps 1,500 cycles (745 of them 64 exponentials a thread), and both groups wait for tiles: one
// comes in 1,500 to 1,600 cycles, its bytes take 1,400.  The rest is the first tile's way (5 us of 57), units' ends and the join.
// With 16 query heads each, 128 rows, the same cache takes 65 us; 2 key heads of 256 columns 71 (one group); one sequence of 131,072
// tokens, 2 key heads of 128 columns, 128 rows 55 us, floor 20 (by themselves the kernel 35, the join of 76 parts of 128 rows 32).
#include "attn_tc.cuh"

namespace gdn {

namespace {

using namespace attn_tc;

// Tiles that a unit's end and the next one's start cost: sums whole 1,100 cycles, the groups' meeting 2,000 to 2,600, outputs
// 2,300 to 3,000, first scores 1,000.  With 0, 2, 4 and 6: 70, 63, 59 and 58 us for the 32 sequences above, and 133, 124 and 116
// (2, 4, 6) for 64 sequences of up to 4,096 tokens, 8 key heads, 4 query heads each.
constexpr int kLead = 6;
constexpr float kSlack = 8.f;                      // powers of two that a score may pass m by

// NG groups; room for RB query rows (products read 128: behind them whatever follows, into lanes that nobody reads).
template <int D, int NG, int RB> struct Shape {
    static constexpr int threads = (5 * NG + 2) * 32;
    static constexpr int units = D == 256 && RB == 128 ? 1 : 2;
    static constexpr int entry = kTile * D * 2, q_block = RB * D * 2;
    static constexpr int fixed = units * q_block + NG * (128 * 8 + 2 * D * 4) + 1024;
    static constexpr int limit = 227 * 1024 - 1024;
    static constexpr int fit = (limit - fixed) / entry, most = fit < kMaxEntries ? fit : kMaxEntries, each = most / NG;
    // Multiples of the groups: an entry then serves tiles of one group alone.  (V's are held longer, but a third for K and two
    // for V left the scores waiting: 67 us against 57.)
    static constexpr int k_entries = NG * (each / 2), entries = NG * each, v_entries = entries - k_entries;
    static constexpr int bytes = fixed + entries * entry;
    static constexpr uint32_t col_o = 128 * NG;    // TMEM: S and P of group g's even and odd tiles at 128 g and 64 on, its O at col_o + g D
    static_assert(k_entries >= NG && v_entries >= NG, "a tile of each group in flight, in entries of its own");
    static_assert(128 * NG + NG * D <= 512, "tensor memory");
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
enum { kBarGroup = 1 };                            // of each group

// Whether the phase of this parity is over.
__device__ __forceinline__ bool test_wait(uint32_t b, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(done) : "r"(b), "r"(parity) : "memory");
    return done != 0;
}

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
    constexpr uint32_t E = S::entries, KE = S::k_entries, VE = S::v_entries, kBlock = kTile * 128, kQBlock = RB * 128;
    extern __shared__ unsigned char raw[];
    __shared__ long long sums[33];
    __shared__ int found[3], spoiled[2][NG];
    __shared__ uint32_t tmem_base;
    __shared__ uint64_t bars[2 * kMaxEntries + 2 * kUnits + 9 * NG];
    __shared__ int pieces_of[kMaxEntries];
    __shared__ Unit units[kUnits];
    unsigned char *base = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    // queries in front of the ring, so that what products read behind them is shared memory of this CTA
    unsigned char *q_mem = base, *ring = base + kUnits * S::q_block;
    float2 *stats = reinterpret_cast<float2 *>(ring + E * S::entry);               // [groups][128]: m and l
    unsigned *spoil = reinterpret_cast<unsigned *>(stats + NG * 128);              // [even, odd units][groups][D]: new tokens whose sum is not finite
    const uint32_t entries = tc::smem_u32(ring), full = tc::smem_u32(bars), empty = full + 8 * kMaxEntries,
                   ufull = empty + 8 * kMaxEntries, uempty = ufull + 8 * kUnits, s_full = uempty + 8 * kUnits, p_ready = s_full + 16 * NG,
                   pv_done = p_ready + 16 * NG, ended = pv_done + 16 * NG, merged = ended + 8 * NG, taken = merged + 8 * NG;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rows = a.d.grp * a.tokens, active = (rows + 31) / 32;                // warps of a group that have rows
    if (tid == 0) {
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
        prefetch_map(&maps.q);
        for (uint32_t e = 0; e < E; ++e) {
            tc::mbar_init(full + 8 * e, 1);
            tc::mbar_init(empty + 8 * e, 1);
        }
        for (int u = 0; u < kUnits; ++u) {
            tc::mbar_init(ufull + 8 * u, 1);
            tc::mbar_init(uempty + 8 * u, 5 * NG);
        }
        // even and odd tiles of a group on barriers of their own: no waiter is ever two phases behind
        for (int g = 0; g < 2 * NG; ++g) {
            tc::mbar_init(s_full + 8 * g, 1);
            tc::mbar_init(p_ready + 8 * g, active);
            tc::mbar_init(pv_done + 8 * g, 1);
        }
        for (int g = 0; g < NG; ++g) {
            tc::mbar_init(ended + 8 * g, 1);
            tc::mbar_init(merged + 8 * g, active);
            tc::mbar_init(taken + 8 * g, active);
            spoiled[0][g] = spoiled[1][g] = 0;
        }
        tc::mbar_fence_init();
    }
    for (int i = tid; i < 2 * NG * D; i += kThreads) spoil[i] = 0u;
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

    if (warp == 4 * NG || warp == 5 * NG + 1) {
        // ------------------------------------------------------------ copies
        const uint32_t kv = warp == 4 * NG ? 0 : 1, at = kv * KE;
        copy_tiles<D, kUnits>(a, w, maps, kv, kv ? VE : KE, entries + at * S::entry, full + 8 * at, empty + 8 * at, ufull, uempty, pieces_of + at,
                              units, (uint32_t)rows * D * 2,
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
        const uint32_t lead = elect_lane(), t_s = tmem + g * 128, t_o = tmem + S::col_o + g * D;
        // Scores of tile `ks` of the group, one ahead at most of the sums of tile `kp`: whatever can go first goes.
        uint32_t se = g, sphase = 0, ks = 0, pe = KE + g, pphase = 0, kp = 0, fresh = 0;      // fresh: tiles that begin a unit's sums
        int u = 0, j = 0, count = 0, opened = 0;            // the unit that the scores are in; whether its queries are there
        bool ok = true, first = true, more = true;
        uint64_t q_desc = 0, t0 = 0;
        auto there = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, test_wait(b, parity)); };
        while (more || opened || kp < ks) {
            bool moved = false;
            if (!opened && more && there(ufull + 8 * (u % kUnits), (u / kUnits) & 1)) {
                const Unit &unit = units[u % kUnits];
                count = unit.count;
                more = unit.more;
                j = (g - unit.seq0) & (NG - 1);
                q_desc = desc_k(tc::smem_u32(q_mem) + (u % kUnits) * S::q_block);
                opened = 1;
                first = true;
                moved = true;
            }
            if (opened && j < count && ks - kp < 2 && there(full + 8 * se, sphase) &&
                (ks < 2 || there(pv_done + 16 * g + 8 * (ks & 1), ((ks - 2) >> 1) & 1))) {
                tc::fence_after_sync();
                const uint64_t k_desc = desc_k(entries + se * S::entry);
#pragma unroll
                for (int c = 0; c < KS; ++c) mma_ss(lead, t_s + (ks & 1) * 64, q_desc + step_k(c, kQBlock), k_desc + step_k(c, kBlock), id_s, c > 0);
                commit(lead, s_full + 16 * g + 8 * (ks & 1));
                commit(lead, empty + 8 * se);
                fresh = first ? fresh | 1u << (ks & 1) : fresh & ~(1u << (ks & 1));
                first = false;
                ++ks;
                j += NG;
                se += NG;
                if (se >= KE) {
                    se -= KE;
                    sphase ^= 1;
                }
                moved = true;
            }
            if (opened && j >= count) {                     // the unit's queries have been used
                commit(lead, uempty + 8 * (u % kUnits));
                ++u;
                opened = 0;
            }
            if (kp < ks && there(full + 8 * pe, pphase) && there(p_ready + 16 * g + 8 * (kp & 1), (kp >> 1) & 1)) {
                tc::fence_after_sync();
                const uint64_t v_desc = desc_mn(entries + pe * S::entry, kBlock);
                const uint32_t t_p = t_s + (kp & 1) * 64;
#pragma unroll
                for (int c = 0; c < 2 * kTile / 16; ++c)    // the leading parts of P, then the rest
                    mma_ts(lead, t_o, t_p + c * 8, v_desc + step_mn(c & (kTile / 16 - 1)), id_pv, c > 0 || !(fresh >> (kp & 1) & 1));
                commit(lead, pv_done + 16 * g + 8 * (kp & 1));
                commit(lead, empty + 8 * pe);
                ++kp;
                pe += NG;
                if (pe >= E) {
                    pe -= VE;
                    pphase ^= 1;
                }
                moved = true;
            }
            if (moved) {
                t0 = 0;
            } else {
                const uint64_t t = tc::globaltimer_ns();
                if (t0 == 0) t0 = t;
                if (!(ok = __all_sync(0xffffffffu, t - t0 <= a.wait_ns))) break;
            }
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
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16, t_s0 = tmem + lanes + g * 128, t_o0 = tmem + lanes + S::col_o, t_o = t_o0 + g * D;
        uint32_t e = KE + g, phase = 0, k = 0;             // V's entry of the group's next tile
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(b, parity, a.wait_ns)); };
        int u = 0;
        for (bool more = true; more; ++u) {
            const uint32_t us = u % kUnits;
            // A group's warps give up together, and clear their marks of two units before together: they meet at its barrier, and
            // what decides is known to all of them.  (Marked then, read in front of the barrier, marked anew behind it.)
            const bool here = ok && tc::mbar_wait(ufull + 8 * us, (u / kUnits) & 1, a.wait_ns);
            if (!bar_all(kBarGroup + g, 128, here && !spoiled[u & 1][g])) {
                if (!bar_all(kBarGroup + g, 128, here)) {
                    ok = false;
                    break;
                }
                // (the other group has taken that unit: this one's warps waited for it in the last one)
                for (int c = tid & 127; c < D; c += 128) spoil[((u & 1) * NG + g) * D + c] = 0u;
                spoiled[u & 1][g] = 0;
                bar_sync(kBarGroup + g, 128);
            }
            const Unit unit = units[us];
            more = unit.more;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(uempty + 8 * us);
            const int first_j = (g - unit.seq0) & (NG - 1), tiles = unit.count > first_j ? (unit.count - first_j + NG - 1) / NG : 0;
            // a group's O and statistics are the other's too until that has taken them
            bool mine = NG == 1 || u == 0;
            auto take_back = [&]() {
                if (!mine) wait(taken + 8 * (NG - 1 - g), (u - 1) & 1);
                mine = true;
            };
            if (!on) continue;
            float m = -INFINITY, l = 0.f;
            // what all rows see lies below `open`, and not below `wide`
            const int open = unit.len - a.tokens + 1, wide = a.window > 0 ? unit.len - a.window : 0;
            const int end = open + token, begin = a.window > 0 ? end - a.window : 0;
            for (int j = first_j; j < unit.count; j += NG) {
                const int i0 = unit.i0 + j * kTile;
                const uint32_t t_s = t_s0 + (k & 1) * 64;
                wait(s_full + 16 * g + 8 * (k & 1), (k >> 1) & 1);
                // V's entry stays this tile's until its product is done; K's may be another tile's by now
                wait(full + 8 * e, phase);
                tc::fence_after_sync();
                const int pieces = pieces_of[e];
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
                    wait(pv_done + 16 * g + 8 * ((k - 1) & 1), ((k - 1) >> 1) & 1);      // the sums are whole
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
                    const uint32_t tile = entries + e * S::entry;
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
                                        atomicOr(spoil + ((u & 1) * NG + g) * D + chunk * 8 + q, who);
                                        x[q >> 1] &= ~half;
                                    }
                                }
                                spoiled[u & 1][g] = 1;
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
                if (ok && lane == 0) tc::mbar_arrive(p_ready + 16 * g + 8 * (k & 1));
                ++k;
                e += NG;
                if (e >= E) {
                    e -= VE;
                    phase ^= 1;
                }
            }
            if (tiles > 0) wait(pv_done + 16 * g + 8 * ((k - 1) & 1), ((k - 1) >> 1) & 1);
            take_back();
            stats[g * 128 + row] = make_float2(m, l);
            tc::fence_before_sync();
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(merged + 8 * g);
            // all warps' statistics and sums (and what any of them spoiled); each group then ends a share of the columns
            for (int i = 0; i < NG; ++i) wait(merged + 8 * i, u & 1);
            tc::fence_after_sync();
            const float2 s0 = stats[row], s1 = NG > 1 ? stats[128 * (NG - 1) + row] : make_float2(-INFINITY, 0.f);
            const float nm = fmaxf(s0.x, s1.x), ref = nm == -INFINITY ? 0.f : nm;
            const float f0 = exp2_fast(s0.x - ref), f1 = exp2_fast(s1.x - ref), total = s0.y * f0 + s1.y * f1;
            // whether the groups have sums of this unit
            const bool one = unit.count > ((0 - unit.seq0) & (NG - 1)), two = NG > 1 && unit.count > ((1 - unit.seq0) & (NG - 1));
            if (ok) {
                const bool bad = spoiled[u & 1][0] || (NG > 1 && spoiled[u & 1][NG - 1]);
                const bool whole = unit.slot < 0, there = row < rows;
                const long long orow = ((long long)unit.n * a.tokens + token) * a.d.hq + unit.h * a.d.grp + row - token * a.d.grp;
                float *part = attn_part(a, blockIdx.x, max(unit.slot, 0));
                const float inv = whole ? (total == 0.f ? 0.f : 1.f / total) : 1.f;
                for (int c = g * (D / NG); c < (g + 1) * (D / NG); c += 16) {
                    float x[16];
                    if (one) {
                        tc::tmem_ld16(t_o0 + c, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] *= f0;
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = 0.f;
                    }
                    if (two) {
                        float y[16];
                        tc::tmem_ld16(t_o0 + D + c, y);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = fmaf(y[i], f1, x[i]);
                    }
                    if (bad) {
                        const unsigned *who = spoil + (u & 1) * NG * D + c;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if ((who[i] | who[(NG - 1) * D + i]) >> token & 1) x[i] = NAN;
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
                if (there && g == 0) {
                    if (!whole) *reinterpret_cast<float2 *>(part + rows * D + 2 * row) = make_float2(nm, total);
                    else if (a.lse) a.lse[orow] = total == 0.f ? -INFINITY : (nm + log2f(total)) * kLn2;
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (NG > 1 && ok && lane == 0) tc::mbar_arrive(taken + 8 * g);
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
    a.lead = kLead;
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
