// attn_decode_tc.cu -- attention of a few new tokens over a paged bf16 cache, on the tensor cores.
//
// The shares, parts and join of attn_decode.cu; here a tile is 64 tokens.  One warp copies tiles with TMA into a ring of
// shared-memory entries (K and V of a tile in entries of their own, 128-byte swizzled).  Groups of four warps compute:
//   S = Q K^T    warp w the tile's tokens 16 w .. 16 w + 15, for the group's query rows
//   P = exp(S - m), the four warps having passed each other the rows' maxima; m, l and o in 32 bits
//   O += P V     warp w the columns D/4 w .. of the group's rows, P passed through shared memory
// so that a byte of K and V is read from shared memory once for up to 32 query rows.  Groups of other rows take the same
// tiles; groups of the same rows (sets) take turns with them, and their sums are added where a unit ends.
//
// HBM-bound by design: 16 rows of m16n8k16 products need 16 operations a byte of the cache, 64 rows 64: at the 600
// TFLOP/s that these products reach on this GPU, 0.2 and 0.7 of the time that the bytes take.  (They run as mma.sync: a
// tcgen05 product has 64 or 128 rows, and the sums over tokens of its transposed form lie across lanes.)
// P is split in two bf16 parts, so that o loses nothing but its own rounding.
#include "attn_tc.cuh"

namespace gdn {

namespace {

using namespace attn_tc;

constexpr int kLead = 1;                           // tiles that a unit's end costs
constexpr int kPPitch = kTile * 2 + 16;            // bytes of a row of P: ldmatrix without bank conflicts

// MT blocks of 16 query rows a group, GR groups of rows, GS sets of each.
template <int D, int MT, int GR, int GS> struct Shape {
    static constexpr int groups = GR * GS, consumers = groups * 128, threads = consumers + 32, rows = 16 * MT * GR;
    static constexpr int units = MT > 1 ? 1 : 2;           // query blocks in flight
    static constexpr int entry = kTile * D * 2, q_pitch = D * 2 + 16, q_block = rows * q_pitch;
    static constexpr int p_block = 16 * MT * kPPitch, merge = 16 * MT * D * 4;     // merge: of each set but the first
    static constexpr int stats = groups * 16 * MT;         // rows of all groups
    static constexpr int fixed = units * q_block + 2 * groups * p_block + GR * (GS - 1) * merge + stats * (4 * 4 * 2 + 8) + 1024;
    static constexpr int limit = 227 * 1024 - 1024;
    static constexpr int fit = (limit - fixed) / entry, turn = 2 * GS;
    // a multiple of the sets' entries: an entry then serves tiles of one set alone, and no waiter is ever two phases
    // behind its barrier
    static constexpr int entries = fit < kMaxEntries ? fit / turn * turn : kMaxEntries;
    static constexpr int bytes = fixed + entries * entry;      // 1,024 of `fixed` to align the entries
    static_assert(entries >= turn && entries % turn == 0, "a tile of each set in flight, in entries of its own");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory"); }
enum { kBarGroup = 1 };              // the first group's named barrier

template <int D, int MT, int GR, int GS>
__global__ void __launch_bounds__((Shape<D, MT, GR, GS>::threads), 1) attn_decode_tc_kernel(const AttnDecodeArgs a, const __grid_constant__ Maps maps) {
    using S = Shape<D, MT, GR, GS>;
    constexpr int KS = D / 16, ROWS = S::rows, GROWS = 16 * MT, NT = D / 32;       // NT: 8-column blocks of a warp's share of O
    constexpr int kUnits = S::units, kThreads = S::threads, kConsumers = S::consumers;
    constexpr uint32_t E = S::entries;
    extern __shared__ unsigned char raw[];
    __shared__ long long sums[33];
    __shared__ int found[3];
    __shared__ uint64_t bars[2 * kMaxEntries + 2 * kUnits + 2 * GR];
    __shared__ int pieces_of[kMaxEntries];                          // which 16-token pieces of an entry's tile are there
    __shared__ Unit units[kUnits];
    unsigned char *base = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    unsigned char *q_mem = base + E * S::entry, *p_mem = q_mem + kUnits * S::q_block;
    float *merge = reinterpret_cast<float *>(p_mem + 2 * S::groups * S::p_block);  // [sets - 1][groups of rows][GROWS][D]
    float *tops = merge + GR * (GS - 1) * GROWS * D;                // [groups][GROWS][4 warps]
    float *totals = tops + S::stats * 4;                            // the same
    float2 *stats = reinterpret_cast<float2 *>(totals + S::stats * 4);   // [groups][GROWS]: m and l
    const uint32_t entries = tc::smem_u32(base), full = tc::smem_u32(bars), empty = full + 8 * kMaxEntries,
                   ufull = empty + 8 * kMaxEntries, uempty = ufull + 8 * kUnits, merged = uempty + 8 * kUnits, taken = merged + 8 * GR;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rows = a.d.grp * a.tokens, row0 = blockIdx.y * ROWS, mine = min(ROWS, rows - row0);
    if (tid == 0) {
        for (uint32_t e = 0; e < E; ++e) {
            tc::mbar_init(full + 8 * e, 1);
            tc::mbar_init(empty + 8 * e, 4 * GR);
        }
        for (int u = 0; u < kUnits; ++u) {
            tc::mbar_init(ufull + 8 * u, 1);
            tc::mbar_init(uempty + 8 * u, kConsumers / 32);
        }
        for (int r = 0; r < GR; ++r) {
            tc::mbar_init(merged + 8 * r, 4 * (GS - 1) + (GS == 1));
            tc::mbar_init(taken + 8 * r, 4);
        }
        tc::mbar_fence_init();
    }
    // rows that pad the query block stay zero
    for (int i = tid; i < kUnits * S::q_block / 16; i += kThreads) reinterpret_cast<uint4 *>(q_mem)[i] = make_uint4(0u, 0u, 0u, 0u);
    tc::fence_async_smem();
    await_previous();
    let_next_start();
    AttnWalk w;
    const bool work = attn_begin<kTile, kThreads>(a, blockIdx.x, sums, found, w);      // synchronises the block
    if (!work) {
        if (blockIdx.y == 0 && tid == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }

    if (warp == kConsumers / 32) {
        // ------------------------------------------------------------ copies
        copy_tiles<D, E, kUnits>(a, w, maps, entries, full, empty, ufull, uempty, pieces_of, units, (uint32_t)mine * D * 2,
                                 [&](uint32_t us, int n, int h, uint32_t bar) {
            for (int r = lane; r < mine; r += 32) {
                const int tok = (row0 + r) / a.d.grp, g = (row0 + r) - tok * a.d.grp;
                tc::bulk_g2s(tc::smem_u32(q_mem) + us * S::q_block + r * S::q_pitch,
                             (const __nv_bfloat16 *)a.q + ((long long)n * a.tokens + tok) * a.ld_q + (long long)(h * a.d.grp + g) * a.hs_q, D * 2,
                             bar);
            }
        });
        return;
    }

    // ---------------------------------------------------------------- products
    const int group = warp >> 2, wg = warp & 3, rg = group % GR, set = group / GR, g = lane >> 2, t4 = lane & 3, row_g = rg * GROWS;
    int token[MT][2];                                   // the new token of this thread's rows
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        token[mt][0] = min((row0 + row_g + mt * 16 + g) / a.d.grp, a.tokens - 1);
        token[mt][1] = min((row0 + row_g + mt * 16 + g + 8) / a.d.grp, a.tokens - 1);
    }
    const uint32_t p_hi = tc::smem_u32(p_mem) + group * 2 * S::p_block, p_lo = p_hi + S::p_block;
    float *my_tops = tops + group * GROWS * 4, *my_totals = totals + group * GROWS * 4;
    // ldmatrix addresses: rows of Q and P, tokens of K and V
    const uint32_t q_lane = (lane & 15) * S::q_pitch + (lane >> 4) * 16, p_lane = (lane & 15) * kPPitch + (lane >> 4) * 16;
    const uint32_t k_token = wg * 16 + (lane & 7) + ((lane >> 4) << 3), k_half = (lane >> 3) & 1;
    const uint32_t v_token = (lane & 7) + (((lane >> 3) & 1) << 3), v_half = lane >> 4;
    uint32_t e = 2 * set, phase = 0;                    // the entry of the set's next tile
    bool ok = true;
    int u = 0;
    for (bool more = true; more; ++u) {
        const uint32_t us = u % kUnits;
        // a group's warps give up together: they meet at its barrier
        if (!bar_all(kBarGroup + group, 128, ok && tc::mbar_wait(ufull + 8 * us, (u / kUnits) & 1, a.wait_ns))) {
            ok = false;
            break;
        }
        const Unit unit = units[us];
        more = unit.more;
        const uint32_t q_base = tc::smem_u32(q_mem) + us * S::q_block + row_g * S::q_pitch + q_lane;
        float m[MT][2], l[MT][2], o[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
            for (int c = 0; c < NT; ++c) o[mt][c][0] = o[mt][c][1] = o[mt][c][2] = o[mt][c][3] = 0.f;
        }
        // what all rows see lies below `open`, and not below `wide`
        const int open = unit.len - a.tokens + 1, wide = a.window > 0 ? unit.len - a.window : 0;
        for (int j = (set - unit.seq0) & (GS - 1); j < unit.count; j += GS) {
            const int i0 = unit.i0 + j * kTile;
            const uint32_t v_e = e + 1;                 // V follows its K
            if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(full + 8 * e, phase, a.wait_ns));
            const int pieces = pieces_of[e];
            const bool masked = pieces != 15 || i0 + kTile > open || i0 < wide;
            float s[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int c = 0; c < 2; ++c) s[mt][c][0] = s[mt][c][1] = s[mt][c][2] = s[mt][c][3] = 0.f;
            const uint32_t k_row = entries + e * S::entry + k_token * 128;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t b[4];
                const uint32_t chunk = 2 * ks + k_half;
                ldsm4(k_row + (chunk >> 3) * (kTile * 128) + (((chunk & 7) ^ (k_token & 7)) << 4), b);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t q[4];
                    ldsm4(q_base + mt * 16 * S::q_pitch + ks * 32, q);
                    mma16816(s[mt][0], q, b[0], b[1]);
                    mma16816(s[mt][1], q, b[2], b[3]);
                }
            }
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(empty + 8 * e);     // what never came is not asked for again
            if (masked) {
                const bool piece = pieces >> wg & 1;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int i = i0 + wg * 16 + c * 8 + t4 * 2 + (x & 1), end = open + token[mt][x >> 1];
                            if (!(piece && i < end && (a.window == 0 || i >= end - a.window))) s[mt][c][x] = -INFINITY;
                        }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float top = fmaxf(fmaxf(s[mt][0][2 * r], s[mt][0][2 * r + 1]), fmaxf(s[mt][1][2 * r], s[mt][1][2 * r + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    if (t4 == 0) my_tops[(mt * 16 + r * 8 + g) * 4 + wg] = top;
                }
            bar_sync(kBarGroup + group, 128);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float4 v = *reinterpret_cast<const float4 *>(my_tops + (mt * 16 + r * 8 + g) * 4);
                    const float nm = fmaxf(m[mt][r], fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) * a.scale_log2);
                    const float ref = nm == -INFINITY ? 0.f : nm, back = exp2_fast(m[mt][r] - ref);
                    m[mt][r] = nm;
                    l[mt][r] *= back;
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        o[mt][c][2 * r] *= back;
                        o[mt][c][2 * r + 1] *= back;
                    }
                    const uint32_t row = (mt * 16 + r * 8 + g) * kPPitch + (wg * 16 + t4 * 2) * 2;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float p0 = exp2_fast(fmaf(s[mt][c][2 * r], a.scale_log2, -ref)),
                                    p1 = exp2_fast(fmaf(s[mt][c][2 * r + 1], a.scale_log2, -ref));
                        l[mt][r] += p0 + p1;
                        const uint32_t hi = pack_bf16(p0, p1);
                        const uint32_t lo = pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
                        asm volatile("st.shared.b32 [%0], %1;" :: "r"(p_hi + row + c * 16), "r"(hi) : "memory");
                        asm volatile("st.shared.b32 [%0], %1;" :: "r"(p_lo + row + c * 16), "r"(lo) : "memory");
                    }
                }
            bar_sync(kBarGroup + group, 128);
            if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(full + 8 * v_e, phase, a.wait_ns));
            const uint32_t v_base = entries + v_e * S::entry;
            auto v_addr = [&](int ks, int pair) {
                const uint32_t chunk = wg * (D / 32) + 2 * pair + v_half, tok = ks * 16 + v_token;
                return v_base + (chunk >> 3) * (kTile * 128) + tok * 128 + (((chunk & 7) ^ (tok & 7)) << 4);
            };
            if (!masked) {
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ++ks) {
                    uint32_t b[NT / 2][4];
#pragma unroll
                    for (int pair = 0; pair < NT / 2; ++pair) ldsm4t(v_addr(ks, pair), b[pair]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t p[4];
                        ldsm4(p_hi + p_lane + mt * 16 * kPPitch + ks * 32, p);
#pragma unroll
                        for (int c = 0; c < NT; ++c) mma16816(o[mt][c], p, b[c >> 1][(c & 1) * 2], b[c >> 1][(c & 1) * 2 + 1]);
                        ldsm4(p_lo + p_lane + mt * 16 * kPPitch + ks * 32, p);
#pragma unroll
                        for (int c = 0; c < NT; ++c) mma16816(o[mt][c], p, b[c >> 1][(c & 1) * 2], b[c >> 1][(c & 1) * 2 + 1]);
                    }
                }
            } else {
                // Places that no row sees may hold anything and read as zero.  A value that is not finite in a place that
                // only some rows see would reach the others as 0 * inf: then each new token's rows are taken by themselves.
                auto kept = [&](int ks, int half, int from, int to) {    // mask of the pair of tokens of a B register
                    const int i = i0 + ks * 16 + half * 8 + t4 * 2;
                    const bool there = pieces >> ks & 1;
                    return (there && i >= from && i < to ? 0xffffu : 0u) | (there && i + 1 >= from && i + 1 < to ? 0xffff0000u : 0u);
                };
                bool odd = false;
                if (a.tokens > 1) {
                    for (int ks = 0; ks < kTile / 16; ++ks)
                        for (int pair = 0; pair < NT / 2; ++pair) {
                            uint32_t b[4];
                            ldsm4t(v_addr(ks, pair), b);
                            const uint32_t k0 = kept(ks, 0, unit.first, unit.len), k1 = kept(ks, 1, unit.first, unit.len);
                            odd |= not_finite2(b[0] & k0) | not_finite2(b[1] & k1) | not_finite2(b[2] & k0) | not_finite2(b[3] & k1);
                        }
                    odd = __any_sync(0xffffffffu, odd);
                }
                for (int pass = 0; pass < (odd ? a.tokens : 1); ++pass) {
                    const int to = odd ? open + pass : unit.len, from = odd ? (a.window > 0 ? to - a.window : 0) : unit.first;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        float x[NT][4];
#pragma unroll
                        for (int c = 0; c < NT; ++c)
#pragma unroll
                            for (int k = 0; k < 4; ++k) x[c][k] = o[mt][c][k];
#pragma unroll
                        for (int ks = 0; ks < kTile / 16; ++ks) {
                            const uint32_t k0 = kept(ks, 0, from, to), k1 = kept(ks, 1, from, to);
                            uint32_t b[NT / 2][4];
#pragma unroll
                            for (int pair = 0; pair < NT / 2; ++pair) {
                                ldsm4t(v_addr(ks, pair), b[pair]);
                                b[pair][0] &= k0; b[pair][1] &= k1; b[pair][2] &= k0; b[pair][3] &= k1;
                            }
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                uint32_t p[4];
                                ldsm4((part ? p_lo : p_hi) + p_lane + mt * 16 * kPPitch + ks * 32, p);
#pragma unroll
                                for (int c = 0; c < NT; ++c) mma16816(x[c], p, b[c >> 1][(c & 1) * 2], b[c >> 1][(c & 1) * 2 + 1]);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < NT; ++c)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (!odd || token[mt][k >> 1] == pass) o[mt][c][k] = x[c][k];
                    }
                }
            }
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(empty + 8 * v_e);
            e += 2 * GS;
            if (e >= E) {
                e -= E;
                phase ^= 1;
            }
        }
        if (ok && lane == 0) tc::mbar_arrive(uempty + 8 * us);
        // the rows' sums over the group's warps; then the sets' together, by the first one, while the others go on
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float v = l[mt][r];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (t4 == 0) my_totals[(mt * 16 + r * 8 + g) * 4 + wg] = v;
            }
        bar_sync(kBarGroup + group, 128);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float4 v = *reinterpret_cast<const float4 *>(my_totals + (mt * 16 + r * 8 + g) * 4);
                l[mt][r] = (v.x + v.y) + (v.z + v.w);
            }
        const int col0 = wg * (D / 4) + t4 * 2;
        if (GS > 1 && set > 0) {
            if (u > 0 && ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(taken + 8 * rg, (u - 1) & 1, a.wait_ns));
            float *mine_o = merge + ((set - 1) * GR + rg) * GROWS * D;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = mt * 16 + r * 8 + g;
#pragma unroll
                    for (int c = 0; c < NT; ++c)
                        *reinterpret_cast<float2 *>(mine_o + row * D + col0 + c * 8) = make_float2(o[mt][c][2 * r], o[mt][c][2 * r + 1]);
                    if (wg == 0 && t4 == 0) stats[group * GROWS + row] = make_float2(m[mt][r], l[mt][r]);
                }
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(merged + 8 * rg);
            continue;
        }
        if (GS > 1 && ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(merged + 8 * rg, u & 1, a.wait_ns));
        if (!ok) continue;
        float *part = attn_part(a, blockIdx.x, max(unit.slot, 0));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int in_group = mt * 16 + r * 8 + g, row = row_g + in_group;
                if (row >= mine) continue;
                // the sets' sums on the largest of their maxima
                float top = m[mt][r];
#pragma unroll
                for (int k = 1; k < GS; ++k) top = fmaxf(top, stats[(k * GR + rg) * GROWS + in_group].x);
                const float ref = top == -INFINITY ? 0.f : top, own = exp2_fast(m[mt][r] - ref);
                float total = l[mt][r] * own;
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    o[mt][c][2 * r] *= own;
                    o[mt][c][2 * r + 1] *= own;
                }
#pragma unroll
                for (int k = 1; k < GS; ++k) {
                    const float2 other = stats[(k * GR + rg) * GROWS + in_group];
                    const float f = exp2_fast(other.x - ref);
                    total = fmaf(other.y, f, total);
                    const float *from = merge + (((k - 1) * GR + rg) * GROWS + in_group) * D + col0;
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        const float2 x = *reinterpret_cast<const float2 *>(from + c * 8);
                        o[mt][c][2 * r] = fmaf(x.x, f, o[mt][c][2 * r]);
                        o[mt][c][2 * r + 1] = fmaf(x.y, f, o[mt][c][2 * r + 1]);
                    }
                }
                const int tok = token[mt][r], head = unit.h * a.d.grp + row0 + row - tok * a.d.grp;
                const long long orow = ((long long)unit.n * a.tokens + tok) * a.d.hq + head;
                const float inv = unit.slot >= 0 ? 1.f : total == 0.f ? 0.f : 1.f / total;
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const float v0 = o[mt][c][2 * r] * inv, v1 = o[mt][c][2 * r + 1] * inv;
                    if (unit.slot >= 0)
                        *reinterpret_cast<float2 *>(part + (row0 + row) * D + col0 + c * 8) = make_float2(v0, v1);
                    else
                        *reinterpret_cast<uint32_t *>((__nv_bfloat16 *)a.out + orow * D + col0 + c * 8) = pack_bf16(v0, v1);
                }
                if (wg == 0 && t4 == 0) {
                    if (unit.slot >= 0)
                        *reinterpret_cast<float2 *>(part + rows * D + 2 * (row0 + row)) = make_float2(top, total);
                    else if (a.lse)
                        a.lse[orow] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
                }
            }
        __syncwarp();
        if (GS > 1 && lane == 0) tc::mbar_arrive(taken + 8 * rg);
    }
    if (!ok && lane == 0) set_error(a.err, GDN_DEVERR_TIMEOUT);
}

template <int D, int MT, int GR, int GS> cudaError_t run(AttnDecodeArgs a, const Maps &maps, cudaStream_t s) {
    using S = Shape<D, MT, GR, GS>;
    const auto kernel = attn_decode_tc_kernel<D, MT, GR, GS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
    if (e != cudaSuccess) return e;
    // blocks of query rows read the same tiles: at the same time, so that the second one finds them in L2
    const int blocks = (a.d.grp * a.tokens + S::rows - 1) / S::rows;
    a.ctas = sm_count() / blocks;
    a.lead = kLead;
    const cudaError_t l = launch_early(kernel, dim3(a.ctas, blocks), S::threads, S::bytes, s, a, maps);
    return l != cudaSuccess ? l : launch_attn_join(a, true, s);
}
template <int D> cudaError_t run_rows(const AttnDecodeArgs &a, const Maps &maps, cudaStream_t s) {
    const int rows = a.d.grp * a.tokens;
    if constexpr (D == 256) {
        // two tiles fill shared memory
        return rows <= 16 ? run<D, 1, 1, 2>(a, maps, s) : run<D, 1, 2, 1>(a, maps, s);
    } else {
        return rows <= 16 ? run<D, 1, 1, 2>(a, maps, s) : rows <= 32 ? run<D, 1, 2, 2>(a, maps, s) : run<D, 1, 4, 1>(a, maps, s);
    }
}

}  // namespace

cudaError_t launch_attn_decode_tc(const AttnDecodeArgs &a, cudaStream_t s) {
    Maps maps;
    if (!encode_pool(&maps.k, a.k_pages, a.d) || !encode_pool(&maps.v, a.v_pages, a.d)) return cudaErrorInvalidValue;
    maps.q = maps.k;
    return a.d.D == 64 ? run_rows<64>(a, maps, s) : a.d.D == 128 ? run_rows<128>(a, maps, s) : run_rows<256>(a, maps, s);
}

}  // namespace gdn
