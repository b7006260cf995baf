// attn_decode_tc.cu -- attention of a few new tokens over a paged bf16 cache, on the tensor cores.
//
// The shares, parts and join of attn_decode.cu; here a tile is 64 tokens.  Two warps copy tiles with TMA into a ring of
// shared-memory entries (K and V of a tile in entries of their own, 128-byte swizzled).  Two sets of four warps take turns
// with the tiles, for up to 16 query rows:
//   S = Q K^T    warp w the tile's tokens 16 w .. 16 w + 15
//   P = exp(S - m), the four warps having passed each other the rows' maxima; m, l and o in 32 bits
//   O += P V     warp w the columns D/4 w .., P passed through shared memory
// and their sums are added where a unit ends.  P is split in two bf16 parts, 16 bits of its 24: that adds 2e-6 to o (of 8,000
// tokens; in 32 bits P and the sums err by 4e-7) in front of its own rounding of 1.7e-3.
//
// HBM-bound: 64 sequences of up to 16,384 tokens, 8 key heads of 128 columns (2.3 GB) take 346 us, 0.98 of the copy rate; one of
// 131,072 tokens, 2 key heads of 256 columns (268 MB) 49 us, 0.81: 2 us until lengths and shares are known, 3 until the first
// tile is there, 3 for the join (a third tile of 256 columns in shared memory, with room for 8 query rows: no gain, 50.7).  One
// token over 700 takes 8.7 us, all latency.  16 rows of m16n8k16 products need 24 operations a byte of the cache (16 of K, 32 of V:
// both parts of P), at the 600 TFLOP/s that they reach on this GPU (16 warps an SM with nothing else) 0.27 of the time that the
// bytes take.  (A tcgen05 product has 64 or 128 rows, and the sums over tokens of its transposed form lie across lanes.)
#include "attn_tc.cuh"

namespace gdn {

namespace {

using namespace attn_tc;

constexpr int kLead = 1;                           // tiles that a unit's end costs (0 to 3: the same times)
constexpr int kPPitch = kTile * 2 + 16;            // bytes of a row of P: ldmatrix without bank conflicts

constexpr int kRows = 16, kSets = 2, kUnits = 2;   // query rows of a product, sets of warps, query blocks in flight
constexpr int kConsumers = kSets * 128, kThreads = kConsumers + 64;

template <int D> struct Shape {
    static constexpr int entry = kTile * D * 2, q_pitch = D * 2 + 16, q_block = kRows * q_pitch;
    static constexpr int p_block = kRows * kPPitch, merge = kRows * D * 4;         // merge: of the second set
    static constexpr int fixed = kUnits * q_block + 2 * kSets * p_block + merge + kSets * kRows * 4 * 4 * 2 + kRows * 8 + 1024;
    static constexpr int limit = 227 * 1024 - 1024;
    static constexpr int fit = (limit - fixed) / entry, turn = 2 * kSets;
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
enum { kBarSet = 1 };                // the first set's named barrier

template <int D> __global__ void __launch_bounds__(kThreads, 1) attn_decode_tc_kernel(const AttnDecodeArgs a, const __grid_constant__ Maps maps) {
    using S = Shape<D>;
    constexpr int KS = D / 16, NT = D / 32;                         // NT: 8-column blocks of a warp's share of O
    constexpr uint32_t E = S::entries, R = E / 2;                   // entries of K, then as many of V
    extern __shared__ unsigned char raw[];
    __shared__ long long sums[33];
    __shared__ int found[3];
    __shared__ uint64_t bars[2 * kMaxEntries + 2 * kUnits + 2];
    __shared__ int pieces_of[kMaxEntries];                          // which 16-token pieces of an entry's tile are there
    __shared__ Unit units[kUnits];
    unsigned char *base = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    unsigned char *q_mem = base + E * S::entry, *p_mem = q_mem + kUnits * S::q_block;
    float *merge = reinterpret_cast<float *>(p_mem + 2 * kSets * S::p_block);      // [kRows][D] of the second set
    float *tops = merge + kRows * D;                                // [sets][kRows][4 warps]
    float *totals = tops + kSets * kRows * 4;                       // the same
    float2 *stats = reinterpret_cast<float2 *>(totals + kSets * kRows * 4);  // [kRows] of the second set: m and l
    const uint32_t entries = tc::smem_u32(base), full = tc::smem_u32(bars), empty = full + 8 * kMaxEntries,
                   ufull = empty + 8 * kMaxEntries, uempty = ufull + 8 * kUnits, merged = uempty + 8 * kUnits, taken = merged + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rows = a.d.grp * a.tokens;
    if (tid == 0) {
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
        for (uint32_t e = 0; e < E; ++e) {
            tc::mbar_init(full + 8 * e, 1);
            tc::mbar_init(empty + 8 * e, 4);
        }
        for (int u = 0; u < kUnits; ++u) {
            tc::mbar_init(ufull + 8 * u, 1);
            tc::mbar_init(uempty + 8 * u, kConsumers / 32);
        }
        tc::mbar_init(merged, 4);
        tc::mbar_init(taken, 4);
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
        if (tid == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }

    if (warp >= kConsumers / 32) {
        // ------------------------------------------------------------ copies
        const uint32_t kv = warp - kConsumers / 32, at = kv * R;
        copy_tiles<D, kUnits>(a, w, maps, kv, R, entries + at * S::entry, full + 8 * at, empty + 8 * at, ufull, uempty, pieces_of + at, units, (uint32_t)rows * D * 2,
                                 [&](uint32_t us, int n, int h, uint32_t bar) {
            if (lane < rows) {
                const int tok = lane / a.d.grp, g = lane - tok * a.d.grp;
                tc::bulk_g2s(tc::smem_u32(q_mem) + us * S::q_block + lane * S::q_pitch,
                             (const __nv_bfloat16 *)a.q + ((long long)n * a.tokens + tok) * a.ld_q + (long long)(h * a.d.grp + g) * a.hs_q, D * 2,
                             bar);
            }
        });
        return;
    }

    // ---------------------------------------------------------------- products
    const int set = warp >> 2, wg = warp & 3, g = lane >> 2, t4 = lane & 3;
    // the new token of this thread's rows
    const int token[2] = {min(g / a.d.grp, a.tokens - 1), min((g + 8) / a.d.grp, a.tokens - 1)};
    const uint32_t p_hi = tc::smem_u32(p_mem) + set * 2 * S::p_block, p_lo = p_hi + S::p_block;
    float *my_tops = tops + set * kRows * 4, *my_totals = totals + set * kRows * 4;
    // ldmatrix addresses: rows of Q and P, tokens of K and V
    const uint32_t q_lane = (lane & 15) * S::q_pitch + (lane >> 4) * 16, p_lane = (lane & 15) * kPPitch + (lane >> 4) * 16;
    const uint32_t k_token = wg * 16 + (lane & 7) + ((lane >> 4) << 3), k_half = (lane >> 3) & 1;
    const uint32_t v_token = (lane & 7) + (((lane >> 3) & 1) << 3), v_half = lane >> 4;
    uint32_t e = set, phase = 0;                        // K's entry of the set's next tile
    bool ok = true;
    int u = 0;
    for (bool more = true; more; ++u) {
        const uint32_t us = u % kUnits;
        // a set's warps give up together: they meet at its barrier
        if (!bar_all(kBarSet + set, 128, ok && tc::mbar_wait(ufull + 8 * us, (u / kUnits) & 1, a.wait_ns))) {
            ok = false;
            break;
        }
        const Unit unit = units[us];
        more = unit.more;
        const uint32_t q_base = tc::smem_u32(q_mem) + us * S::q_block + q_lane;
        float m[2], l[2], o[NT][4];
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int c = 0; c < NT; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
        // what all rows see lies below `open`, and not below `wide`
        const int open = unit.len - a.tokens + 1, wide = a.window > 0 ? unit.len - a.window : 0;
        for (int j = (set - unit.seq0) & (kSets - 1); j < unit.count; j += kSets) {
            const int i0 = unit.i0 + j * kTile;
            const uint32_t v_e = R + e;
            if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(full + 8 * e, phase, a.wait_ns));
            const int pieces = pieces_of[e];
            const bool masked = pieces != 15 || i0 + kTile > open || i0 < wide;
            float s[2][4];
#pragma unroll
            for (int c = 0; c < 2; ++c) s[c][0] = s[c][1] = s[c][2] = s[c][3] = 0.f;
            const uint32_t k_row = entries + e * S::entry + k_token * 128;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t b[4];
                const uint32_t chunk = 2 * ks + k_half;
                ldsm4(k_row + (chunk >> 3) * (kTile * 128) + (((chunk & 7) ^ (k_token & 7)) << 4), b);
                uint32_t q[4];
                ldsm4(q_base + ks * 32, q);
                mma16816(s[0], q, b[0], b[1]);
                mma16816(s[1], q, b[2], b[3]);
            }
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(empty + 8 * e);     // what never came is not asked for again
            if (masked) {
                const bool piece = pieces >> wg & 1;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int i = i0 + wg * 16 + c * 8 + t4 * 2 + (x & 1), end = open + token[x >> 1];
                        if (!(piece && i < end && (a.window == 0 || i >= end - a.window))) s[c][x] = -INFINITY;
                    }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float top = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (t4 == 0) my_tops[(r * 8 + g) * 4 + wg] = top;
            }
            bar_sync(kBarSet + set, 128);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float4 v = *reinterpret_cast<const float4 *>(my_tops + (r * 8 + g) * 4);
                const float nm = fmaxf(m[r], fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) * a.scale_log2);
                const float ref = nm == -INFINITY ? 0.f : nm, back = exp2_fast(m[r] - ref);
                m[r] = nm;
                l[r] *= back;
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    o[c][2 * r] *= back;
                    o[c][2 * r + 1] *= back;
                }
                const uint32_t row = (r * 8 + g) * kPPitch + (wg * 16 + t4 * 2) * 2;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float p0 = exp2_fast(fmaf(s[c][2 * r], a.scale_log2, -ref)),
                                p1 = exp2_fast(fmaf(s[c][2 * r + 1], a.scale_log2, -ref));
                    l[r] += p0 + p1;
                    const uint32_t hi = pack_bf16(p0, p1);
                    const uint32_t lo = pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
                    asm volatile("st.shared.b32 [%0], %1;" :: "r"(p_hi + row + c * 16), "r"(hi) : "memory");
                    asm volatile("st.shared.b32 [%0], %1;" :: "r"(p_lo + row + c * 16), "r"(lo) : "memory");
                }
            }
            bar_sync(kBarSet + set, 128);
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
                    uint32_t p[4];
                    ldsm4(p_hi + p_lane + ks * 32, p);
#pragma unroll
                    for (int c = 0; c < NT; ++c) mma16816(o[c], p, b[c >> 1][(c & 1) * 2], b[c >> 1][(c & 1) * 2 + 1]);
                    ldsm4(p_lo + p_lane + ks * 32, p);
#pragma unroll
                    for (int c = 0; c < NT; ++c) mma16816(o[c], p, b[c >> 1][(c & 1) * 2], b[c >> 1][(c & 1) * 2 + 1]);
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
                    float x[NT][4];
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[c][k] = o[c][k];
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
                            ldsm4((part ? p_lo : p_hi) + p_lane + ks * 32, p);
#pragma unroll
                            for (int c = 0; c < NT; ++c) mma16816(x[c], p, b[c >> 1][(c & 1) * 2], b[c >> 1][(c & 1) * 2 + 1]);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (!odd || token[k >> 1] == pass) o[c][k] = x[c][k];
                }
            }
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(empty + 8 * v_e);
            e += kSets;
            if (e >= R) {
                e -= R;
                phase ^= 1;
            }
        }
        if (ok && lane == 0) tc::mbar_arrive(uempty + 8 * us);
        // the rows' sums over the set's warps; then both sets' together, by the first one, while the other goes on
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float v = l[r];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if (t4 == 0) my_totals[(r * 8 + g) * 4 + wg] = v;
        }
        bar_sync(kBarSet + set, 128);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float4 v = *reinterpret_cast<const float4 *>(my_totals + (r * 8 + g) * 4);
            l[r] = (v.x + v.y) + (v.z + v.w);
        }
        const int col0 = wg * (D / 4) + t4 * 2;
        if (set > 0) {
            if (u > 0 && ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(taken, (u - 1) & 1, a.wait_ns));
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r * 8 + g;
#pragma unroll
                for (int c = 0; c < NT; ++c)
                    *reinterpret_cast<float2 *>(merge + row * D + col0 + c * 8) = make_float2(o[c][2 * r], o[c][2 * r + 1]);
                if (wg == 0 && t4 == 0) stats[row] = make_float2(m[r], l[r]);
            }
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(merged);
            continue;
        }
        if (ok) ok = __all_sync(0xffffffffu, tc::mbar_wait(merged, u & 1, a.wait_ns));
        if (!ok) continue;
        float *part = attn_part(a, blockIdx.x, max(unit.slot, 0));
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = r * 8 + g;
            if (row >= rows) continue;
            // both sums on the larger of the maxima
            const float2 other = stats[row];
            const float top = fmaxf(m[r], other.x), ref = top == -INFINITY ? 0.f : top;
            const float own = exp2_fast(m[r] - ref), f = exp2_fast(other.x - ref), total = fmaf(other.y, f, l[r] * own);
            const int head = unit.h * a.d.grp + row - token[r] * a.d.grp;
            const long long orow = ((long long)unit.n * a.tokens + token[r]) * a.d.hq + head;
            const float inv = unit.slot >= 0 ? 1.f : total == 0.f ? 0.f : 1.f / total;
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const float2 x = *reinterpret_cast<const float2 *>(merge + row * D + col0 + c * 8);
                const float v0 = fmaf(x.x, f, o[c][2 * r] * own) * inv, v1 = fmaf(x.y, f, o[c][2 * r + 1] * own) * inv;
                if (unit.slot >= 0)
                    *reinterpret_cast<float2 *>(part + row * D + col0 + c * 8) = make_float2(v0, v1);
                else
                    *reinterpret_cast<uint32_t *>((__nv_bfloat16 *)a.out + orow * D + col0 + c * 8) = pack_bf16(v0, v1);
            }
            if (wg == 0 && t4 == 0) {
                if (unit.slot >= 0)
                    *reinterpret_cast<float2 *>(part + rows * D + 2 * row) = make_float2(top, total);
                else if (a.lse)
                    a.lse[orow] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
            }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(taken);
    }
    if (!ok && lane == 0) set_error(a.err, GDN_DEVERR_TIMEOUT);
}

template <int D> cudaError_t run(AttnDecodeArgs a, const Maps &maps, cudaStream_t s) {
    using S = Shape<D>;
    const auto kernel = attn_decode_tc_kernel<D>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes);
    if (e != cudaSuccess) return e;
    a.ctas = sm_count();
    a.lead = kLead;
    const cudaError_t l = launch_early(kernel, dim3(a.ctas), kThreads, S::bytes, s, a, maps);
    return l != cudaSuccess ? l : launch_attn_join(a, true, s);
}

}  // namespace

cudaError_t launch_attn_decode_tc(const AttnDecodeArgs &a, cudaStream_t s) {
    Maps maps;
    if (!encode_pool(&maps.k, a.k_pages, a.d) || !encode_pool(&maps.v, a.v_pages, a.d)) return cudaErrorInvalidValue;
    maps.q = maps.k;
    return a.d.D == 64 ? run<64>(a, maps, s) : a.d.D == 128 ? run<128>(a, maps, s) : run<256>(a, maps, s);
}

}  // namespace gdn
