// ssm_scan_tc.cu -- the state space scan on the tensor cores: bf16 activations,
// d_state and head_dim of 64 or 128.
//
// A chunk of 128 tokens of one sequence, cs_r the summed log-decay of its tokens
// 0..r, S the state that enters it:
//   Y[r]  = sum_{i<=r} (C_r . B_i) exp(cs_r - cs_i) dt_i x_i  +  exp(cs_r) S^T C_r
//   S'    = exp(cs_127) S + dS,   dS = sum_i exp(cs_127 - cs_i) dt_i B_i x_i^T
// as four products on tcgen05, the accumulators in TMEM:
//   G  = C B^T                        (128 x 128 tokens)
//   Y2 = C S                          scaled by exp(cs_r) in place
//   Y  = Y2 + P X,  P[r][i] = G[r][i] exp(cs_r - cs_i) dt_i for i <= r
//   dS = (w X)^T B, w_i = exp(cs_127 - cs_i) dt_i
// A CTA walks the chunks of one segment for one unit: 128 value columns, one
// head of 128 or two heads of 64 of the same group, which share C, B and G.
//
// Precision.  B, C and x are exact 16-bit operands.  P and the copy of S that
// Y2 reads are rounded to bf16 (half a step each, like y itself).  The state is
// a 32-bit output that goes on for the whole sequence: it stays in fp32 and is
// updated by fp32 multiply-adds outside the tensor core, and w x enters dS in
// three bf16 parts (2^-26 of each value), smallest first, in a fresh
// accumulator per chunk: the tensor core truncates its sums, which would bias a
// state that it carried along itself.  w comes from a suffix sum of the
// log-decays (exact where it matters, near the chunk's end).  Log-decays are
// clamped at -60 a token: exp(-60) is nothing beside what the token adds, and
// differences of running sums keep their meaning.
//
// Roles (24 warps, one CTA per SM): warp 0 loads tiles by TMA, warp 1 issues
// the products, warp 2 stores y by TMA; A: log-decays, then G -> P; B: the
// state; C (two groups of 64 columns): Y2's scaling, the skip, the gate, y;
// D: the parts of w X.  Tiles (128 tokens x 128 columns, 128-byte swizzle) go
// through one ring in the order C, B, X, z; y leaves in the place of X.
//
// Bound by instruction issue (conversions between TMEM, registers and shared
// memory), not by memory or the tensor cores.
#include <cuda.h>   // CUtensorMap (the encoder itself is reached through the runtime)

#include <cstring>

#include "ssm_common.cuh"
#include "tc_sm103.cuh"

namespace gdn {

namespace {

constexpr int kL = 128;                        // tokens of a chunk
constexpr int kThreads = 24 * 32;
constexpr int kSlots = 5;
constexpr int kTile = kL * 128 * 2;            // bytes of a ring slot
constexpr int kHalfTile = kTile / 2;           // 128 rows x 128 bytes: one TMA box
constexpr int kXwPart = 16 * 128 * 2;          // one bf16 part of w X for 16 tokens (MN-major)
constexpr int kXwBuf = 3 * kXwPart;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLog = -60.0f;

// TMEM columns
constexpr uint32_t kColS = 0, kColDS = 128, kColY = 256, kColG = 384;

template <int N, int HU> struct TcSmem {
    static constexpr int RING = 0;
    static constexpr int S = RING + kSlots * kTile;          // bf16 state, 128 rows (value columns) x N
    static constexpr int XW = S + N * 256;
    static constexpr int ARR = XW + 2 * kXwBuf;              // [2][HU][3][128]: cp, w, e
    static constexpr int SUM = ARR + 2 * HU * 3 * 512;       // [2][HU][4] warp sums, then [2][HU] decays
    static constexpr int BAR = SUM + 2 * HU * 4 * 4 + 2 * HU * 4;
    static constexpr int NBAR = 2 * kSlots + 20;
    static constexpr int SLOT = (BAR + 7) / 8 * 8 + NBAR * 8;
    static constexpr int BYTES = SLOT + 16;
    static_assert(BYTES <= 232448, "shared memory of an SM");
};

// Barriers behind the ring's full[] and empty[].
// Where a waiter may be a phase
// behind (DS, A, ST), even and odd chunks have a barrier each: the next phase of either then
// needs the waiter's own progress.
enum { B_G = 0, B_P, B_S, B_XF0, B_XF1, B_XE0, B_XE1, B_DS0, B_DS1, B_Y2, B_YC, B_Y, B_YE, B_A0, B_A1, B_ST0, B_ST1,
       B_WG, B_FIX, B_END, B_COUNT };

// 128-byte-swizzled operands: rows of 128 bytes, 8-row groups of 1,024 bytes, 64-element blocks
// kHalfTile apart.  K-major: the row index is M or N, a 16-wide K step is 32 bytes further.
// MN-major: the row index is K, a 16-wide K step is 2,048 bytes further.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) { return tc::smem_desc(saddr, 16, 1024) | (2ull << 61); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
    return tc::smem_desc(saddr, kHalfTile, 1024) | (2ull << 61);
}
// K step ks of a K-major operand of up to 128 columns, in 16-byte units of the start address.
__device__ __forceinline__ uint64_t step_k(int ks) { return (uint64_t)((ks >> 2) * (kHalfTile >> 4) + (ks & 3) * 2); }
__device__ __forceinline__ uint64_t step_mn(int ks) { return (uint64_t)(ks * 128); }

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        :: "r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
           "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
           "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]),
           "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
           "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tma_store_2d(const void *tmap, uint32_t src_saddr, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
                 :: "l"(tmap), "r"(src_saddr), "r"(x), "r"(y) : "memory");
}
// 2^x, two units in the last place at most: its results are rounded to bf16.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

}  // namespace

struct SsmMaps {
    CUtensorMap x, b, c, z, y;
};

template <int N, int HU, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_scan_tc_kernel(const __grid_constant__ SsmScanArgs a, const __grid_constant__ SsmMaps maps) {
    using L = TcSmem<N, HU>;
    constexpr int P = 128 / HU;
    static_assert(L::NBAR == 2 * kSlots + B_COUNT, "barriers");
    extern __shared__ __align__(1024) unsigned char sm[];
    const SsmDims &d = a.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_group = (d.per + HU - 1) / HU, units = d.groups * per_group;
    const int unit = blockIdx.x % units, g = unit / per_group, k0 = unit % per_group;
    const int h0 = g * d.per + k0 * HU, heads = min(HU, d.per - k0 * HU);
    SsmSegment sg;
    if (!ssm_segment(a, blockIdx.x / units, sg)) return;
    if (STATES && (sg.last || sg.slot < 0)) return;
    const long long out_cols = (long long)d.heads * P;
    if (sg.slot < 0) {
        __nv_bfloat16 *y = (__nv_bfloat16 *)a.y + (long long)h0 * P;
        const int vecs = heads * P / 8;
        for (long long i = tid; i < (sg.t1 - sg.t0) * vecs; i += kThreads)
            *reinterpret_cast<uint4 *>(y + (sg.t0 + i / vecs) * out_cols + (i % vecs) * 8) = make_uint4(0, 0, 0, 0);
        return;
    }
    const int chunks = (int)((sg.t1 - sg.t0 + kL - 1) / kL);
    const int tail = (int)((sg.t1 - sg.t0) - (long long)(chunks - 1) * kL);   // tokens of the last chunk
    const bool partial = chunks > 0 && tail < kL;
    const bool has_z = !STATES && a.z != nullptr;
    const int tpc = STATES ? 2 : has_z ? 4 : 3;        // tiles of a chunk: [C] B X [z]
    const int tB = STATES ? 0 : 1, tX = tB + 1, tZ = 3;

    const uint32_t sbase = tc::smem_u32(sm), bars = sbase + (L::BAR + 7) / 8 * 8;
    auto bar_full = [&](int s) { return bars + 8u * s; };
    auto bar_empty = [&](int s) { return bars + 8u * (kSlots + s); };
    auto bar = [&](int k) { return bars + 8u * (2 * kSlots + k); };
    float *arr = reinterpret_cast<float *>(sm + L::ARR);          // [stage][head][cp, w, e][128]
    float *sums = reinterpret_cast<float *>(sm + L::SUM);         // [stage][head][4]
    float *decs = sums + 2 * HU * 4;                              // [stage][head]
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(sm + L::SLOT);

    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) { tc::mbar_init(bar_full(s), 1); tc::mbar_init(bar_empty(s), 1); }
        const int counts[B_COUNT] = {1, 128, 128, 128, 128, 1, 1, 1, 1, 1, 256, 1, 256, 128, 128, 256, 256, 4, 128, 1};
        for (int k = 0; k < B_COUNT; ++k) tc::mbar_init(bar(k), counts[k]);
        tc::mbar_fence_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(sbase + L::SLOT, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    bool ok = true;
    // bounded waits; a whole warp agrees on the outcome
    auto wait1 = [&](uint32_t b, uint32_t parity) { return ok = ok && tc::mbar_wait(b, parity & 1u, a.wait_ns); };
    auto wait = [&](uint32_t b, uint32_t parity) {
        const bool got = ok && tc::mbar_wait(b, parity & 1u, a.wait_ns);
        return ok = __all_sync(0xffffffffu, got);
    };
    // tile j of chunk c: its slot and how often the slot was used before
    auto slot_of_tile = [&](int c, int j) { return (c * tpc + j) % kSlots; };
    auto use_of_tile = [&](int c, int j) { return (uint32_t)((c * tpc + j) / kSlots); };
    auto tile_addr = [&](int c, int j) { return sbase + L::RING + slot_of_tile(c, j) * kTile; };

    const int wq = warp & 3;                       // TMEM lanes of a warp: 32 wq ..
    const int row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;

    if (warp == 0) {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            int issued = 0;
            for (int c = 0; c < chunks && ok; ++c) {
                const int t = (int)(sg.t0 + (long long)c * kL);
                for (int j = 0; j < tpc; ++j) {
                    const int s = slot_of_tile(c, j);
                    const uint32_t use = use_of_tile(c, j);
                    if (use > 0 && !wait1(bar_empty(s), use - 1)) break;
                    const bool bc = j <= tB;               // C or B
                    const CUtensorMap *m = j == tX ? &maps.x : j == tB ? &maps.b : bc ? &maps.c : &maps.z;
                    const int col = bc ? g * N : h0 * P, boxes = bc ? N / 64 : 2;
                    tc::mbar_arrive_expect_tx(bar_full(s), boxes * kHalfTile);
                    for (int q = 0; q < boxes; ++q)
                        tc::tma_load_2d(tile_addr(c, j) + q * kHalfTile, m, col + q * 64, t, bar_full(s));
                    ++issued;
                }
            }
            if (!ok)                                       // copies in flight land before the CTA ends
                for (int k = max(0, issued - kSlots); k < issued; ++k)
                    tc::mbar_wait(bar_full(k % kSlots), (uint32_t)(k / kSlots) & 1u, a.wait_ns);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- products
        if (lane == 0) {
            constexpr uint32_t id_full = tc::idesc_bf16(128, 128);
            constexpr uint32_t id_px = tc::idesc_bf16(128, P) | tc::kTransB;
            constexpr uint32_t id_ds = tc::idesc_bf16(128, N) | tc::kTransA | tc::kTransB;
            const uint64_t dS = desc_k(sbase + L::S);
            for (int c = 0; c < chunks; ++c) {
                if (!wait1(bar_full(slot_of_tile(c, tB)), use_of_tile(c, tB))) break;
                const uint32_t tb = tile_addr(c, tB);
                if (!STATES) {
                    if (!wait1(bar_full(slot_of_tile(c, 0)), use_of_tile(c, 0))) break;
                    if (partial && c == chunks - 1 && !wait1(bar(B_FIX), 0)) break;
                    tc::fence_after_sync();
                    const uint64_t dC = desc_k(tile_addr(c, 0)), dB = desc_k(tb);
#pragma unroll
                    for (int k = 0; k < N / 16; ++k)
                        tc::mma_bf16(tmem + kColG, dC + step_k(k), dB + step_k(k), id_full, k > 0);
                    tc::mma_commit(bar(B_G));
                    if (!wait1(bar(B_S), c) || (c > 0 && !wait1(bar(B_YE), c - 1))) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int k = 0; k < N / 16; ++k)
                        tc::mma_bf16(tmem + kColY, dC + step_k(k), dS + step_k(k), id_full, k > 0);
                    tc::mma_commit(bar(B_Y2));
                    tc::mma_commit(bar_empty(slot_of_tile(c, 0)));
                } else if (!wait1(bar(B_S), c)) {
                    break;
                }
                const uint64_t dBt = desc_mn(tb);
                for (int e = 0; e < 8; ++e) {
                    const uint32_t use = (uint32_t)(c * 4 + (e >> 1));
                    if (!wait1(bar(B_XF0 + (e & 1)), use)) break;
                    tc::fence_after_sync();
                    const uint32_t xw = sbase + L::XW + (e & 1) * kXwBuf;
#pragma unroll
                    for (int part = 2; part >= 0; --part)      // smallest first
                        tc::mma_bf16(tmem + kColDS, tc::mnmaj_desc(xw + part * kXwPart, 128, 0), dBt + step_mn(e),
                                     id_ds, e > 0 || part < 2);
                    tc::mma_commit(bar(B_XE0 + (e & 1)));
                }
                if (!ok) break;
                tc::mma_commit(bar(B_DS0 + (c & 1)));
                tc::mma_commit(bar_empty(slot_of_tile(c, tB)));
                if (STATES) {
                    tc::mma_commit(bar_empty(slot_of_tile(c, tX)));
                } else {
                    if (!wait1(bar(B_P), c) || !wait1(bar(B_YC), c)) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int hh = 0; hh < HU; ++hh) {
                        const uint64_t dX = desc_mn(tile_addr(c, tX) + hh * kHalfTile);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc::mma_bf16_ta(tmem + kColY + hh * P, tmem + kColG + 32 * (k >> 1) + 16 * hh + 8 * (k & 1),
                                            dX + step_mn(k), id_px, 1);
                    }
                    tc::mma_commit(bar(B_Y));
                }
            }
            tc::mma_commit(bar(B_END));                    // nothing in flight when the CTA ends
            ok = tc::mbar_wait(bar(B_END), 0, a.wait_ns) && ok;
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ y out
        if (!STATES && lane == 0) {
            for (int c = 0; c < chunks; ++c) {
                if (!wait1(bar(B_ST0 + (c & 1)), (uint32_t)(c >> 1))) break;
                if (!(partial && c == chunks - 1)) {
                    for (int q = 0; q < heads * P / 64; ++q)
                        tma_store_2d(&maps.y, tile_addr(c, tX) + q * kHalfTile, h0 * P + q * 64,
                                     (int)(sg.t0 + (long long)c * kL));
                    tc::bulk_commit();
                    tc::bulk_wait_read_all();
                }
                tc::mbar_arrive(bar_empty(slot_of_tile(c, tX)));
                if (has_z) tc::mbar_arrive(bar_empty(slot_of_tile(c, tZ)));
            }
            tc::bulk_wait_all();
        }
    } else if (warp >= 4 && warp < 8) {
        // --------------------------------------------- A: log-decays, G -> P
        float rate[HU], bias[HU];
        double log_sum[HU];
#pragma unroll
        for (int hh = 0; hh < HU; ++hh) {
            const int h = h0 + min(hh, heads - 1);
            rate[hh] = -expf(a.A_log[h]);
            bias[hh] = a.dt_bias ? a.dt_bias[h] : 0.f;
            log_sum[hh] = 0.0;
        }
        const __nv_bfloat16 *pdt = (const __nv_bfloat16 *)a.dt;
        float raw[HU];
        auto fetch = [&](int c) {
            const long long t = sg.t0 + (long long)c * kL + row;
#pragma unroll
            for (int hh = 0; hh < HU; ++hh)
                raw[hh] = t < sg.t1 ? to_f32(pdt[t * a.ld_dt + h0 + min(hh, heads - 1)]) : 0.f;
        };
        if (chunks > 0) fetch(0);
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            const bool valid = sg.t0 + (long long)c * kL + row < sg.t1;
            float pre[HU], suf[HU], dt[HU];
#pragma unroll
            for (int hh = 0; hh < HU; ++hh) {
                dt[hh] = valid && hh < heads ? ssm_dt(raw[hh], bias[hh], d) : 0.f;
                const float lg = valid && hh < heads ? fmaxf(rate[hh] * dt[hh], kMinLog) : 0.f;
                float p = lg, s = lg;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float u = __shfl_up_sync(0xffffffffu, p, o), v = __shfl_down_sync(0xffffffffu, s, o);
                    if (lane >= o) p += u;
                    if (lane + o < 32) s += v;
                }
                if (lane == 31) sums[(st * HU + hh) * 4 + wq] = p;
                pre[hh] = p;
                const float after = __shfl_down_sync(0xffffffffu, s, 1);
                suf[hh] = lane < 31 ? after : 0.f;
            }
            if (c + 1 < chunks) fetch(c + 1);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(B_WG));
            if (!wait(bar(B_WG), c)) break;
            // chunk c - 2 is done with this stage of the arrays (C's part by G of chunk
            // c - 1, which came behind its last product)
            if (c >= 2 && !wait(bar(B_DS0 + st), (uint32_t)(c >> 1) - 1)) break;
            float csl[HU];
#pragma unroll
            for (int hh = 0; hh < HU; ++hh) {
                const float4 ws = load4f(sums + (st * HU + hh) * 4);
                const float w4[4] = {ws.x, ws.y, ws.z, ws.w};
                float before = 0.f, behind = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k < wq) before += w4[k];
                    if (3 - k > wq) behind += w4[3 - k];
                }
                const float cs = pre[hh] + before;
                csl[hh] = cs * kLog2e;
                float *to = arr + ((st * HU + hh) * 3) * 128 + row;
                to[0] = valid ? csl[hh] - log2f(dt[hh]) : __int_as_float(0x7f800000);
                to[128] = valid ? expf(suf[hh] + behind) * dt[hh] : 0.f;
                to[256] = expf(cs);
                if (row == 0) decs[st * HU + hh] = expf(ws.x + ws.y + ws.z + ws.w);
                if (STATES) log_sum[hh] += (double)(ws.x + ws.y) + (double)(ws.z + ws.w);
            }
            tc::mbar_arrive(bar(B_A0 + st));
            if (STATES) continue;
            if (!wait(bar(B_A0 + st), (uint32_t)(c >> 1))) break;
            if (partial && c == chunks - 1) {
                // rows behind the sequence's end: a neighbour's tokens, whatever they hold
                if (!wait(bar_full(slot_of_tile(c, tB)), use_of_tile(c, tB)) ||
                    !wait(bar_full(slot_of_tile(c, tX)), use_of_tile(c, tX)))
                    break;
                if (!valid) {
                    unsigned char *B = sm + L::RING + slot_of_tile(c, tB) * kTile + row * 128;
                    unsigned char *X = sm + L::RING + slot_of_tile(c, tX) * kTile + row * 128;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
#pragma unroll
                        for (int q = 0; q < N / 64; ++q)
                            *reinterpret_cast<uint4 *>(B + q * kHalfTile + k * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            *reinterpret_cast<uint4 *>(X + q * kHalfTile + k * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                tc::fence_async_smem();
                tc::mbar_arrive(bar(B_FIX));
            }
            if (!wait(bar(B_G), c)) break;
            tc::fence_after_sync();
            for (int j = 0; j < 4; ++j) {
                uint32_t p[16];
                if (j > wq) {                              // above the diagonal
#pragma unroll
                    for (int i = 0; i < 16; ++i) p[i] = 0u;
#pragma unroll
                    for (int hh = 0; hh < HU; ++hh) tmem_st16(tmem + lanes + kColG + 32 * j + 16 * hh, p);
                    continue;
                }
                float G[32];
                tc::tmem_ld32(tmem + lanes + kColG + 32 * j, G);
                const int limit = j == wq ? lane : 31;
#pragma unroll
                for (int hh = 0; hh < HU; ++hh) {
                    const float *cp = arr + ((st * HU + hh) * 3) * 128 + 32 * j;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 k = load4f(cp + i);
                        float v[4] = {exp2_fast(csl[hh] - k.x), exp2_fast(csl[hh] - k.y), exp2_fast(csl[hh] - k.z),
                                      exp2_fast(csl[hh] - k.w)};
#pragma unroll
                        for (int q = 0; q < 4; ++q) v[q] = i + q <= limit ? v[q] * G[i + q] : 0.f;
                        p[i / 2] = pack_bf16(v[0], v[1]);
                        p[i / 2 + 1] = pack_bf16(v[2], v[3]);
                    }
                    tmem_st16(tmem + lanes + kColG + 32 * j + 16 * hh, p);
                }
            }
            tmem_wait_st();
            tc::fence_before_sync();
            tc::mbar_arrive(bar(B_P));
        }
        if (STATES && ok && row == 0)
#pragma unroll
            for (int hh = 0; hh < HU; ++hh)
                if (hh < heads) a.seg_log[(long long)sg.entry * d.heads + h0 + hh] = (float)log_sum[hh];
    } else if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------ B: the state
        const int hh = row / P, h = h0 + hh;
        const bool mine = hh < heads;
        const long long head = (long long)N * P, all = head * d.heads, at = (long long)h * head + row % P;
        const float *from = nullptr;
        if (!STATES && mine) {
            if (sg.entry >= 0) from = a.enter + (long long)sg.entry * all + at;
            else if (a.state_in) from = a.state_in + (long long)sg.slot * all + at;
        }
        unsigned char *Srow = sm + L::S + row * 128;
        auto put_row = [&](int j, const float (&v)[32]) {      // columns 32 j .. of this row, bf16
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 u = make_uint4(pack_bf16(v[8 * k], v[8 * k + 1]), pack_bf16(v[8 * k + 2], v[8 * k + 3]),
                                           pack_bf16(v[8 * k + 4], v[8 * k + 5]), pack_bf16(v[8 * k + 6], v[8 * k + 7]));
                const int ch = (j & 1) * 4 + k;
                *reinterpret_cast<uint4 *>(Srow + (j >> 1) * kHalfTile + ((ch ^ (row & 7)) << 4)) = u;
            }
        };
#pragma unroll 1
        for (int j = 0; j < N / 32; ++j) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = from ? from[(long long)(32 * j + i) * P] : 0.f;
            tmem_st32(tmem + lanes + kColS + 32 * j, v);
            if (!STATES) put_row(j, v);
        }
        tmem_wait_st();
        // a chunk's decay is read before its state is announced, so before the products that let A
        // write the next but one there
        float dec = 0.f;
        auto announce = [&](int c) {
            if (c >= chunks) return;
            if (!STATES) tc::fence_async_smem();
            tc::fence_before_sync();
            if (!wait(bar(B_A0 + (c & 1)), (uint32_t)(c >> 1))) return;
            dec = decs[(c & 1) * HU + hh];
            tc::mbar_arrive(bar(B_S));
        };
        announce(0);
        for (int c = 0; c < chunks; ++c) {
            if (!wait(bar(B_DS0 + (c & 1)), (uint32_t)(c >> 1))) break;
            tc::fence_after_sync();
            const bool next = c + 1 < chunks;
#pragma unroll 1
            for (int j = 0; j < N / 32; ++j) {
                float v[32], s[32];
                tc::tmem_ld32(tmem + lanes + kColDS + 32 * j, v);
                tc::tmem_ld32(tmem + lanes + kColS + 32 * j, s);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = fmaf(dec, s[i], v[i]);
                tmem_st32(tmem + lanes + kColS + 32 * j, v);
                // the wait above also says that Y2 of this chunk has read the tile
                if (!STATES && next) put_row(j, v);
            }
            tmem_wait_st();
            announce(c + 1);
        }
        float *to = nullptr;
        if (STATES) to = a.enter + (long long)(sg.entry + 1) * all + at;
        else if (sg.last && a.state_out) to = a.state_out + (long long)sg.slot * all + at;
        if (ok && to && chunks > 0) {
#pragma unroll 1
            for (int j = 0; j < N / 32; ++j) {
                float v[32];
                tc::tmem_ld32(tmem + lanes + kColS + 32 * j, v);
                if (mine)
#pragma unroll
                    for (int i = 0; i < 32; ++i) to[(long long)(32 * j + i) * P] = v[i];
            }
        } else if (ok && to && mine) {                         // no tokens: the state as it came, bit for bit
            for (int i = 0; i < N; ++i) to[(long long)i * P] = from ? from[(long long)i * P] : 0.f;
        }
    } else if (warp >= 12 && warp < 20) {
        // ------------------------------------------------- C: outputs (half = 64 columns)
        if (!STATES) {
            const int half = (warp - 12) >> 2, hh = HU == 2 ? half : 0;
            const bool mine = hh < heads;
            const float skip = a.D && mine ? a.D[h0 + hh] : 0.f;
            const uint32_t ycol = tmem + lanes + kColY + half * 64;
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                if (!wait(bar(B_A0 + st), (uint32_t)(c >> 1)) || !wait(bar(B_Y2), c)) break;
                tc::fence_after_sync();
                const float e = arr[((st * HU + hh) * 3 + 2) * 128 + row];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[32];
                    tc::tmem_ld32(ycol + 32 * j, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= e;
                    tmem_st32(ycol + 32 * j, v);
                }
                tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(bar(B_YC));
                if (!wait(bar_full(slot_of_tile(c, tX)), use_of_tile(c, tX)) ||
                    (has_z && !wait(bar_full(slot_of_tile(c, tZ)), use_of_tile(c, tZ))) || !wait(bar(B_Y), c))
                    break;
                tc::fence_after_sync();
                unsigned char *X = sm + L::RING + slot_of_tile(c, tX) * kTile + half * kHalfTile + row * 128;
                const unsigned char *Z = sm + L::RING + slot_of_tile(c, tZ) * kTile + half * kHalfTile + row * 128;
                const bool short_chunk = partial && c == chunks - 1;
                const bool direct = short_chunk && mine && row < tail;
                __nv_bfloat16 *yrow = (__nv_bfloat16 *)a.y + (sg.t0 + (long long)c * kL + row) * out_cols +
                                      (long long)h0 * P + half * 64;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[32];
                    tc::tmem_ld32(ycol + 32 * j, v);
                    if (j == 1) {
                        tc::fence_before_sync();
                        tc::mbar_arrive(bar(B_YE));
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t off = (uint32_t)(((j * 4 + k) ^ (row & 7)) << 4);
                        const uint4 xv = *reinterpret_cast<const uint4 *>(X + off);
                        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
                        float o[8];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            o[2 * q] = fmaf(skip, bf16_lo(xs[q]), v[8 * k + 2 * q]);
                            o[2 * q + 1] = fmaf(skip, bf16_hi(xs[q]), v[8 * k + 2 * q + 1]);
                        }
                        if (has_z) {
                            const uint4 zv = *reinterpret_cast<const uint4 *>(Z + off);
                            const uint32_t zs[4] = {zv.x, zv.y, zv.z, zv.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                o[2 * q] *= silu_fast(bf16_lo(zs[q]));
                                o[2 * q + 1] *= silu_fast(bf16_hi(zs[q]));
                            }
                        }
                        const uint4 u = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]),
                                                   pack_bf16(o[6], o[7]));
                        if (!short_chunk) *reinterpret_cast<uint4 *>(X + off) = u;
                        else if (direct) *reinterpret_cast<uint4 *>(yrow + j * 32 + k * 8) = u;
                    }
                }
                tc::fence_async_smem();
                tc::mbar_arrive(bar(B_ST0 + st));
            }
        }
    } else if (warp >= 20) {
        // ------------------------------------------------- D: w X in three parts
        // 16 tokens at a time: a thread's token, and two of its 16 blocks of 8 columns
        const int k = (tid & 7) + 8 * ((tid >> 3) & 1), pb0 = (tid - 640) >> 4;
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            if (!wait(bar(B_A0 + st), (uint32_t)(c >> 1)) ||
                !wait(bar_full(slot_of_tile(c, tX)), use_of_tile(c, tX)))
                break;
            const unsigned char *X = sm + L::RING + slot_of_tile(c, tX) * kTile;
            const int count = c == chunks - 1 ? tail : kL;
            for (int e = 0; e < 8; ++e) {
                const int n = c * 8 + e, buf = e & 1;
                if (n >= 2 && !wait(bar(B_XE0 + buf), (uint32_t)((n >> 1) - 1))) break;
                const int tok = e * 16 + k;
                unsigned char *to = sm + L::XW + buf * kXwBuf;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int pb = pb0 + 8 * q;
                    const float w = arr[((st * HU + (HU == 2 ? q : 0)) * 3 + 1) * 128 + tok];
                    uint4 xv = *reinterpret_cast<const uint4 *>(X + q * kHalfTile + tok * 128 + (((pb & 7) ^ (tok & 7)) << 4));
                    if (tok >= count) xv = make_uint4(0, 0, 0, 0);
                    const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
                    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v0 = w * bf16_lo(xs[i]), v1 = w * bf16_hi(xs[i]);
                        hi[i] = pack_bf16(v0, v1);
                        v0 -= bf16_lo(hi[i]); v1 -= bf16_hi(hi[i]);
                        mid[i] = pack_bf16(v0, v1);
                        v0 -= bf16_lo(mid[i]); v1 -= bf16_hi(mid[i]);
                        lo[i] = pack_bf16(v0, v1);
                    }
                    const uint32_t off = tc::mnmaj_off(pb * 8, k, 128);
                    *reinterpret_cast<uint4 *>(to + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(to + kXwPart + off) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                    *reinterpret_cast<uint4 *>(to + 2 * kXwPart + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                tc::fence_async_smem();
                tc::mbar_arrive(bar(B_XF0 + buf));
            }
            if (!ok) break;
        }
    }
    if (!ok) set_error(a.err, GDN_DEVERR_TIMEOUT);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
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

// A [T][width] bf16 view with rows ld elements apart, in boxes of 128 rows x 64 columns.
bool encode(CUtensorMap *m, const void *base, long long ld, long long width, long long T) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)T}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64u, (cuuint32_t)kL}, estr[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, int HU, bool STATES>
cudaError_t run(const SsmScanArgs &a, const SsmMaps &m, unsigned grid, cudaStream_t s) {
    auto kern = ssm_scan_tc_kernel<N, HU, STATES>;
    constexpr int bytes = TcSmem<N, HU>::BYTES;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, bytes, s>>>(a, m);
    return cudaGetLastError();
}

}  // namespace

bool ssm_tc_supported(const SsmDims &d) { return (d.N == 64 || d.N == 128) && (d.P == 64 || d.P == 128); }

int ssm_tc_units(const SsmDims &d) {
    const int hu = 128 / d.P;
    return d.groups * ((d.per + hu - 1) / hu);
}

cudaError_t launch_ssm_scan_tc(const SsmScanArgs &a, bool states, unsigned segments, cudaStream_t s) {
    SsmMaps m;
    const long long hp = (long long)a.d.heads * a.d.P, gn = (long long)a.d.groups * a.d.N;
    if (a.T > 0) {
        if (!encode(&m.x, a.x, a.ld_x, hp, a.T) || !encode(&m.b, a.b, a.ld_bc, gn, a.T) ||
            !encode(&m.c, a.c, a.ld_bc, gn, a.T) || !encode(&m.y, a.y, hp, hp, a.T))
            return cudaErrorInvalidValue;
        if (a.z) {
            if (!encode(&m.z, a.z, a.ld_z, hp, a.T)) return cudaErrorInvalidValue;
        } else {
            m.z = m.x;
        }
    } else {
        memset(&m, 0, sizeof m);       // no tokens: the maps are not used
    }
    const unsigned grid = (unsigned)ssm_tc_units(a.d) * segments;
#define GDN_SSM_TC(N, HU) return states ? run<N, HU, true>(a, m, grid, s) : run<N, HU, false>(a, m, grid, s)
    if (a.d.N == 64) {
        if (a.d.P == 64) GDN_SSM_TC(64, 2);
        GDN_SSM_TC(64, 1);
    }
    if (a.d.P == 64) GDN_SSM_TC(128, 2);
    GDN_SSM_TC(128, 1);
#undef GDN_SSM_TC
}

}  // namespace gdn
