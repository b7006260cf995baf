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
// three bf16 parts (all its 24 bits), smallest first, in a fresh
// accumulator per chunk: the tensor core truncates its sums, which would bias a
// state that it carried along itself.  w comes from a suffix sum of the
// log-decays (exact where it matters, near the chunk's end).  Log-decays are
// clamped at -88 a token, whose exponential is below the least normal number
// and comes out as 0: what a token forgets is the same with the clamp, also
// where it adds nothing, and differences of running sums keep their meaning.
//
// Roles (30 or 32 warps, one CTA per SM): warp 0 loads the tiles of C, B and x by TMA (one slot of
// shared memory, two and two) and has z brought into L2; warp 1 issues G, Y2 and P X, warp 3 dS;
// warp 2 stores y, which takes the place of x in its tile, by TMA; E (a warp per head and chunk
// parity): the log-decays' sums and their exponentials, up to two chunks ahead, and the search for
// values of x that are not finite; A: G -> P, which takes the place of G in TMEM; B: Y2's scaling,
// then the state; C (two groups of 64 columns): the skip, the gate, y; D (two groups, 16 tokens each
// in turn; four where no outputs are computed): the parts of w X.
//
// Bound by the chain of a chunk's steps from Y2 through its scaling and P X to the output's warps,
// about 8,000 cycles, and by the latency of each role's steps between TMEM, registers and shared
// memory (half of the issue slots are used, the tensor cores for a third of the time), not by memory.
// 8,192 tokens of 32 heads, 128 x 128 states, in 4 segments: the states' pass 36 us, the chain of
// states 8 us, the pass with outputs 82 us, 117 us together with early launches, 2.3 TB/s of what has
// to be moved; 16 prompts of 256 to 4,096 tokens, 64 heads of 128 x 64: 384 us, 3.4 TB/s; 65,536
// tokens of 8 heads, 64 x 64: 93 us.  The form of single tokens takes 1,190 us for the first of these.
#include <cuda.h>   // CUtensorMap (the encoder itself is reached through the runtime)

#include <climits>

#include "ssm_common.cuh"
#include "tc_sm103.cuh"

namespace gdn {

namespace {

constexpr int kL = 128;                        // tokens of a chunk
template <int HU> constexpr int kThreads = (28 + 2 * HU) * 32;
constexpr int kSlots = 5;                      // C, two of B, two of X
constexpr int kTile = kL * 128 * 2;            // bytes of a ring slot
constexpr int kHalfTile = kTile / 2;           // 128 rows x 128 bytes: one TMA box
constexpr int kXwPart = 16 * 128 * 2;          // one bf16 part of w X for 16 tokens (MN-major)
constexpr int kXwBuf = 3 * kXwPart;
constexpr float kMinLog = -88.0f;

// TMEM columns
constexpr uint32_t kColS = 0, kColDS = 128, kColY = 256, kColG = 384;

template <int N, int HU> struct TcSmem {
    static constexpr int RING = 0;
    static constexpr int S = RING + kSlots * kTile;          // bf16 state, 128 rows (value columns) x N
    static constexpr int XW = S + N * 256;
    static constexpr int ARR = XW + 2 * kXwBuf;              // [2][HU][5][128]: cs, cp, w, e, v
    static constexpr int DEC = ARR + 2 * HU * 5 * 512;       // [2][HU] chunk decays
    static constexpr int LOG = DEC + 2 * HU * 4;             // [2][HU] doubles: summed log-decays
    static constexpr int BAD = LOG + 2 * HU * 8;             // [128]: first token whose x is not finite
    static constexpr int BAR = BAD + 512;
    static constexpr int NBAR = 2 * kSlots + 29;
    static constexpr int SLOT = (BAR + 7) / 8 * 8 + NBAR * 8;
    static constexpr int BYTES = SLOT + 16;                  // TMEM address, the two flags
    static_assert(BYTES <= 232448, "shared memory of an SM");
};

// Barriers behind the ring's full[] and empty[].
// Where a waiter may be a phase
// behind (G, S, DS, Y, A, ST), even and odd chunks have a barrier each: the next phase of either then
// needs the waiter's own progress.
enum { B_G0 = 0, B_G1, B_P, B_S0, B_S1, B_XF, B_XE = B_XF + 4, B_DS0 = B_XE + 4, B_DS1, B_Y2, B_YC, B_Y0, B_Y1, B_YE, B_A0, B_A1, B_ST0, B_ST1,
       B_CLEAN0, B_CLEAN1, B_FIX, B_END, B_END2, B_COUNT };

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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
           "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16f(uint32_t taddr, const float (&v)[16]) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    tmem_st16(taddr, r);
}
// Two loads of 16 columns behind one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t t0, uint32_t t1, float (&a)[16], float (&b)[16]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t0), "r"(t1) : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) { a[i] = __uint_as_float(r[i]); b[i] = __uint_as_float(r[16 + i]); }
}
// A bounded wait.  Waiting warps share the issue slots and the instruction cache with the working
// ones, so all but the first poll is out of line, a few instructions long, and the wall clock is
// read once in 256 polls.  A wait that ran out sets the CTA's flag: the roles then run on without
// waiting (over their own tiles and rows, with no copy started), the state is not stored, and the
// error is reported.
__device__ __forceinline__ uint32_t poll(uint32_t b, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done) : "r"(b), "r"(parity) : "memory");
    return done;
}
__device__ __forceinline__ uint32_t poll8(uint32_t b, uint32_t parity) {
    uint32_t done;
#define GDN_POLL                                                                   \
    "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"                    \
    "@p bra DONE%=;\n\t"
    asm volatile(
        "{\n\t.reg .pred p;\n\t" GDN_POLL GDN_POLL GDN_POLL GDN_POLL GDN_POLL GDN_POLL GDN_POLL GDN_POLL
        "DONE%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done) : "r"(b), "r"(parity) : "memory");
#undef GDN_POLL
    return done;
}
__device__ __noinline__ void poll_to_limit(uint32_t b, uint32_t parity, uint64_t limit_ns, uint32_t flag) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (poll8(b, parity)) return;
        if ((i & 31u) != 0) continue;
        uint32_t over;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(over) : "r"(flag) : "memory");
        const uint64_t t = tc::globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (over) return;
        if (t - t0 > limit_ns) asm volatile("st.volatile.shared.u32 [%0], 1;" :: "r"(flag) : "memory");
    }
}
// What is in flight when a CTA ends (products, copies into its shared memory) completes by itself
// within microseconds; waited for even after a wait ran out.
__device__ __noinline__ bool poll_in_flight(uint32_t b, uint32_t parity) {
    const uint64_t t0 = tc::globaltimer_ns();
    while (!poll8(b, parity))
        if (tc::globaltimer_ns() - t0 > 100000000ull) return false;
    return true;
}
// Products, commits, copies and arrivals of one lane (`lead`) of a warp that stays together: the
// instructions take their operands from warp-uniform registers, and in a branch of one lane the
// compiler would move every operand there in a loop of its own (several times the product's time).
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
__device__ __forceinline__ void arrive(uint32_t lead, uint32_t b) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}\n"
        :: "r"(b), "r"(lead) : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t lead, uint32_t b, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}\n"
        :: "r"(b), "r"(bytes), "r"(lead) : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t lead, uint32_t dst, const void *tmap, int x, int y, uint32_t b) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}\n"
        :: "r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(b), "r"(lead) : "memory");
}
__device__ __forceinline__ void tma_store(uint32_t lead, const void *tmap, uint32_t src, int x, int y) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n\t}\n"
        :: "l"(tmap), "r"(src), "r"(x), "r"(y), "r"(lead) : "memory");
}
__device__ __forceinline__ void tma_prefetch(uint32_t lead, const void *tmap, int x, int y) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\t"
        "@q cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n\t}\n"
        :: "l"(tmap), "r"(x), "r"(y), "r"(lead) : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ f32x2 bf16_pair(uint32_t v) { return pack2(bf16_lo(v), bf16_hi(v)); }
__device__ __forceinline__ uint32_t pack_bf16(f32x2 v) {
    const float2 f = unpack2(v);
    return pack_bf16(f.x, f.y);
}
// 32 bytes (a memory sector) of a row, in one load where the row starts on 32 bytes.
__device__ __forceinline__ void load_32b(const uint4 *p, bool wide, uint32_t (&v)[8]) {
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(p));
    } else {
        const uint4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}
// The larger one; NaN stays NaN (a decay rate of NaN must not become the clamp).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// v SiLU(z): approximate exp and reciprocal, two values at a time.
__device__ __forceinline__ f32x2 gate2(f32x2 v, f32x2 z) {
    const float2 t = unpack2(mul2(z, pack2(-kLog2e, -kLog2e)));
    const float2 q = unpack2(add2(pack2(exp2_fast(t.x), exp2_fast(t.y)), pack2(1.f, 1.f)));
    return mul2(v, mul2(z, pack2(rcp_fast(q.x), rcp_fast(q.y))));
}

// P X multiplies a token's x with the zeros of the rows in front of it too, where a value that is
// not finite would become NaN.  So x goes into that product with zeros in the places of such
// values, and the outputs of their columns from their tokens on are NaN, as the sums over a state
// of infinities or NaN are.  The search is the log-decay warps', which have time to spare (by the
// output warps it cost 6 %).  A warp looks at 128 tokens by 64 columns of x:
__device__ __forceinline__ bool not_finite(const unsigned char *x, int lane) {
    uint32_t any = 0u;
#pragma unroll 4
    for (int k = 0; k < 32; ++k) {
        const uint4 v = *reinterpret_cast<const uint4 *>(x + (k * 32 + lane) * 16);
        any |= ((v.x & 0x7fff7fffu) + 0x00800080u) | ((v.y & 0x7fff7fffu) + 0x00800080u) |
               ((v.z & 0x7fff7fffu) + 0x00800080u) | ((v.w & 0x7fff7fffu) + 0x00800080u);
    }
    return (any & 0x80008000u) != 0;
}
// ... puts the zeros in, and keeps the first token of each column (rows from `count` on: no tokens)
__device__ __noinline__ void clean(unsigned char *x, int lane, int count, int *from, int token) {
    for (int i = lane; i < count * 64; i += 32) {
        const int row = i >> 6, col = i & 63;
        uint16_t *v = reinterpret_cast<uint16_t *>(x + row * 128 + (((col >> 3) ^ (row & 7)) << 4)) + (col & 7);
        if ((*v & 0x7f80u) != 0x7f80u) continue;
        *v = 0;
        atomicMin(from + col, token + row);
    }
}
// 64 columns of a row of y, in memory or (row & 7 to undo) in a tile
__device__ __noinline__ void spoil(unsigned char *y, int swizzle, const int *from, int token) {
    for (int i = 0; i < 64; ++i)
        if (token >= from[i]) *(reinterpret_cast<uint16_t *>(y + (((i >> 3) ^ swizzle) << 4)) + (i & 7)) = 0x7fff;
}

}  // namespace

// TMEM column of P's tokens 16 j .. 16 j + 15 (8 columns, two tokens each) of a unit's head: in the
// 16 columns that G's tokens 16 j .. had, so that a warp overwrites only what it has read.
__device__ __forceinline__ uint32_t p_col(int j, int hh) { return kColG + 16 * j + 8 * hh; }

struct SsmMaps {
    CUtensorMap x, b, c, z, y;
};

template <int N, int HU, bool STATES>
__global__ void __launch_bounds__(kThreads<HU>, 1)
    ssm_scan_tc_kernel(const __grid_constant__ SsmScanArgs a, const __grid_constant__ SsmMaps maps) {
    using L = TcSmem<N, HU>;
    constexpr int P = 128 / HU;
    static_assert(L::NBAR == 2 * kSlots + B_COUNT, "barriers");
    extern __shared__ __align__(1024) unsigned char sm[];
    const SsmDims &d = a.d;
    // (the shuffles tell the compiler that a value is the same in a whole warp)
    auto uniform = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const int per_group = (d.per + HU - 1) / HU, units = d.groups * per_group;
    const int unit = blockIdx.x % units, g = unit / per_group, k0 = unit % per_group;
    const int h0 = g * d.per + k0 * HU, heads = min(HU, d.per - k0 * HU);
    SsmSegment sg;
    let_next_start();
    const bool run = ssm_segment<STATES>(a, blockIdx.x / units, sg);
    if (!STATES && (!run || sg.slot < 0)) await_previous();
    if (!run) return;
    if (STATES && (sg.last || sg.slot < 0)) return;
    const long long out_cols = (long long)d.heads * P;
    if (sg.slot < 0) {
        __nv_bfloat16 *y = (__nv_bfloat16 *)a.y + (long long)h0 * P;
        const int vecs = heads * P / 8;
        for (long long i = tid; i < (sg.t1 - sg.t0) * vecs; i += kThreads<HU>)
            *reinterpret_cast<uint4 *>(y + (sg.t0 + i / vecs) * out_cols + (i % vecs) * 8) = make_uint4(0, 0, 0, 0);
        return;
    }
    const int first = uniform((int)sg.t0);                         // its first token
    const int chunks = uniform((int)((sg.t1 - sg.t0 + kL - 1) / kL));
    const int tail = uniform((int)(sg.t1 - sg.t0)) - (chunks - 1) * kL;      // tokens of the last chunk
    const bool partial = chunks > 0 && tail < kL;
    const bool has_z = !STATES && a.z != nullptr;
    const bool z_wide = (((uintptr_t)a.z | (uintptr_t)(a.ld_z * 2)) & 31u) == 0;      // rows on 32 bytes

    const uint32_t sbase = tc::smem_u32(sm), bars = sbase + (L::BAR + 7) / 8 * 8;
    auto bar_full = [&](int s) { return bars + 8u * s; };
    auto bar_empty = [&](int s) { return bars + 8u * (kSlots + s); };
    auto bar = [&](int k) { return bars + 8u * (2 * kSlots + k); };
    float *arr = reinterpret_cast<float *>(sm + L::ARR);
    // one of a chunk's arrays (0 cs, 1 cp, 2 w, 3 e, 4 v, see role E), and its decays
    auto array = [&](int st, int hh, int k) { return arr + ((st * HU + hh) * 5 + k) * 128; };
    float *decs = reinterpret_cast<float *>(sm + L::DEC);
    double *logs = reinterpret_cast<double *>(sm + L::LOG);
    int *bad_from = reinterpret_cast<int *>(sm + L::BAD);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(sm + L::SLOT), *gave_up = tmem_slot + 1,
                      *any_bad = tmem_slot + 2;

    if (tid == 0) {
        *gave_up = 0;
        *any_bad = 0;
        for (int s = 0; s < kSlots; ++s) { tc::mbar_init(bar_full(s), 1); tc::mbar_init(bar_empty(s), 1); }
        const int counts[B_COUNT] = {1, 1, 128, 128, 128, 128, 128, 128, 128, 1, 1, 1, 1, 1, 1, 1, 128, 1, 1, 256, HU, HU,
                                     256, 256, HU, HU, 128, 1, 1};
        for (int k = 0; k < B_COUNT; ++k) tc::mbar_init(bar(k), counts[k]);
        tc::mbar_fence_init();
    }
    if (!STATES && tid < 128) bad_from[tid] = INT_MAX;
    if (warp == 1) {
        tc::tmem_alloc(sbase + L::SLOT, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);

    auto wait = [&](uint32_t b, uint32_t parity) {
        if (!poll(b, parity & 1u)) poll_to_limit(b, parity & 1u, a.wait_ns, sbase + L::SLOT + 4);
        __syncwarp();
    };
    // the slots of a chunk's tiles (also their barriers), and the parity of their use
    auto slot_b = [&](int c) { return 1 + (c & 1); };
    auto slot_x = [&](int c) { return 3 + (c & 1); };
    auto half = [&](int c) { return (uint32_t)c >> 1; };
    auto tile = [&](int slot) { return sbase + L::RING + slot * kTile; };
    constexpr int kSlotC = 0;

    // Groups of D's warps, and a buffer of w X for each: without outputs the warps of
    // role C and the slot of tile C serve as well.
    constexpr int kGroups = STATES ? 4 : 2, kFirstD = STATES ? 12 : 20;
    auto xw_buffer = [&](int buf) { return sbase + (buf < 2 ? L::XW + buf * kXwBuf : L::RING + (buf - 2) * kXwBuf); };
    // dS has a second set of columns where there is room for one (without outputs: Y's)
    constexpr bool kTwoDS = STATES || N == 64;
    auto col_ds = [&](int c) { return kTwoDS && (c & 1) ? (N == 64 ? kColDS + 64 : kColY) : kColDS; };
    const int wq = warp & 3;                       // TMEM lanes of a warp: 32 wq ..
    const int row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;

    if (warp == 0) {
        // ------------------------------------------------------------- loads
        const uint32_t lead = elect_lane();
        auto load = [&](int slot, const CUtensorMap *m, int col, int boxes, int t) {
            expect_tx(lead, bar_full(slot), boxes * kHalfTile);
            for (int q = 0; q < boxes; ++q)
                tma_load(lead, tile(slot) + q * kHalfTile, m, col + q * 64, t, bar_full(slot));
        };
        int c = 0;
#pragma unroll 1
        for (; c < chunks && !*gave_up; ++c) {
            const int t = first + c * kL;
            if (c >= 2) wait(bar_empty(slot_b(c)), half(c) - 1);
            if (*gave_up) break;
            load(slot_b(c), &maps.b, g * N, N / 64, t);
            if (!STATES) {
                if (c >= 1) wait(bar_empty(kSlotC), c - 1);
                if (*gave_up) break;
                load(kSlotC, &maps.c, g * N, N / 64, t);
                if (has_z) {                           // z goes straight to registers later: into L2 for now
                    tma_prefetch(lead, &maps.z, h0 * P, t);
                    tma_prefetch(lead, &maps.z, h0 * P + 64, t);
                }
            }
            if (c >= 2) wait(bar_empty(slot_x(c)), half(c) - 1);
            if (*gave_up) break;
            if (c == 0 && (STATES || sg.entry < 0) && (a.lose & LOSE_SSM_TILE_COPY))             // tests only
                expect_tx(lead, bar_full(slot_x(c)), kTile);
            else load(slot_x(c), &maps.x, h0 * P, 2, t);
        }
        // copies in flight land before the CTA ends (a slot whose last copy was not started runs out)
        if (*gave_up) {
            for (int k = max(0, c - 2); k <= min(c, chunks - 1); ++k) {
                poll_in_flight(bar_full(slot_b(k)), half(k) & 1u);
                if (!STATES) poll_in_flight(bar_full(kSlotC), k & 1u);
                poll_in_flight(bar_full(slot_x(k)), half(k) & 1u);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------- products: G, Y2, P X
        if (!STATES) {
            const uint32_t lead = elect_lane();
            constexpr uint32_t id_full = tc::idesc_bf16(128, 128);
            constexpr uint32_t id_px = tc::idesc_bf16(128, P) | tc::kTransB;
            const uint64_t dS = desc_k(sbase + L::S), dC = desc_k(tile(kSlotC));
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                wait(bar_full(kSlotC), c);
                wait(bar_full(slot_b(c)), half(c));
                if (partial && c == chunks - 1) wait(bar(B_FIX), 0);
                tc::fence_after_sync();
                const uint64_t dB = desc_k(tile(slot_b(c)));
#pragma unroll
                for (int k = 0; k < N / 16; ++k) mma_ss(lead, tmem + kColG, dC + step_k(k), dB + step_k(k), id_full, k > 0);
                commit(lead, bar(B_G0 + (c & 1)));
                wait(bar(B_S0 + (c & 1)), half(c));
                if (c > 0) wait(bar(B_YE), c - 1);
                tc::fence_after_sync();
#pragma unroll
                for (int k = 0; k < N / 16; ++k) mma_ss(lead, tmem + kColY, dC + step_k(k), dS + step_k(k), id_full, k > 0);
                commit(lead, bar(B_Y2));
                commit(lead, bar_empty(kSlotC));
                wait(bar_full(slot_x(c)), half(c));
                wait(bar(B_CLEAN0 + (c & 1)), half(c));
                wait(bar(B_YC), c);
                wait(bar(B_P), c);
                tc::fence_after_sync();
#pragma unroll
                for (int hh = 0; hh < HU; ++hh) {
                    const uint64_t dX = desc_mn(tile(slot_x(c)) + hh * kHalfTile);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_ts(lead, tmem + kColY + hh * P, tmem + p_col(k, hh), dX + step_mn(k), id_px, 1);
                }
                commit(lead, bar(B_Y0 + (c & 1)));
            }
            commit(lead, bar(B_END));                      // nothing in flight when the CTA ends
            if (!poll_in_flight(bar(B_END), 0)) *gave_up = 1;
        }
    } else if (warp == 3) {
        // -------------------------------------------------------- product: dS
        const uint32_t lead = elect_lane();
        constexpr uint32_t id_ds = tc::idesc_bf16(128, N) | tc::kTransA | tc::kTransB;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            wait(bar_full(slot_b(c)), half(c));
            if (partial && c == chunks - 1) wait(bar(B_FIX), 0);
            // dS(c)'s columns are free: of the chunk before, or with two sets the one before that
            if (!kTwoDS) wait(bar(B_S0 + (c & 1)), half(c));
            else if (c >= 1) wait(bar(B_S0 + ((c - 1) & 1)), half(c - 1));
            const uint64_t dBt = desc_mn(tile(slot_b(c)));
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                const int buf = e % kGroups;
                wait(bar(B_XF + buf), (uint32_t)(c * (8 / kGroups) + e / kGroups));
                tc::fence_after_sync();
                const uint64_t dW = tc::mnmaj_desc(xw_buffer(buf), 128, 0);
#pragma unroll
                for (int part = 2; part >= 0; --part)      // smallest first
                    mma_ss(lead, tmem + col_ds(c), dW + part * (kXwPart >> 4), dBt + step_mn(e), id_ds, e > 0 || part < 2);
                commit(lead, bar(B_XE + buf));
            }
            if (!STATES) wait(bar(B_G0 + (c & 1)), half(c));   // G has read B too before the slot is given back
            commit(lead, bar(B_DS0 + (c & 1)));
            commit(lead, bar_empty(slot_b(c)));
            if (STATES) commit(lead, bar_empty(slot_x(c)));
        }
        commit(lead, bar(B_END2));
        if (!poll_in_flight(bar(B_END2), 0)) *gave_up = 1;
    } else if (warp == 2) {
        // ------------------------------------------------------------ y out
        if (!STATES) {
            const uint32_t lead = elect_lane();
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                wait(bar(B_ST0 + (c & 1)), half(c));
                if (!(partial && c == chunks - 1) && !*gave_up) {
                    for (int q = 0; q < heads * P / 64; ++q)
                        tma_store(lead, &maps.y, tile(slot_x(c)) + q * kHalfTile, h0 * P + q * 64, first + c * kL);
                    tc::bulk_commit();                     // (empty groups in the other lanes)
                    tc::bulk_wait_read_all();
                }
                __syncwarp();
                arrive(lead, bar_empty(slot_x(c)));
            }
            tc::bulk_wait_all();
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------- A: G -> P
        if (!STATES) {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                if (partial && c == chunks - 1) {
                    // rows behind the sequence's end: a neighbour's tokens, whatever they hold
                    wait(bar_full(slot_b(c)), half(c));
                    wait(bar_full(slot_x(c)), half(c));
                    if (row >= tail) {
                        unsigned char *B = sm + L::RING + slot_b(c) * kTile + row * 128;
                        unsigned char *X = sm + L::RING + slot_x(c) * kTile + row * 128;
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
                wait(bar(B_A0 + st), half(c));
                wait(bar(B_G0 + st), half(c));
                tc::fence_after_sync();
                // Tokens i in front of this warp's rows, 16 at a time: exp(cs_r - cs_i) dt_i is
                // exp(cs_r - cs of the 16's last) v_i, both factors' exponents below zero.
#pragma unroll 1
                for (int j = 0; j < 2 * wq; ++j) {
                    float G[16];
                    tc::tmem_ld16(tmem + lanes + kColG + 16 * j, G);
#pragma unroll
                    for (int hh = 0; hh < HU; ++hh) {
                        const float *cs = array(st, hh, 0), *v = array(st, hh, 4) + 16 * j;
                        const float u = exp2_fast(cs[row] - cs[16 * j + 15]);
                        const f32x2 u2 = pack2(u, u);
                        uint32_t p[8];
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(v + i);
                            p[i / 2] = pack_bf16(mul2(mul2(pack2(G[i], G[i + 1]), k.x), u2));
                            p[i / 2 + 1] = pack_bf16(mul2(mul2(pack2(G[i + 2], G[i + 3]), k.y), u2));
                        }
                        tmem_st8(tmem + lanes + p_col(j, hh), p);
                    }
                }
                // Tokens beside the rows: exponents of their own.  What is above the diagonal, finite or
                // not, is left out of the product's result.
#pragma unroll 1
                for (int j = 2 * wq; j < 2 * wq + 2; ++j) {
                    float G[16];
                    tc::tmem_ld16(tmem + lanes + kColG + 16 * j, G);
#pragma unroll
                    for (int hh = 0; hh < HU; ++hh) {
                        const float csr = array(st, hh, 0)[row];
                        const f32x2 cs = pack2(csr, csr);
                        const float *cp = array(st, hh, 1) + 16 * j;
                        uint32_t p[8];
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(cp + i);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const int n = i + 2 * q;
                                const float2 u = unpack2(add2(cs, q ? k.y : k.x));
                                const float2 v = unpack2(mul2(pack2(exp2_fast(u.x), exp2_fast(u.y)), pack2(G[n], G[n + 1])));
                                p[n / 2] = pack_bf16(16 * j + n <= row ? v.x : 0.f, 16 * j + n + 1 <= row ? v.y : 0.f);
                            }
                        }
                        tmem_st8(tmem + lanes + p_col(j, hh), p);
                    }
                }
                const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll 1
                for (int j = 2 * wq + 2; j < 8; ++j)                      // above the diagonal
#pragma unroll 1
                    for (int hh = 0; hh < HU; ++hh) tmem_st8(tmem + lanes + p_col(j, hh), zero);
                tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(bar(B_P));
            }
        }
    } else if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------ B: the state
        const int hh = row / P, h = h0 + hh;
        const bool mine = hh < heads;
        const long long head = (long long)N * P, all = head * d.heads, at = (long long)h * head + row % P;
        const float *from = nullptr;
        if (!STATES && sg.entry >= 0) await_previous();        // the state that enters the segment
        if (!STATES && mine) {
            if (sg.entry >= 0) from = a.enter + (long long)sg.entry * all + at;
            else if (a.state_in) from = a.state_in + (long long)sg.slot * all + at;
        }
        unsigned char *Srow = sm + L::S + row * 128;
        auto put_row = [&](int j, const float (&v)[16]) {      // columns 16 j .. of this row, bf16
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 u = make_uint4(pack_bf16(v[8 * k], v[8 * k + 1]), pack_bf16(v[8 * k + 2], v[8 * k + 3]),
                                           pack_bf16(v[8 * k + 4], v[8 * k + 5]), pack_bf16(v[8 * k + 6], v[8 * k + 7]));
                const int ch = (j & 3) * 2 + k;
                *reinterpret_cast<uint4 *>(Srow + (j >> 2) * kHalfTile + ((ch ^ (row & 7)) << 4)) = u;
            }
        };
#pragma unroll 1
        for (int j = 0; j < N / 16; ++j) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = from ? from[(long long)(16 * j + i) * P] : 0.f;
            tmem_st16f(tmem + lanes + kColS + 16 * j, v);
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
            wait(bar(B_A0 + (c & 1)), half(c));
            dec = decs[(c & 1) * HU + hh];
            tc::mbar_arrive(bar(B_S0 + (c & 1)));
        };
        announce(0);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            if (!STATES) {
                // Y2 of this chunk times exp(cs): row r of the chunk on this thread
                wait(bar(B_Y2), c);
                tc::fence_after_sync();
#pragma unroll 1
                for (int j = 0; j < 8; ++j) {
                    const float e = array(c & 1, HU == 2 ? j >> 2 : 0, 3)[row];
                    const f32x2 e2 = pack2(e, e);
                    float v[16];
                    tc::tmem_ld16(tmem + lanes + kColY + 16 * j, v);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 u = unpack2(mul2(pack2(v[i], v[i + 1]), e2));
                        v[i] = u.x;
                        v[i + 1] = u.y;
                    }
                    tmem_st16f(tmem + lanes + kColY + 16 * j, v);
                }
                tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(bar(B_YC));
            }
            wait(bar(B_DS0 + (c & 1)), half(c));
            tc::fence_after_sync();
            const bool next = c + 1 < chunks;
#pragma unroll 1
            for (int j = 0; j < N / 16; ++j) {
                float v[16], s[16];
                tmem_ld16x2(tmem + lanes + col_ds(c) + 16 * j, tmem + lanes + kColS + 16 * j, v, s);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = fmaf(dec, s[i], v[i]);
                tmem_st16f(tmem + lanes + kColS + 16 * j, v);
                if (!STATES && next) put_row(j, v);            // Y2 of this chunk has read the tile
            }
            tmem_wait_st();
            announce(c + 1);
        }
        float *to = nullptr;
        if (STATES) to = a.enter + (long long)(sg.entry + 1) * all + at;
        else if (sg.last && a.state_out) to = a.state_out + (long long)sg.slot * all + at;
        // a segment in front of this one whose state was not computed: its log-decay is +inf
        bool lost = false;
        if (!STATES && to && mine) {
            for (int k = sg.entry - sg.index + lane; k < sg.entry; k += 32)
                lost |= a.seg_log[(long long)k * d.heads + h] > 0.f;
            lost = __any_sync(0xffffffffu, lost);              // (a warp's rows are of one head)
        }
        if (*gave_up || lost) to = nullptr;
        if (to && chunks > 0) {
#pragma unroll 1
            for (int j = 0; j < N / 16; ++j) {
                float v[16];
                tc::tmem_ld16(tmem + lanes + kColS + 16 * j, v);
                if (mine)
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[(long long)(16 * j + i) * P] = v[i];
            }
        } else if (to && mine) {                         // no tokens: the state as it came, bit for bit
            for (int i = 0; i < N; ++i) to[(long long)i * P] = from ? from[(long long)i * P] : 0.f;
        }
    } else if (warp >= 12 && warp < kFirstD) {
        // ------------------------------------------------- C: outputs (side = 64 columns)
        if (!STATES) {
            const int side = (warp - 12) >> 2, hh = HU == 2 ? side : 0;
            const bool mine = hh < heads;
            const float skip = a.D && mine ? a.D[h0 + hh] : 0.f;
            const f32x2 skip2 = pack2(skip, skip);
            const uint32_t ycol = tmem + lanes + kColY + side * 64;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const int st = c & 1;
                const bool short_chunk = partial && c == chunks - 1;
                const bool live = mine && !(short_chunk && row >= tail);
                const long long t = sg.t0 + (long long)c * kL + row;
                const uint4 *zrow = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.z + t * a.ld_z +
                                                                    (long long)h0 * P + side * 64);
                uint32_t zn[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};   // z of the next 16 columns
                if (has_z && live) load_32b(zrow, z_wide, zn);
                wait(bar_full(slot_x(c)), half(c));
                unsigned char *X = sm + L::RING + slot_x(c) * kTile + side * kHalfTile + row * 128;
                wait(bar(B_DS0 + st), half(c));            // D has read the tile that y replaces
                wait(bar(B_Y0 + st), half(c));
                tc::fence_after_sync();
                __nv_bfloat16 *yrow = (__nv_bfloat16 *)a.y + t * out_cols + (long long)h0 * P + side * 64;
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    float v[16];
                    tc::tmem_ld16(ycol + 16 * j, v);
                    if (j == 3) {
                        tc::fence_before_sync();
                        tc::mbar_arrive(bar(B_YE));
                    }
                    uint32_t zc[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) zc[k] = zn[k];
                    if (has_z && live && j < 3) load_32b(zrow + 2 * j + 2, z_wide, zn);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t off = (uint32_t)(((j * 2 + k) ^ (row & 7)) << 4);
                        const uint4 xv = *reinterpret_cast<const uint4 *>(X + off);
                        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
                        f32x2 o[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            o[q] = fma2(skip2, bf16_pair(xs[q]), pack2(v[8 * k + 2 * q], v[8 * k + 2 * q + 1]));
                        if (has_z) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) o[q] = gate2(o[q], bf16_pair(zc[4 * k + q]));
                        }
                        const uint4 u = make_uint4(pack_bf16(o[0]), pack_bf16(o[1]), pack_bf16(o[2]), pack_bf16(o[3]));
                        if (!short_chunk) *reinterpret_cast<uint4 *>(X + off) = u;
                        else if (live) *reinterpret_cast<uint4 *>(yrow + j * 16 + k * 8) = u;
                    }
                }
                if (*any_bad && (live || !short_chunk))
                    spoil(short_chunk ? (unsigned char *)yrow : X, short_chunk ? 0 : row & 7, bad_from + side * 64, c * kL + row);
                tc::fence_async_smem();
                tc::mbar_arrive(bar(B_ST0 + st));
            }
        }
    } else if (warp >= kFirstD && warp < 28) {
        // ------------------------------------------------- D: w X in three parts
        // Group b takes every kGroups-th sixteen of tokens: a thread's token, and two of its 16
        // blocks of 8 columns.  Each part is the next 8 bits of the value, cut off: the three hold
        // all 24.
        const int t128 = (tid - kFirstD * 32) & 127, buf = uniform((tid - kFirstD * 32) >> 7);
        const int k = (t128 & 7) + 8 * ((t128 >> 3) & 1), pb0 = t128 >> 4;
        unsigned char *to = sm + (xw_buffer(buf) - sbase);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            wait(bar(B_A0 + st), half(c));
            wait(bar_full(slot_x(c)), half(c));
            const unsigned char *X = sm + L::RING + slot_x(c) * kTile;
            const int count = c == chunks - 1 ? tail : kL;
#pragma unroll 1
            for (int e = buf; e < 8; e += kGroups) {
                const int tok = e * 16 + k, n = c * (8 / kGroups) + e / kGroups;
                uint4 xv[2];
                float w[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    w[q] = array(st, HU == 2 ? q : 0, 2)[tok];
                    xv[q] = *reinterpret_cast<const uint4 *>(X + q * kHalfTile + tok * 128 + ((pb0 ^ (tok & 7)) << 4));
                    if (tok >= count) xv[q] = make_uint4(0, 0, 0, 0);
                }
                if (n >= 1) wait(bar(B_XE + buf), (uint32_t)(n - 1));
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t xs[4] = {xv[q].x, xv[q].y, xv[q].z, xv[q].w};
                    uint32_t part[3][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f32x2 v = mul2(pack2(w[q], w[q]), bf16_pair(xs[i]));
#pragma unroll
                        for (int r = 0; r < 3; ++r) {
                            const float2 f = unpack2(v);
                            const uint32_t f0 = __float_as_uint(f.x), f1 = __float_as_uint(f.y);
                            part[r][i] = __byte_perm(f0, f1, 0x7632);
                            if (r < 2) v = add2(v, pack2(-bf16_hi(f0), -bf16_hi(f1)));
                        }
                    }
                    const uint32_t off = tc::mnmaj_off((pb0 + 8 * q) * 8, k, 128);
#pragma unroll
                    for (int r = 0; r < 3; ++r)
                        *reinterpret_cast<uint4 *>(to + r * kXwPart + off) =
                            make_uint4(part[r][0], part[r][1], part[r][2], part[r][3]);
                }
                tc::fence_async_smem();
                tc::mbar_arrive(bar(B_XF + buf));
            }
        }
    } else if (warp >= 28) {
        // ------------ E: log-decays of one head in every other chunk, four tokens a lane
        // cs_i summed from the chunk's start, in powers of two; cp_i = log2(dt_i) - cs_i; w_i from
        // the sum behind i; e_i = exp(cs_i); v_i = dt_i exp(cs of the last of i's 16 - cs_i); the
        // chunk's decay.  Tokens behind the end: no weight.
        const int st = (warp - 28) / HU, hh = (warp - 28) % HU;
        const bool mine = hh < heads;
        const int h = h0 + min(hh, heads - 1);
        const float rate = -expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
        const __nv_bfloat16 *pdt = (const __nv_bfloat16 *)a.dt + h;
        double log_sum = 0.0;
        float raw[4];
        auto fetch = [&](int c) {
            const long long t = sg.t0 + (long long)c * kL + 4 * lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i] = t + i < sg.t1 ? to_f32(pdt[(t + i) * a.ld_dt]) : 0.f;
        };
        if (st < chunks) fetch(st);
#pragma unroll 1
        for (int c = st; c < chunks; c += 2) {
            const int count = c == chunks - 1 ? tail : kL;
            float dt[4], g[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool valid = 4 * lane + i < count && mine;
                dt[i] = valid ? ssm_dt(raw[i], bias, d) : 0.f;
                g[i] = valid ? max_nan(rate * dt[i], kMinLog) : 0.f;
            }
            if (c + 2 < chunks) fetch(c + 2);
            const float sum = (g[0] + g[1]) + (g[2] + g[3]);
            float pre = sum, suf = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, pre, o), v = __shfl_down_sync(0xffffffffu, suf, o);
                if (lane >= o) pre += u;
                if (lane + o < 32) suf += v;
            }
            const float total = __shfl_sync(0xffffffffu, pre, 31);
            float before = __shfl_up_sync(0xffffffffu, pre, 1), behind = __shfl_down_sync(0xffffffffu, suf, 1);
            if (lane == 0) before = 0.f;
            if (lane == 31) behind = 0.f;
            float cs[4], cp[4], w[4], e[4], v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                before += g[i];
                cs[i] = before * kLog2e;
                e[i] = exp2_fast(cs[i]);
                cp[i] = 4 * lane + i < count ? __log2f(dt[i]) - cs[i] : -__int_as_float(0x7f800000);
            }
            const float last = __shfl_sync(0xffffffffu, cs[3], lane | 3);
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                v[i] = exp2_fast(last - cs[i]) * dt[i];
                w[i] = exp2_fast(behind * kLog2e) * dt[i];
                behind += g[i];
            }
            if (STATES && lane == 0) log_sum += (double)total;

            // chunk c - 2 is done with these arrays: its decay was read before its dS, w before dS was
            // done, cp and e before its last product
            if (c >= 2) {
                wait(bar(B_DS0 + st), half(c) - 1);
                if (!STATES) wait(bar(B_Y0 + st), half(c) - 1);
                if (kTwoDS) wait(bar(B_S0 + st), half(c) - 1);      // (else implied by its dS)
            }
            store4f(array(st, hh, 0) + 4 * lane, make_float4(cs[0], cs[1], cs[2], cs[3]));
            store4f(array(st, hh, 1) + 4 * lane, make_float4(cp[0], cp[1], cp[2], cp[3]));
            store4f(array(st, hh, 2) + 4 * lane, make_float4(w[0], w[1], w[2], w[3]));
            store4f(array(st, hh, 3) + 4 * lane, make_float4(e[0], e[1], e[2], e[3]));
            store4f(array(st, hh, 4) + 4 * lane, make_float4(v[0], v[1], v[2], v[3]));
            if (lane == 0) decs[st * HU + hh] = exp2_fast(total * kLog2e);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(bar(B_A0 + st));
            if (!STATES) {
                wait(bar_full(slot_x(c)), half(c));
                const int q0 = HU == 2 ? hh : 0, q1 = HU == 2 ? hh + 1 : 2;      // its head's 64 columns, or 128
#pragma unroll 1
                for (int q = q0; q < q1; ++q) {
                    unsigned char *X = sm + L::RING + slot_x(c) * kTile + q * kHalfTile;
                    if (!__any_sync(0xffffffffu, not_finite(X, lane))) continue;
                    wait(bar(B_DS0 + st), half(c));        // (D reads x as it is)
                    clean(X, lane, count, bad_from + q * 64, c * kL);
                    *any_bad = 1;
                    tc::fence_async_smem();
                    __syncwarp();
                }
                arrive(lane == 0, bar(B_CLEAN0 + st));
            }
        }
        if (STATES && lane == 0) logs[st * HU + hh] = log_sum;
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (!STATES) await_previous();
    if (tid == 0 && *gave_up) set_error(a.err, GDN_DEVERR_TIMEOUT);
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
    if (STATES && tid < heads)
        a.seg_log[(long long)sg.entry * d.heads + h0 + tid] =
            *gave_up ? __int_as_float(0x7f800000) : (float)(logs[tid] + logs[HU + tid]);
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
    if (!STATES && a.seg_len < a.T) return launch_early(kern, dim3(grid), kThreads<HU>, bytes, s, a, m);
    kern<<<grid, kThreads<HU>, bytes, s>>>(a, m);
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
    if (!encode(&m.x, a.x, a.ld_x, hp, a.T) || !encode(&m.b, a.b, a.ld_bc, gn, a.T) ||
        !encode(&m.c, a.c, a.ld_bc, gn, a.T) || !encode(&m.y, a.y, hp, hp, a.T))
        return cudaErrorInvalidValue;
    if (a.z) {
        if (!encode(&m.z, a.z, a.ld_z, hp, a.T)) return cudaErrorInvalidValue;
    } else {
        m.z = m.x;
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
