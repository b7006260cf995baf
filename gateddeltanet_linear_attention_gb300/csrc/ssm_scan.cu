// ssm_scan.cu -- the selective state space scan over packed prompts: the fp32
// kernel that serves every size and type, and the cutting of long sequences
// into segments that run side by side.
//
// Per head (B, C of its group), with a_t = exp(A dt_t), A = -exp(A_log):
//   S_t[n][p] = a_t S_{t-1}[n][p] + dt_t B_t[n] x_t[p]
//   y_t[p]    = (sum_n C_t[n] S_t[n][p] + D x_t[p]) SiLU(z_t[p])
//
// Segments: the map from a segment's entering state to its leaving one is
// S -> exp(sum of its log-decays) S + E, E being the leaving state from zero.
// So a first pass computes every segment's E and summed log-decay at once, a
// short second one chains them, and the last one runs all segments with
// outputs, each from the state that enters it.
#include <climits>

#include "ssm_common.cuh"

namespace gdn {

namespace {

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// ------------------------------------------------------------- segment map
// seg_base and enter_base: exclusive scans over the sequences of their segments
// (one at least) and of the entering states that are kept (none for a sequence
// of one segment).  Sequences whose entries would not fit (lengths that sum to
// more than T: malformed cu_seqlens) get no segment and are reported.
__global__ void __launch_bounds__(1024) ssm_segment_map_kernel(SsmScanArgs a) {
    __shared__ long long ws_seg[32], ws_ent[32];   // 64 bits: malformed lengths may sum to any size
    __shared__ long long run_seg, run_ent;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long max_seg = (long long)a.n_seqs + a.max_enter / 2, max_ent = a.max_enter;
    if (tid == 0) run_seg = run_ent = 0;
    __syncthreads();
    for (int n0 = 0; n0 < a.n_seqs; n0 += 1024) {
        const int n = n0 + tid;
        long long seg = 0, ent = 0;
        if (n < a.n_seqs) {
            long long s, e;
            seq_bounds(a.cu, n, a.T, a.err, s, e);
            seg = e > s ? (e - s + a.seg_len - 1) / a.seg_len : 1;
            ent = seg > 1 ? seg : 0;
        }
        auto scan = [&](long long v) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            return v;
        };
        const long long is = scan(seg), ie = scan(ent);
        if (lane == 31) { ws_seg[warp] = is; ws_ent[warp] = ie; }
        __syncthreads();
        if (warp == 0) {
            const long long vs = scan(ws_seg[lane]), ve = scan(ws_ent[lane]);
            ws_seg[lane] = vs;
            ws_ent[lane] = ve;
        }
        __syncthreads();
        const long long bs = run_seg + (warp ? ws_seg[warp - 1] : 0) + is - seg;
        const long long be = run_ent + (warp ? ws_ent[warp - 1] : 0) + ie - ent;
        if (n < a.n_seqs) {
            if (be + ent > max_ent) set_error(a.err, GDN_DEVERR_CU_SEQLENS);
            a.seg_base[n] = (int)(bs < max_seg ? bs : max_seg);
            a.enter_base[n] = (int)(be < max_ent ? be : max_ent);
        }
        __syncthreads();
        if (tid == 0) {
            run_seg += ws_seg[31];
            run_ent += ws_ent[31];
        }
        __syncthreads();
    }
    if (tid == 0) {
        a.seg_base[a.n_seqs] = (int)(run_seg < max_seg ? run_seg : max_seg);
        a.enter_base[a.n_seqs] = (int)(run_ent < max_ent ? run_ent : max_ent);
    }
}

// ------------------------------------------------------------ chained states
// enter[0] = the initial state, enter[k+1] = exp(log-decay of segment k) *
// enter[k] + (what pass 1 left in enter[k+1]); one thread per float4 of a head.
// The loads of kAhead segments are in flight at once: only the multiply-adds
// form a chain.  Bound by latency: 32 heads of 128 x 128 in 4 segments 8 us alone,
// 17 MB from L2, most of it behind the pass in front of it.
__global__ void __launch_bounds__(256) ssm_chain_states_kernel(SsmScanArgs a) {
    constexpr int kAhead = 8;
    let_next_start();
    const int h = blockIdx.x, vec = a.d.N * a.d.P / 4, lane = threadIdx.x & 31;
    const int i = blockIdx.y * 256 + threadIdx.x;
    const long long head = (long long)a.d.N * a.d.P, all = head * a.d.heads;
    const bool small = a.n_seqs <= kWarpSeqs;
    SsmCut mine{0, 0, -1};
    if (small) mine = ssm_warp_cut(a, lane);
    await_previous();
    // The sequences of two segments or more in turn: of a small batch all at once in the lanes, every
    // gridDim.z-th of them this CTA's; of a larger one 32 of this CTA's own at a time.
    unsigned cut = __ballot_sync(0xffffffffu, small && mine.segs > 1);
    const int stride = gridDim.z;
    int next = small ? a.n_seqs : blockIdx.z, first = 0, turn = 0;
    for (;;) {
        if (cut == 0) {
            if (next >= a.n_seqs) break;
            first = next;
            const int n = first + lane * stride;
            if (n < a.n_seqs) {
                mine.entry0 = a.enter_base[n];
                mine.segs = a.seg_base[n + 1] - a.seg_base[n];
            }
            cut = __ballot_sync(0xffffffffu, n < a.n_seqs && mine.segs > 1);
            next = a.n_seqs - first > 32 * stride ? first + 32 * stride : a.n_seqs;
            continue;
        }
        const int k = __ffs(cut) - 1, n = small ? k : first + k * stride;
        cut &= cut - 1;
        if (small && turn++ % gridDim.z != blockIdx.z) continue;
        const int e0 = __shfl_sync(0xffffffffu, mine.entry0, k), segs = __shfl_sync(0xffffffffu, mine.segs, k);
        if (e0 + segs > a.max_enter) continue;                 // (too many: malformed, reported)
        const int slot = slot_of(a.state_idx, n, a.d.n_slots, a.err);
        if (slot < 0 || i >= vec) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.state_in) v = load4f(a.state_in + (long long)slot * all + h * head + 4 * i);
        float *at = a.enter + (long long)e0 * all + h * head + 4 * i;
        store4f(at, v);
        for (int k0 = 1; k0 < segs; k0 += kAhead) {
            float4 u[kAhead];
            float g[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (k0 + k < segs) {
                    u[k] = load4f(at + (k0 + k) * all);
                    g[k] = a.seg_log[(long long)(e0 + k0 + k - 1) * a.d.heads + h];
                }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (k0 + k < segs) {
                    const float f = expf(g[k]);
                    v = make_float4(fmaf(f, v.x, u[k].x), fmaf(f, v.y, u[k].y), fmaf(f, v.z, u[k].z), fmaf(f, v.w, u[k].w));
                    store4f(at + (k0 + k) * all, v);
                }
        }
    }
}

// ----------------------------------------------------------------- the scan
// One CTA walks the tokens of one (segment, head) with the head's N x P fp32
// state in registers: a thread owns 4 columns p and NPT rows n, packed in pairs
// of n so that one packed multiply-add serves two state elements.  Tokens come
// in blocks of TB through shared memory, the next block's loads in flight
// while this one is computed; the row slices' parts of y are summed per block.
// Bound by the fp32 units, 3 packed operations per two state elements and token, where the batch
// fills the GPU (256 sequences of 512 tokens, 8 heads of 64 x 64: 784 us, 44 % of their rate; 8,192
// tokens of 32 heads, 128 x 128, cut: 1,227 us), and by a token's latency, 225 ns, where it does not
// (7 sequences of up to 256 tokens: 57 us).
// STATES: pass 1, no outputs: the leaving state from zero and the log-decay.
// WIDE: 4 to 16 rows a thread, as many threads as 256 allow, for batches that do not fill the GPU.
// ALONE: the same with 128 registers a thread, for batches of up to two CTAs or so an SM, where loads
// further ahead are worth more than a third CTA.
enum { WHOLE, WIDE, ALONE };
template <int N, int P, int SHAPE> struct ScanShape {
    static constexpr int MOST = SHAPE != WHOLE ? N * P / 1024 : N * P / 128;
    static constexpr int NPT = MOST >= 16 ? 16 : MOST < 4 ? 4 : MOST;  // rows of a thread
    static constexpr int LP = P / 4;                                   // threads across the columns
    static constexpr int NS = N / NPT;                                 // row slices
    static constexpr int NT = LP * NS;
    // CTAs that an SM's registers are to hold (0: as many as it comes to).  128 x 128 states whole: two,
    // 100 sequences of 512 tokens, 16 heads, 1,951 us, and 2,217 with the one that it came to; smaller
    // ones spill for it (256 sequences of 512 tokens, 8 heads of 64 x 64: 784 us, with eight 937).
    static constexpr int RESIDENT = SHAPE == ALONE || NT == 256 && SHAPE == WHOLE ? 512 / NT : 0;
    static constexpr int TB = 8;
    static constexpr int ROW = P + 2 * N;                              // x | B | C of a token
    static constexpr int VPT = (TB * ROW / 4 + NT - 1) / NT;           // vectors of a thread
    static constexpr int OPT = (TB * LP + NT - 1) / NT;                // output (and z) vectors of a thread
};
template <typename TA> struct Vec4Of { using type = float4; };
template <> struct Vec4Of<__nv_bfloat16> { using type = uint2; };
__device__ __forceinline__ float4 vec4_f32(float4 v) { return v; }
__device__ __forceinline__ float4 vec4_f32(uint2 v) { return bf16x4_f32(v); }

template <int N, int P, typename TA, bool STATES, int SHAPE>
__global__ void __launch_bounds__(ScanShape<N, P, SHAPE>::NT, (ScanShape<N, P, SHAPE>::RESIDENT)) ssm_scan_kernel(SsmScanArgs a) {
    using Sh = ScanShape<N, P, SHAPE>;
    using V4 = typename Vec4Of<TA>::type;
    constexpr int NPT = Sh::NPT, LP = Sh::LP, NS = Sh::NS, NT = Sh::NT, TB = Sh::TB, ROW = Sh::ROW,
                  VPT = Sh::VPT, OPT = Sh::OPT;
    __shared__ __align__(16) float tok[TB][ROW];
    __shared__ __align__(16) float part[STATES ? 1 : TB][NS][P];
    __shared__ float s_dt[TB], s_g[TB], s_a[TB];
    const SsmDims &d = a.d;
    const int tid = threadIdx.x, h = blockIdx.x % d.heads, g = h / d.per;
    SsmSegment sg;
    let_next_start();
    const bool run = ssm_segment<STATES>(a, blockIdx.x / d.heads, sg);
    // a sequence that is not cut needs nothing of the passes in front of this one
    if (!STATES && (!run || sg.entry >= 0 || sg.slot < 0)) await_previous();
    if (!run) return;
    if (STATES && (sg.last || sg.slot < 0)) return;
    const long long out_cols = (long long)d.heads * P;
    if (sg.slot < 0) {
        TA *y = (TA *)a.y;
        for (long long i = tid; i < (sg.t1 - sg.t0) * LP; i += NT)
            store4f(y + (sg.t0 + i / LP) * out_cols + (long long)h * P + (i % LP) * 4,
                    make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    const int lp = tid % LP, ns = tid / LP, p0 = lp * 4, n0 = ns * NPT;
    const long long head = (long long)N * P, all = head * d.heads;
    f32x2 S[NPT / 2][4];
    {
        const float *from = nullptr;
        if (!STATES) {
            if (sg.entry >= 0) from = a.enter + (long long)sg.entry * all;
            else if (a.state_in) from = a.state_in + (long long)sg.slot * all;
        }
#pragma unroll
        for (int i = 0; i < NPT / 2; ++i) {
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
            if (from) {
                u = load4f(from + h * head + (long long)(n0 + 2 * i) * P + p0);
                v = load4f(from + h * head + (long long)(n0 + 2 * i + 1) * P + p0);
            }
            S[i][0] = pack2(u.x, v.x); S[i][1] = pack2(u.y, v.y);
            S[i][2] = pack2(u.z, v.z); S[i][3] = pack2(u.w, v.w);
        }
    }
    const float rate = -expf(a.A_log[h]), bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    const float skip = a.D ? a.D[h] : 0.f;
    double log_sum = 0.0;
    V4 raw[VPT], zraw[OPT];                    // the next block's x, B and C, this block's z
    float raw_dt = 0.f;
    auto fetch = [&](long long t0) {          // the block at t0 into registers
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * NT + tid, r = v / (ROW / 4), c = (v % (ROW / 4)) * 4;
            const long long t = t0 + r;
            if (r < TB && t < sg.t1) {
                const TA *src;
                if (c < P) src = (const TA *)a.x + t * a.ld_x + (long long)h * P + c;
                else if (c < P + N) src = (const TA *)a.b + t * a.ld_bc + (long long)g * N + (c - P);
                else src = (const TA *)a.c + t * a.ld_bc + (long long)g * N + (c - P - N);
                raw[i] = *reinterpret_cast<const V4 *>(src);
            }
        }
        if (tid < TB && t0 + tid < sg.t1)
            raw_dt = to_f32(((const TA *)a.dt)[(t0 + tid) * a.ld_dt + h]);
    };
    fetch(sg.t0);
    for (long long tb = sg.t0; tb < sg.t1; tb += TB) {
        const int count = (int)(sg.t1 - tb < TB ? sg.t1 - tb : TB);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * NT + tid, r = v / (ROW / 4), c = (v % (ROW / 4)) * 4;
            if (r < count) store4f(&tok[r][c], vec4_f32(raw[i]));
        }
        if (tid < count) {
            const float dt = ssm_dt(raw_dt, bias, d);
            s_dt[tid] = dt;
            s_g[tid] = rate * dt;
            s_a[tid] = expf(rate * dt);
        }
        __syncthreads();
        if (!STATES && a.z) {
#pragma unroll
            for (int k = 0; k < OPT; ++k) {
                const int i = k * NT + tid, r = i / LP;
                if (r < count)
                    zraw[k] = *reinterpret_cast<const V4 *>((const TA *)a.z + (tb + r) * a.ld_z + (long long)h * P +
                                                            (i % LP) * 4);
            }
        }
        if (tb + TB < sg.t1) fetch(tb + TB);
        if (STATES) {
            float sum = 0.f;
            for (int r = 0; r < count; ++r) sum += s_g[r];
            log_sum += (double)sum;
        }
        for (int r = 0; r < count; ++r) {
            const float4 x = load4f(&tok[r][p0]);
            const float dt = s_dt[r], dec = s_a[r];
            const f32x2 a2 = pack2(dec, dec);
            const f32x2 x2[4] = {pack2(dt * x.x, dt * x.x), pack2(dt * x.y, dt * x.y),
                                 pack2(dt * x.z, dt * x.z), pack2(dt * x.w, dt * x.w)};
            f32x2 acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int i = 0; i < NPT / 2; i += 2) {
                const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(&tok[r][P + n0 + 2 * i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    S[i][j] = fma2(a2, S[i][j], mul2(B.x, x2[j]));
                    S[i + 1][j] = fma2(a2, S[i + 1][j], mul2(B.y, x2[j]));
                }
                if (!STATES) {
                    const ulonglong2 C =
                        *reinterpret_cast<const ulonglong2 *>(&tok[r][P + N + n0 + 2 * i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[j] = fma2(S[i][j], C.x, acc[j]);
                        acc[j] = fma2(S[i + 1][j], C.y, acc[j]);
                    }
                }
            }
            if (!STATES) {
                float4 o;
                float2 q;
                q = unpack2(acc[0]); o.x = q.x + q.y;
                q = unpack2(acc[1]); o.y = q.x + q.y;
                q = unpack2(acc[2]); o.z = q.x + q.y;
                q = unpack2(acc[3]); o.w = q.x + q.y;
                store4f(&part[r][ns][p0], o);
            }
        }
        __syncthreads();
        if (!STATES) {
            TA *y = (TA *)a.y;
#pragma unroll
            for (int k = 0; k < OPT; ++k) {
                const int i = k * NT + tid, r = i / LP, c = (i % LP) * 4;
                if (r >= count) break;
                const long long t = tb + r;
                float4 o = load4f(&part[r][0][c]);
#pragma unroll
                for (int n = 1; n < NS; ++n) {
                    const float4 q = load4f(&part[r][n][c]);
                    o.x += q.x; o.y += q.y; o.z += q.z; o.w += q.w;
                }
                const float4 x = load4f(&tok[r][c]);
                o.x = fmaf(skip, x.x, o.x); o.y = fmaf(skip, x.y, o.y);
                o.z = fmaf(skip, x.z, o.z); o.w = fmaf(skip, x.w, o.w);
                if (a.z) {
                    const float4 z = vec4_f32(zraw[k]);
                    o.x *= silu_for<TA>(z.x); o.y *= silu_for<TA>(z.y);
                    o.z *= silu_for<TA>(z.z); o.w *= silu_for<TA>(z.w);
                }
                store4f(y + t * out_cols + (long long)h * P + c, o);
            }
            __syncthreads();
        }
    }
    float *to = nullptr;
    if (STATES) to = a.enter + (long long)(sg.entry + 1) * all;
    else if (sg.last && a.state_out) to = a.state_out + (long long)sg.slot * all;
    if (to) {
#pragma unroll
        for (int i = 0; i < NPT / 2; ++i) {
            const float2 q0 = unpack2(S[i][0]), q1 = unpack2(S[i][1]), q2 = unpack2(S[i][2]),
                         q3 = unpack2(S[i][3]);
            store4f(to + h * head + (long long)(n0 + 2 * i) * P + p0, make_float4(q0.x, q1.x, q2.x, q3.x));
            store4f(to + h * head + (long long)(n0 + 2 * i + 1) * P + p0,
                    make_float4(q0.y, q1.y, q2.y, q3.y));
        }
    }
    if (!STATES) await_previous();
    if (STATES && tid == 0) a.seg_log[(long long)sg.entry * d.heads + h] = (float)log_sum;
}

// ---------------------------------------------------------------- launching
namespace {

bool has_tensor_form(const SsmDims &d, bool act_bf16) { return act_bf16 && ssm_tc_supported(d); }
// The tensor-core form, but for batches of few tokens a sequence, which leave its chunks of 128 all but
// empty: it takes 12 to 18 us per round of CTAs whatever the lengths, the form of single tokens a time that
// grows with them.  Batches of equal lengths are even at 30 to 46 tokens a sequence.  But the host knows
// the mean alone, and where one sequence has most of the tokens the form of single tokens is the slower
// one, by the more the fewer the sequences.  So the limit is 8 tokens a sequence, and 24 from ten rounds
// on.  Single tokens / tensor cores, equal lengths | one long sequence among single tokens, us:
//   190 sequences of 8 heads of 64 x 64 (5 rounds), 8 tokens in the mean  37 / 75 | 166 / 89, 16 tokens 45 / 75 | 167 / 92
//   95 of 32 heads of 128 x 64 (10 rounds), 16 tokens 112 / 181 | 229 / 205, 24 tokens 140 / 179 | 255 / 209
//   190 of 32 heads of 128 x 128 (40 rounds), 16 tokens 345 / 655 | 543 / 698, 24 tokens 442 / 653 | 704 / 717, 32 tokens 546 / 649 | 967 / 736
// and one sequence of 32 heads of 128 x 64, 24 tokens 18 / 29, 48 tokens 27 / 27, 64 tokens 30 / 26.
bool on_tensor_cores(const SsmDims &d, bool act_bf16, long long T, long long n_seqs) {
    if (!has_tensor_form(d, act_bf16)) return false;
    const long long few = n_seqs * ssm_tc_units(d) >= 10LL * sm_count() ? 24 : 8;
    return T > 32 && T > few * n_seqs;
}

// CTAs of an SM that a batch is cut for, in the form of single tokens.
constexpr int resident_ctas(int N, int P) { return N * P >= 16384 ? 2 : N * P >= 8192 ? 4 : 8; }

// Segments that run side by side when one sequence has the GPU to itself: the resident CTAs over
// those of one segment (heads, or units of the tensor-core form, one CTA per SM there).
int segments_wanted(const SsmDims &d, bool tensor) {
    int want;
    if (tensor) {
        want = sm_count() / ssm_tc_units(d);
    } else {
        want = sm_count() * resident_ctas(d.N, d.P) / d.heads;
    }
    return want < 1 ? 1 : want;
}

// Tokens of a segment: whole chunks of 128, 256 or more.  A batch whose sequences fill the GPU by
// themselves is then not cut: none of them is longer than its share of T.  (8,192 tokens of 32
// heads, 128 x 128: 117 us in 4 segments, 275 in one; fp32, 4,096 tokens of 8 heads, 64 x 64: 117
// and 828.  Four sequences of 2,048 tokens, which lose by it: 91 us and 83.)
long long segment_len(const SsmDims &d, bool tensor, long long T) {
    const int want = segments_wanted(d, tensor);
    const long long len = ((T + want - 1) / want + 127) / 128 * 128;
    return len < 256 ? 256 : len;
}

// Sequences of k >= 2 segments keep k entering states, and have more than
// (k - 1) seg_len tokens.
long long max_entries(long long T, long long seg_len) { return seg_len >= T ? 0 : 2 * (T / seg_len); }

struct ScanWs {
    size_t seg, ent, log, enter, size;
};
ScanWs scan_ws(const SsmDims &d, long long entries, long long n_seqs) {
    ScanWs w{};
    if (entries == 0) return w;
    size_t at = 0;
    w.seg = at; at += align256((size_t)(n_seqs + 1) * 4);
    w.ent = at; at += align256((size_t)(n_seqs + 1) * 4);
    w.log = at; at += align256((size_t)entries * d.heads * 4);
    w.enter = at; at += (size_t)entries * d.heads * d.N * d.P * 4;
    w.size = at;
    return w;
}

template <int N, int P, typename TA, bool STATES, int SHAPE>
cudaError_t run_scan_as(const SsmScanArgs &a, unsigned grid, cudaStream_t s) {
    constexpr int NT = ScanShape<N, P, SHAPE>::NT;
    auto kern = ssm_scan_kernel<N, P, TA, STATES, SHAPE>;
    if (!STATES && a.seg_len < a.T) return launch_early(kern, dim3(grid), NT, 0, s, a);
    kern<<<grid, NT, 0, s>>>(a);
    return cudaGetLastError();
}

template <int N, int P, typename TA, bool STATES>
cudaError_t run_scan(const SsmScanArgs &a, unsigned segments, cudaStream_t s) {
    const unsigned grid = a.d.heads * segments;   // the heads of a group side by side: B and C come from L2
    constexpr bool kTwoShapes = ScanShape<N, P, WIDE>::NPT != ScanShape<N, P, WHOLE>::NPT;
    // the first pass has no more CTAs than a batch is cut for
    constexpr int kMost = STATES ? resident_ctas(N, P) : INT_MAX;
    // (fp32, 8 heads of 64 x 64, CTAs counted as if every segment were there: 16 sequences of 512 tokens,
    // 384 CTAs, alone 119 us, wide 146, whole 242; 48 of 60 tokens, 472 CTAs, alone 39, wide 33; 50 of 256
    // tokens, 800 CTAs, alone 129, wide 108; 256 of 512 tokens wide 997, whole 784)
    if constexpr (!kTwoShapes) {
        return run_scan_as<N, P, TA, STATES, WHOLE>(a, grid, s);
    } else {
        if (grid <= 3 * (unsigned)sm_count()) return run_scan_as<N, P, TA, STATES, ALONE>(a, grid, s);
        if constexpr (kMost > 6) {
            if (grid > 6 * (unsigned)sm_count()) return run_scan_as<N, P, TA, STATES, WHOLE>(a, grid, s);
        }
        return run_scan_as<N, P, TA, STATES, WIDE>(a, grid, s);
    }
}

template <int N, int P, typename TA>
cudaError_t run_scan_pass(const SsmScanArgs &a, bool states, unsigned segments, cudaStream_t s) {
    return states ? run_scan<N, P, TA, true>(a, segments, s) : run_scan<N, P, TA, false>(a, segments, s);
}
template <int N, typename TA> cudaError_t run_scan_p(const SsmScanArgs &a, bool states, unsigned segments, cudaStream_t s) {
    switch (a.d.P) {
        case 32: return run_scan_pass<N, 32, TA>(a, states, segments, s);
        case 64: return run_scan_pass<N, 64, TA>(a, states, segments, s);
        default: return run_scan_pass<N, 128, TA>(a, states, segments, s);
    }
}
template <typename TA> cudaError_t run_scan_np(const SsmScanArgs &a, bool states, unsigned segments, cudaStream_t s) {
    switch (a.d.N) {
        case 16: return run_scan_p<16, TA>(a, states, segments, s);
        case 32: return run_scan_p<32, TA>(a, states, segments, s);
        case 64: return run_scan_p<64, TA>(a, states, segments, s);
        default: return run_scan_p<128, TA>(a, states, segments, s);
    }
}

}  // namespace

// Grows with T: segments are 256 tokens or longer, and a batch has no more than are wanted.
size_t ssm_scan_ws_bytes(const SsmDims &d, bool act_bf16, long long T, long long n_seqs) {
    long long most = segments_wanted(d, false);        // of either form: a smaller batch may take the other
    if (has_tensor_form(d, act_bf16) && segments_wanted(d, true) > most) most = segments_wanted(d, true);
    return most < 2 ? 0 : scan_ws(d, 2 * (T / 256 < most ? T / 256 : most), n_seqs).size;
}

size_t ssm_scan_carve(SsmScanArgs &a, bool act_bf16, void *ws) {
    a.seg_len = segment_len(a.d, on_tensor_cores(a.d, act_bf16, a.T, a.n_seqs), a.T);
    a.max_enter = (int)max_entries(a.T, a.seg_len);
    const ScanWs w = scan_ws(a.d, a.max_enter, a.n_seqs);
    char *p = (char *)ws;
    if (w.size == 0 || !p) return w.size;
    a.seg_base = (int *)(p + w.seg);
    a.enter_base = (int *)(p + w.ent);
    a.seg_log = (float *)(p + w.log);
    a.enter = (float *)(p + w.enter);
    return w.size;
}

cudaError_t launch_ssm_scan(const SsmScanArgs &a, bool act_bf16, cudaStream_t s) {
    const bool cut = a.seg_len < a.T;
    // with states only: the segments that are not their sequence's last
    const unsigned all = cut ? (unsigned)(a.n_seqs + a.max_enter / 2) : (unsigned)a.n_seqs;
    auto pass = [&](bool states) {
        const unsigned segments = states ? (unsigned)(a.max_enter / 2) : all;
        if (on_tensor_cores(a.d, act_bf16, a.T, a.n_seqs)) return launch_ssm_scan_tc(a, states, segments, s);
        return act_bf16 ? run_scan_np<__nv_bfloat16>(a, states, segments, s) : run_scan_np<float>(a, states, segments, s);
    };
    if (cut) {
        cudaError_t e = cudaSuccess;
        if (a.n_seqs > kWarpSeqs) {
            ssm_segment_map_kernel<<<1, 1024, 0, s>>>(a);
            e = cudaGetLastError();
        }
        if (e == cudaSuccess) e = pass(true);
        const int most = a.n_seqs <= kWarpSeqs ? a.max_enter / 2 : 32;          // sequences that are cut
        const dim3 chain(a.d.heads, (a.d.N * a.d.P / 4 + 255) / 256, a.n_seqs < most ? a.n_seqs : most);
        if (e == cudaSuccess) e = launch_early(ssm_chain_states_kernel, chain, 256, 0, s, a);
        if (e != cudaSuccess) return e;
    }
    return pass(false);
}

}  // namespace gdn
