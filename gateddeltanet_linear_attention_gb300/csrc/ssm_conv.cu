// ssm_conv.cu -- the causal convolution of the state space mixer over packed
// prompts, and the one-token step (convolution, then scan).
#include "ssm_common.cuh"

namespace gdn {

namespace {

constexpr int kVec = 4;          // channels of a thread
constexpr int kConvThreads = 128;
constexpr int kRun = 16;         // tokens of a thread
constexpr int kStepThreads = 128; // of the one-token state kernel
constexpr int kBatch = 8;        // tokens whose loads are issued together

// Four channels as the memory holds them, and as fp32.
__device__ __forceinline__ float4 load_raw(const float *p) { return load4f(p); }
__device__ __forceinline__ uint2 load_raw(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ void raw_f32(const float4 &r, float (&v)[4]) { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
__device__ __forceinline__ void raw_f32(const uint2 &r, float (&v)[4]) { raw_f32(bf16x4_f32(r), v); }
template <typename T> __device__ __forceinline__ void load4(const T *p, float (&v)[4]) { raw_f32(load_raw(p), v); }
template <typename T> __device__ __forceinline__ void store4(T *p, const float (&v)[4]) {
    store4f(p, make_float4(v[0], v[1], v[2], v[3]));
}

// Sequence that holds token t, or -1 (in front of the first or behind the last one).
__device__ __forceinline__ int seq_of(const int32_t *cu, int n_seqs, long long t) {
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return cu[lo] <= t ? lo : -1;
}

// Looks at all pairs of bounds, a thread of the grid's first column of blocks at each.  (Out of line: as
// a part of the kernel it cost it registers.)
__device__ __noinline__ void check_bounds(const int32_t *cu, int n_seqs, long long T, unsigned *err) {
    for (long long n = blockIdx.x * (long long)kConvThreads + threadIdx.x; n < n_seqs; n += gridDim.x * (long long)kConvThreads) {
        long long s, e;
        seq_bounds(cu, (int)n, T, err, s, e);
    }
}

}  // namespace

// ------------------------------------------------------------- packed prompts
// out_t[c] = SiLU(bias[c] + sum_j w[c][j] x_{t-3+j}[c]).  A thread owns 4
// channels of kRun packed tokens and slides the three-token window in
// registers.  HBM-bound: the input once (three tokens in kRun again, from L2)
// and the output once.
//
// The history is replaced by the same launch: the thread whose run holds a
// sequence's first token also computes the two tokens behind it (the ones that
// still reach into the history) wherever they lie, so it alone reads that
// history and may then overwrite it.  The two tokens' own run leaves them out.
//
// Bound by the memory's latency: the tokens in flight are the blocks of an SM times kBatch.  bf16:
// 8 blocks (8,192 tokens of 8,192 channels: 51 us, 5.25 TB/s; 7 blocks 53 us, 6 blocks 55 us, 10
// blocks of fewer registers 56 us); fp32, whose loads need more registers, 6 (17.3 us a ragged batch
// of 46 MB; 7 blocks 18.4, 8 blocks 19.4).  Runs of 32 tokens: 51 us and 20.6 us.
template <typename TA>
__global__ void __launch_bounds__(kConvThreads, sizeof(TA) == 2 ? 8 : 6) ssm_conv_kernel(SsmConvArgs a) {
    using Raw = decltype(load_raw((const TA *)nullptr));
    const SsmDims &d = a.d;
    const int c0 = (blockIdx.y * kConvThreads + threadIdx.x) * kVec;
    // every pair of bounds is looked at by some block: a run below stops at the first sequence behind it
    if (blockIdx.y == 0) check_bounds(a.cu, a.n_seqs, a.T, a.err);
    if (c0 >= d.ch) return;
    const TA *__restrict__ x = (const TA *)a.x + c0;
    TA *__restrict__ out = (TA *)a.out + c0;
    TA *hist = (TA *)a.conv_state;
    const long long r0 = (long long)blockIdx.x * kRun, r1 = r0 + kRun < a.T ? r0 + kRun : a.T;
    f32x2 w[4][2], bias[2] = {0ull, 0ull};             // of pairs of channels
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float u[4], v[4];
        load4((const TA *)a.w + (long long)(c0 + 2 * i) * 4, u);
        load4((const TA *)a.w + (long long)(c0 + 2 * i + 1) * 4, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j][i] = pack2(u[j], v[j]);
    }
    if (a.bias) {
        float u[4];
        load4((const TA *)a.bias + c0, u);
        bias[0] = pack2(u[0], u[1]);
        bias[1] = pack2(u[2], u[3]);
    }

    // first sequence that has a token at r0 or later
    int n = seq_of(a.cu, a.n_seqs, r0);
    if (n < 0) n = 0;
    for (; n < a.n_seqs; ++n) {
        long long s, e;
        seq_bounds(a.cu, n, a.T, a.err, s, e);
        if (s >= r1) break;
        if (e <= r0 || e <= s) continue;
        const int slot = slot_of(a.state_idx, n, d.n_slots, a.err);
        const bool starts = s >= r0;                   // this run holds its first token
        const long long head_end = s + 3 < e ? s + 3 : e;
        long long t = starts ? s : (r0 > head_end ? r0 : head_end);
        const long long end = (starts && head_end > r1) ? head_end : (e < r1 ? e : r1);
        if (t >= end && !starts) continue;
        if (slot < 0) {
            const float zero[kVec] = {0.f, 0.f, 0.f, 0.f};
            for (; t < end; ++t) store4(out + t * d.ch, zero);
            continue;
        }
        float win[3][kVec];
        if (starts) {
#pragma unroll
            for (int j = 0; j < 3; ++j)
#pragma unroll
                for (int i = 0; i < kVec; ++i) win[j][i] = 0.f;
            if (hist) {
                TA *hp = hist + ((long long)slot * d.ch + c0) * 3;
                float u[3][4];
#pragma unroll
                for (int i = 0; i < 3; ++i) load4(hp + 4 * i, u[i]);
#pragma unroll
                for (int i = 0; i < kVec; ++i)
#pragma unroll
                    for (int j = 0; j < 3; ++j) win[j][i] = u[(3 * i + j) / 4][(3 * i + j) % 4];
                // the new history: the last three inputs, of the old history where e - s < 3
                float last[3][kVec];
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const long long tt = e - 3 + j;
                    if (tt >= s) {
                        load4(x + tt * a.ld_x, last[j]);
                    } else {
                        const int k = (int)(tt - s + 3);
#pragma unroll
                        for (int i = 0; i < kVec; ++i)
                            last[j][i] = k == 1 ? win[1][i] : k == 2 ? win[2][i] : win[0][i];
                    }
                }
                float v[3][4];
#pragma unroll
                for (int i = 0; i < kVec; ++i)
#pragma unroll
                    for (int j = 0; j < 3; ++j) v[(3 * i + j) / 4][(3 * i + j) % 4] = last[j][i];
#pragma unroll
                for (int i = 0; i < 3; ++i) store4(hp + 4 * i, v[i]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j) load4(x + (t - 3 + j) * a.ld_x, win[j]);
        }
        f32x2 past[3][2];                              // the window in pairs of channels
#pragma unroll
        for (int j = 0; j < 3; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) past[j][i] = pack2(win[j][2 * i], win[j][2 * i + 1]);
        auto emit = [&](const float (&cur)[kVec], long long at) {
            float o[kVec];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x2 x = pack2(cur[2 * i], cur[2 * i + 1]);
                const float2 v = unpack2(
                    fma2(w[3][i], x, fma2(w[2][i], past[2][i], fma2(w[1][i], past[1][i], fma2(w[0][i], past[0][i], bias[i])))));
                o[2 * i] = silu_for<TA>(v.x);
                o[2 * i + 1] = silu_for<TA>(v.y);
                past[0][i] = past[1][i];
                past[1][i] = past[2][i];
                past[2][i] = x;
            }
            store4(out + at * d.ch, o);
        };
        for (; t + kBatch <= end; t += kBatch) {       // the loads of kBatch tokens in flight at once
            Raw raw[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) raw[k] = load_raw(x + (t + k) * a.ld_x);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                float cur[kVec];
                raw_f32(raw[k], cur);
                emit(cur, t + k);
            }
        }
        for (; t < end; ++t) {
            float cur[kVec];
            load4(x + t * a.ld_x, cur);
            emit(cur, t);
        }
    }
}

cudaError_t launch_ssm_conv(const SsmConvArgs &a, bool act_bf16, cudaStream_t s) {
    const dim3 grid((unsigned)((a.T + kRun - 1) / kRun),
                    (unsigned)((a.d.ch / kVec + kConvThreads - 1) / kConvThreads));
    if (act_bf16) ssm_conv_kernel<__nv_bfloat16><<<grid, kConvThreads, 0, s>>>(a);
    else ssm_conv_kernel<float><<<grid, kConvThreads, 0, s>>>(a);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ one token
// Convolution step: one thread per channel; the history is shifted in place by
// its only reader and the fp32 result goes to the workspace.  Bound by latency:
// 64 sequences of 8,192 channels 6 us alone, 0.7 TB/s, most of it hidden behind the
// state's loads.
template <typename TA>
__global__ void __launch_bounds__(256) ssm_step_conv_kernel(SsmStepArgs a) {
    // the state kernel may start loading states now; it waits for this grid before it reads `ws`
    let_next_start();
    const SsmDims &d = a.d;
    const int n = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if (c >= d.ch) return;
    const int slot = slot_of(a.state_idx, n, d.n_slots, a.err);
    if (slot < 0) return;
    TA *hp = (TA *)a.conv_state + ((long long)slot * d.ch + c) * 3;
    const TA h0 = hp[0], h1 = hp[1], h2 = hp[2], cur = ((const TA *)a.x)[(long long)n * a.ld_x + c];
    float w[4];
    taps_f32(load_taps((const TA *)a.w, c), w);
    const float b = a.bias ? to_f32(((const TA *)a.bias)[c]) : 0.f;
    hp[0] = h1; hp[1] = h2; hp[2] = cur;
    a.ws[(long long)n * d.ch + c] =
        silu_f(fmaf(w[3], to_f32(cur), fmaf(w[2], to_f32(h2), fmaf(w[1], to_f32(h1), fmaf(w[0], to_f32(h0), b)))));
}

// State step: one CTA per (sequence, head, 32 columns) reads its part of the
// state once, writes it once and reduces y over the rows.  HBM-bound on the
// state.  32 columns: whole 128-byte lines, and parts small enough that many
// CTAs of an SM overlap their loads and stores.  Launched while the convolution
// step still runs: the state's loads are issued before its results are awaited.
// 64 sequences of 32 heads, 128 x 128: the step takes 47 us, 5.9 TB/s of states,
// 0.87 of a plain copy's rate.
template <int N, int P, typename TA>
__global__ void __launch_bounds__(kStepThreads) ssm_step_state_kernel(SsmStepArgs a) {
    constexpr int LP = 8, NS = kStepThreads / LP, RPT = N / NS;     // 16 row slices
    __shared__ __align__(16) float part[NS][32];
    const SsmDims &d = a.d;
    constexpr int parts = P / 32;
    const int h = blockIdx.x / parts, n = blockIdx.y, g = h / d.per, tid = threadIdx.x;
    const int p0 = (blockIdx.x % parts) * 32 + (tid % LP) * 4, ns = tid / LP;
    const int slot = slot_of(a.state_idx, n, d.n_slots, a.err);
    TA *y = (TA *)a.y + ((long long)n * d.heads + h) * P;
    if (slot < 0) {
        if (tid < LP) store4f(y + p0, make_float4(0.f, 0.f, 0.f, 0.f));
        await_previous();
        return;
    }
    float *S = a.state + ((long long)slot * d.heads + h) * N * P;
    float4 m[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) m[i] = load4f(S + (long long)(ns + i * NS) * P + p0);
    const float dt = ssm_dt(to_f32(((const TA *)a.dt)[(long long)n * a.ld_dt + h]),
                            a.dt_bias ? a.dt_bias[h] : 0.f, d);
    const float dec = expf(-expf(a.A_log[h]) * dt), skip = a.D ? a.D[h] : 0.f;
    float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.z && tid < LP) z = load4f((const TA *)a.z + (long long)n * a.ld_z + (long long)h * P + p0);
    await_previous();
    const float *row = a.ws + (long long)n * d.ch;
    const float *B = row + d.heads * P + g * N, *C = B + d.groups * N;
    const float4 x = load4f(row + h * P + p0);
    float b[RPT], c[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        b[i] = B[ns + i * NS];
        c[i] = C[ns + i * NS];
    }
    const float4 u = make_float4(dt * x.x, dt * x.y, dt * x.z, dt * x.w);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        m[i].x = fmaf(dec, m[i].x, b[i] * u.x); m[i].y = fmaf(dec, m[i].y, b[i] * u.y);
        m[i].z = fmaf(dec, m[i].z, b[i] * u.z); m[i].w = fmaf(dec, m[i].w, b[i] * u.w);
        acc.x = fmaf(c[i], m[i].x, acc.x); acc.y = fmaf(c[i], m[i].y, acc.y);
        acc.z = fmaf(c[i], m[i].z, acc.z); acc.w = fmaf(c[i], m[i].w, acc.w);
        store4f(S + (long long)(ns + i * NS) * P + p0, m[i]);
    }
    store4f(&part[ns][(tid % LP) * 4], acc);
    __syncthreads();
    if (tid < LP) {
        float4 o = load4f(&part[0][tid * 4]);
#pragma unroll
        for (int k = 1; k < NS; ++k) {
            const float4 q = load4f(&part[k][tid * 4]);
            o.x += q.x; o.y += q.y; o.z += q.z; o.w += q.w;
        }
        o.x = fmaf(skip, x.x, o.x); o.y = fmaf(skip, x.y, o.y);
        o.z = fmaf(skip, x.z, o.z); o.w = fmaf(skip, x.w, o.w);
        if (a.z) {
            o.x *= silu_f(z.x); o.y *= silu_f(z.y); o.z *= silu_f(z.z); o.w *= silu_f(z.w);
        }
        store4f(y + p0, o);
    }
}

size_t ssm_step_ws_bytes(const SsmDims &d, long long n) { return (size_t)n * d.ch * 4; }

namespace {
template <int N, int P, typename TA> cudaError_t run_step(const SsmStepArgs &a, cudaStream_t s) {
    ssm_step_conv_kernel<TA><<<dim3((a.d.ch + 255) / 256, a.n), 256, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_early(ssm_step_state_kernel<N, P, TA>, dim3(a.d.heads * (P / 32), a.n), kStepThreads, 0, s, a);
}
template <int N, typename TA> cudaError_t run_step_p(const SsmStepArgs &a, cudaStream_t s) {
    switch (a.d.P) {
        case 32: return run_step<N, 32, TA>(a, s);
        case 64: return run_step<N, 64, TA>(a, s);
        default: return run_step<N, 128, TA>(a, s);
    }
}
template <typename TA> cudaError_t run_step_np(const SsmStepArgs &a, cudaStream_t s) {
    switch (a.d.N) {
        case 16: return run_step_p<16, TA>(a, s);
        case 32: return run_step_p<32, TA>(a, s);
        case 64: return run_step_p<64, TA>(a, s);
        default: return run_step_p<128, TA>(a, s);
    }
}
}  // namespace

cudaError_t launch_ssm_step(const SsmStepArgs &a, bool act_bf16, cudaStream_t s) {
    return act_bf16 ? run_step_np<__nv_bfloat16>(a, s) : run_step_np<float>(a, s);
}

}  // namespace gdn
