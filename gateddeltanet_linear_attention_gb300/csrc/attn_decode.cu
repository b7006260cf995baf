// attn_decode.cu -- attention of a few new tokens over a paged cache.
//
//   s_i = scale q . k_i,   m = max s,   l = sum exp(s - m),   o = sum exp(s - m) v_i / l
//
// One pass over the visible tokens with the running m, l and o of each query row; the tiles of
// all sequences and key heads are one line cut into equal shares (AttnWalk).  A unit that one CTA
// holds whole is written at once; of the others every CTA leaves its (m, l, o), and the join kernel
// adds them up in the order of the tokens: no atomics, equal calls give equal bits.
#include "attn_common.cuh"

namespace gdn {

namespace {

constexpr int kSimtTile = 32;

// The 32-bit form, on the CUDA cores: RPW query rows a warp, a tile of 32 tokens in shared memory, a token a lane for the
// scores and D / 32 columns a lane for the sums.  The next tile is on its way while one is worked on, the pages of the one
// behind it are looked up.  Bound by its reads of shared memory and multiply-adds (a warp reads all of a tile for its rows): 64
// sequences of 256 to 8,192 tokens, 8 key heads of 128 columns, 4 query heads each (2.1 GB) 556 us, 0.56 of the copy rate (1,258
// with a tile loaded and worked on in turn); 32 of them, 4 key heads, 12 rows each 307 us, 0.28; 16 of up to 4,096, 4 key heads,
// 64 rows each 237 us, 0.07 (eight rows a warp: 342, registers).
// Exponentials are ex2.approx: 2^-22 of a weight and zeros below 2^-126, in a sum whose scores err by more (16 roundings of 2^-24
// and more, times their size).
// Two tiles of 256 columns leave room for one CTA an SM: with many rows it is twice as large.
template <int D, int RPW> constexpr int simt_threads = D == 256 && RPW == 4 ? 512 : 256;
template <int D, int RPW>
__global__ void __launch_bounds__((simt_threads<D, RPW>)) attn_decode_simt_kernel(const AttnDecodeArgs a) {
    constexpr int THREADS = simt_threads<D, RPW>, TILE = kSimtTile, LDK = D + 4, CPL = D / 32, WARPS = THREADS / 32, RB = WARPS * RPW, BUFFER = TILE * (LDK + D);
    constexpr int PASS = THREADS / (D / 4);            // tokens that the block copies at a time
    static_assert(16 % PASS == 0, "of one piece of a page");
    extern __shared__ float4 smem4[];
    float *tiles = reinterpret_cast<float *>(smem4), *qs = tiles + 2 * BUFFER;
    __shared__ long long sums[33];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rows = a.d.grp * a.tokens, row0 = blockIdx.y * RB;
    await_previous();
    let_next_start();
    AttnWalk w;
    if (!attn_begin<TILE, THREADS>(a, blockIdx.x, sums, found, w)) {
        if (blockIdx.y == 0 && tid == 0) a.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    const float *kp = (const float *)a.k_pages, *vp = (const float *)a.v_pages;
    // the tile to copy next, and the pages of its two pieces of 16 tokens (-1: masked)
    AttnWalk next = w;
    int page[2], there_now = 0, buffer = 0;
    auto look_up = [&]() {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int i = (next.s.tile0 + next.t) * TILE + p * 16;
            page[p] = -1;
            if (i < next.s.len && i + 16 > next.s.first) {
                page[p] = a.table[(long long)next.s.row * a.d.max_pages + (i >> a.d.page_shift)];
                if (page[p] < 0 || page[p] >= a.d.n_pages) {
                    set_error(a.err, GDN_DEVERR_PAGE);
                    page[p] = -1;
                }
            }
        }
    };
    auto copy = [&](int to) {                               // what is masked is zero; which pieces are there
        const int i0 = (next.s.tile0 + next.t) * TILE, c = tid % (D / 4) * 4;
        const uint32_t ks = (uint32_t)__cvta_generic_to_shared(tiles + to * BUFFER), vs = ks + TILE * LDK * 4;
#pragma unroll
        for (int t0 = 0; t0 < TILE; t0 += PASS) {
            const int t = t0 + tid / (D / 4), i = i0 + t, from = page[t0 >> 4];
            const bool in = from >= 0 && i < next.s.len && i >= next.s.first;
            const long long at = in ? (((long long)from * a.d.hkv + next.h) * a.d.page + (i & (a.d.page - 1))) * D + c : 0;
            const int bytes = in ? 16 : 0;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(ks + (t * LDK + c) * 4), "l"(kp + at), "r"(bytes) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(vs + (t * D + c) * 4), "l"(vp + at), "r"(bytes) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return (page[0] >= 0 ? 1 : 0) | (page[1] >= 0 ? 2 : 0);
    };
    look_up();
    int there_next = copy(0);
    attn_next<TILE>(a, next);
    if (next.left > 0) look_up();
    bool unit_first = true;               // this unit is the CTA's first one
    while (w.left > 0) {
        const bool whole_front = w.t == 0;
        const int n = w.n, h = w.h;
        const AttnSeq s = w.s;
        // query rows in 32 bits
        __syncthreads();
        for (int i = tid; i < RB * (D / 4); i += THREADS) {
            const int r = row0 + i / (D / 4), c = i % (D / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int tok = r / a.d.grp, g = r % a.d.grp;
                v = load4f((const float *)a.q + ((long long)n * a.tokens + tok) * a.ld_q + (long long)(h * a.d.grp + g) * a.hs_q + c);
            }
            reinterpret_cast<float4 *>(qs)[i] = v;
        }
        float m[RPW], l[RPW], o[RPW][CPL];
        int end[RPW], begin[RPW];
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
            const int row = row0 + warp * RPW + r;
            end[r] = row < rows ? s.len - a.tokens + 1 + row / a.d.grp : 0;
            begin[r] = a.window > 0 ? end[r] - a.window : 0;
#pragma unroll
            for (int c = 0; c < CPL; ++c) o[r][c] = 0.f;
        }
        bool unit_end;
        do {
            const int i0 = (s.tile0 + w.t) * TILE;
            const float *ks = tiles + buffer * BUFFER, *vs = ks + TILE * LDK;
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();              // the tile is there, and the one before has been read
            there_now = there_next;
            if (next.left > 0) {
                there_next = copy(buffer ^ 1);
                attn_next<TILE>(a, next);
                if (next.left > 0) look_up();
            }
            buffer ^= 1;
            unit_end = attn_next<TILE>(a, w);
            if (row0 + warp * RPW >= rows) continue;
            float sc[RPW];
#pragma unroll
            for (int r = 0; r < RPW; ++r) sc[r] = 0.f;
            for (int c = 0; c < D; c += 4) {
                const float4 kv = *reinterpret_cast<const float4 *>(ks + lane * LDK + c);
#pragma unroll
                for (int r = 0; r < RPW; ++r) {
                    const float4 q = *reinterpret_cast<const float4 *>(qs + (warp * RPW + r) * D + c);
                    sc[r] = fmaf(q.x, kv.x, fmaf(q.y, kv.y, fmaf(q.z, kv.z, fmaf(q.w, kv.w, sc[r]))));
                }
            }
            const int i = i0 + lane;
            const bool there = (there_now >> (lane >> 4) & 1) && i >= s.first && i < s.len;
            float p[RPW];
            unsigned seen[RPW];
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                const bool see = there && i < end[r] && i >= begin[r];
                seen[r] = __ballot_sync(0xffffffffu, see);
                float top = see ? sc[r] : -INFINITY;
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                const float nm = fmaxf(m[r], top * a.scale_log2), ref = nm == -INFINITY ? 0.f : nm;
                const float back = exp2_fast(m[r] - ref);
                p[r] = see ? exp2_fast(fmaf(sc[r], a.scale_log2, -ref)) : 0.f;
                m[r] = nm;
                l[r] = l[r] * back + p[r];
#pragma unroll
                for (int c = 0; c < CPL; ++c) o[r][c] *= back;
            }
            for (int t = 0; t < TILE; ++t) {
                float v[CPL];
                if constexpr (CPL == 2) {
                    const float2 x = *reinterpret_cast<const float2 *>(vs + t * D + lane * 2);
                    v[0] = x.x; v[1] = x.y;
                } else {
#pragma unroll
                    for (int c = 0; c < CPL; c += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(vs + t * D + lane * 4 + c * 32);
                        v[c] = x.x; v[c + 1] = x.y; v[c + 2] = x.z; v[c + 3] = x.w;
                    }
                }
#pragma unroll
                for (int r = 0; r < RPW; ++r) {
                    if (seen[r] >> t & 1u) {      // what a row does not see may hold anything
                        const float pt = __shfl_sync(0xffffffffu, p[r], t);
#pragma unroll
                        for (int c = 0; c < CPL; ++c) o[r][c] = fmaf(pt, v[c], o[r][c]);
                    }
                }
            }
        } while (!unit_end && w.left > 0);
        // the unit's rows: whole, or a part for the join kernel
        const bool whole = whole_front && unit_end;
        const int slot = unit_first ? 0 : 1;
        float *part = attn_part(a, blockIdx.x, slot);
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
            const int row = row0 + warp * RPW + r;
            // a largest score above the range leaves no weight to any token
            if (m[r] == INFINITY) l[r] = NAN;
            const float lsum = warp_sum(l[r]);
            if (row < rows) {
                const int tok = row / a.d.grp, g = row % a.d.grp;
                const long long orow = ((long long)n * a.tokens + tok) * a.d.hq + h * a.d.grp + g;
                const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    const int col = CPL == 2 ? lane * 2 + c : lane * 4 + (c >> 2) * 128 + (c & 3);
                    if (whole) ((float *)a.out)[orow * D + col] = o[r][c] * inv;
                    else part[row * D + col] = o[r][c];
                }
                if (lane == 0) {
                    if (whole) {
                        if (a.lse) a.lse[orow] = lsum == 0.f ? -INFINITY : (m[r] + log2f(lsum)) * kLn2;
                    } else {
                        part[rows * D + 2 * row] = m[r];
                        part[rows * D + 2 * row + 1] = lsum;
                    }
                }
            }
        }
        if (w.left == 0 && blockIdx.y == 0 && tid == 0) {
            // the CTA that holds a unit's front joins it: the CTAs behind that hold the rest
            int parts = 0;
            if (!unit_end && whole_front) parts = 1 + (int)((s.tiles - w.t + w.per - 1) / w.per);
            a.joins[blockIdx.x] = make_int4(n, h, slot, parts);
        }
        unit_first = false;
    }
}

// Adds up the parts of the units that several CTAs hold: part p of the unit whose front is CTA c's lies in CTA c + p.  Blocks
// (c, y) take query rows.  What a part counts, 2^(m_p - max m), is known from the statistics, so the sums' loads wait for
// nothing and four are under way (two, three, eight: slower, by loads that wait or registers): a row a group of D / 4 threads,
// or, of more than 16 parts, a row by all groups.  Against groups that carry m and l from part to part: 76 parts of 8 rows, 256
// columns, 52 -> 49 us a call; 64 rows, one sequence of 700 tokens 16.3 -> 12.6; 3 rows, 700 tokens 8.1 -> 8.7, where a row by
// all groups would be as fast, and slower (10.3 against 9.5) with 6 rows of 64 columns.  Fixed orders throughout.
constexpr int kJoinThreads = 256, kJoinRows = 16, kJoinAhead = 4;
__device__ __forceinline__ void add_part(float4 &x, const float4 &o, float f) {
    x = make_float4(fmaf(o.x, f, x.x), fmaf(o.y, f, x.y), fmaf(o.z, f, x.z), fmaf(o.w, f, x.w));
}
template <typename T, int D> __global__ void __launch_bounds__(kJoinThreads, 5) attn_join_kernel(const AttnDecodeArgs a) {
    constexpr int COLS = D / 4, GROUPS = kJoinThreads / COLS, WARPS = kJoinThreads / 32, AHEAD = kJoinAhead;
    static_assert(kAttnMaxCtas <= 2 * kJoinThreads, "two parts a thread");
    __shared__ float4 acc[GROUPS][COLS];
    __shared__ float factor[kAttnMaxCtas], tops[WARPS], totals[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = tid / COLS, col = tid % COLS, rows = a.d.grp * a.tokens;
    let_next_start();
    await_previous();
    const int4 j = a.joins[blockIdx.x];
    if (j.w < 2) return;
    const int parts = min(j.w, a.ctas - (int)blockIdx.x);
    auto part = [&](int p) { return attn_part(a, blockIdx.x + p, p == 0 ? j.z : 0); };
    auto write = [&](int row, float4 x, float m, float l) {
        const long long orow = ((long long)j.x * a.tokens + row / a.d.grp) * a.d.hq + j.y * a.d.grp + row % a.d.grp;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        store4f((T *)a.out + orow * D + col * 4, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
        if (col == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    };
    if (parts <= 16) {
        // a row a group: 16 lanes have the statistics, a part each
        const unsigned mask = 0xffffu << (lane & 16);
        for (int row = blockIdx.y * GROUPS + group; row < rows; row += gridDim.y * GROUPS) {
            float2 ml = make_float2(-INFINITY, 0.f);
            if ((lane & 15) < parts) ml = *reinterpret_cast<const float2 *>(part(lane & 15) + rows * D + 2 * row);
            float4 o[AHEAD], x = make_float4(0.f, 0.f, 0.f, 0.f);
            auto load = [&](int p0) {
#pragma unroll
                for (int k = 0; k < AHEAD; ++k)
                    if (p0 + k < parts) o[k] = *reinterpret_cast<const float4 *>(part(p0 + k) + row * D + col * 4);
            };
            load(0);
            float m = ml.x;
#pragma unroll
            for (int k = 8; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, k));
            const float f = exp2_fast(ml.x - (m == -INFINITY ? 0.f : m));
            float l = ml.y * f;
#pragma unroll
            for (int k = 8; k > 0; k >>= 1) l += __shfl_xor_sync(mask, l, k);
            for (int p0 = 0; p0 < parts; p0 += AHEAD) {
                if (p0 > 0) load(p0);
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const float g = __shfl_sync(mask, f, (p0 + k) & 15, 16);
                    if (p0 + k < parts) add_part(x, o[k], g);
                }
            }
            write(row, x, m, l);
        }
        return;
    }
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        float2 ml[2];
        float4 o[AHEAD];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int p = tid + k * kJoinThreads;
            ml[k] = p < parts ? *reinterpret_cast<const float2 *>(part(p) + rows * D + 2 * row) : make_float2(-INFINITY, 0.f);
        }
        auto load = [&](int p0) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (p0 + k * GROUPS < parts) o[k] = *reinterpret_cast<const float4 *>(part(p0 + k * GROUPS) + row * D + col * 4);
        };
        load(group);
        float m = fmaxf(ml[0].x, ml[1].x);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        __syncthreads();                                    // the row before has been read
        if (lane == 0) tops[warp] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WARPS; ++k) m = fmaxf(m, tops[k]);
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int p = tid + k * kJoinThreads;
            const float f = exp2_fast(ml[k].x - ref);
            if (p < parts) factor[p] = f;
            l = fmaf(ml[k].y, f, l);
        }
        l = warp_sum(l);
        if (lane == 0) totals[warp] = l;
        __syncthreads();
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = group; p0 < parts; p0 += AHEAD * GROUPS) {
            if (p0 > group) load(p0);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (p0 + k * GROUPS < parts) add_part(x, o[k], factor[p0 + k * GROUPS]);
        }
        acc[group][col] = x;
        __syncthreads();
        if (group != 0) continue;
        for (int k = 1; k < GROUPS; ++k) {
            const float4 y = acc[k][col];
            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        l = 0.f;
        for (int k = 0; k < WARPS; ++k) l += totals[k];
        write(row, x, m, l);
    }
}

template <int D, int RPW> cudaError_t run_simt(AttnDecodeArgs a, cudaStream_t s) {
    constexpr int THREADS = simt_threads<D, RPW>, RB = THREADS / 32 * RPW, smem = (2 * kSimtTile * (2 * D + 4) + RB * D) * 4;
    const auto kernel = attn_decode_simt_kernel<D, RPW>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    if (2 * (smem + 1024) > 227 * 1024) a.ctas = sm_count();      // one CTA an SM
    const int rows = a.d.grp * a.tokens;
    const cudaError_t e = launch_early(kernel, dim3(a.ctas, (rows + RB - 1) / RB), THREADS, smem, s, a);
    return e != cudaSuccess ? e : launch_attn_join(a, false, s);
}
template <int D> cudaError_t run_rows(const AttnDecodeArgs &a, cudaStream_t s) {
    const int rows = a.d.grp * a.tokens;
    return rows <= 8 ? run_simt<D, 1>(a, s) : rows <= 16 ? run_simt<D, 2>(a, s) : run_simt<D, 4>(a, s);
}

int most_ctas() {
    const int n = sm_count() * kAttnCtasPerSm;
    return n < kAttnMaxCtas ? n : kAttnMaxCtas;
}

}  // namespace

size_t attn_decode_ws_bytes(const AttnDims &d, int rows) {
    return (size_t)most_ctas() * (sizeof(int4) + 2 * (size_t)attn_part_floats(rows, d.D) * 4);
}

void attn_decode_carve(AttnDecodeArgs &a, void *ws) {
    a.ctas = most_ctas();
    a.lead = 0;
    a.joins = (int4 *)ws;
    a.parts = (float *)(a.joins + a.ctas);
}

cudaError_t launch_attn_join(const AttnDecodeArgs &a, bool act_bf16, cudaStream_t s) {
    const int rows = a.d.grp * a.tokens;
    const dim3 grid(a.ctas, rows < kJoinRows ? rows : kJoinRows);
    if (act_bf16)
        return a.d.D == 64 ? launch_early(attn_join_kernel<__nv_bfloat16, 64>, grid, kJoinThreads, 0, s, a)
             : a.d.D == 128 ? launch_early(attn_join_kernel<__nv_bfloat16, 128>, grid, kJoinThreads, 0, s, a)
                            : launch_early(attn_join_kernel<__nv_bfloat16, 256>, grid, kJoinThreads, 0, s, a);
    return a.d.D == 64 ? launch_early(attn_join_kernel<float, 64>, grid, kJoinThreads, 0, s, a)
         : a.d.D == 128 ? launch_early(attn_join_kernel<float, 128>, grid, kJoinThreads, 0, s, a)
                        : launch_early(attn_join_kernel<float, 256>, grid, kJoinThreads, 0, s, a);
}

// bf16: where 16 query rows hold all of a key head's, their products keep up with the memory and a call's ends are short: against
// the kernel of many rows one sequence of 700 tokens, 8 rows takes 8.2 us to 12.3, one of 131,072, 2 key heads of 256 columns, 8 rows
// 49.2 to 55.0, 32 of up to 8,192, 16 rows 52.4 to 54.2; only where a large batch has few rows is this one slower (64 of up to 16,384
// tokens, 8 key heads, 4 rows: 348 to 338, floor 339).  Above 16 rows it would read each tile again.
cudaError_t launch_attn_decode(const AttnDecodeArgs &a, bool act_bf16, cudaStream_t s) {
    if (!act_bf16) return a.d.D == 64 ? run_rows<64>(a, s) : a.d.D == 128 ? run_rows<128>(a, s) : run_rows<256>(a, s);
    return a.d.grp * a.tokens <= 16 ? launch_attn_decode_tc(a, s) : launch_attn_decode_rows(a, s);
}

}  // namespace gdn
