// block_norm.cu -- the norms around a block of a residual stream, fused with
// the block's gate and the residual scale, and their gradients.
//
//   n  = p rstd(p) w1            rstd(v) = 1 / sqrt(mean(v^2) + eps)
//   r' = r + s sigmoid(gate) n
//   h  = r' rstd(r') w2
//
// One pass over the rows: p, gate and r are read once, r' and h written once,
// and the row lives in registers between its two sums.  HBM-bound.  A row
// belongs to a warp (short rows) or to a CTA; CTAs walk the rows in a grid
// stride, which keeps the weights in registers and lets the loads of the next
// row be issued before the sums of this one.
#include "ssm_common.cuh"

namespace gdn {

namespace {

constexpr int kWarpRows = 4;       // rows of a CTA where a warp owns a row

// Eight values of a row as the memory holds them.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void from(const unsigned char *p, bool in) {
        a = b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in) { a = load4f((const float *)p); b = load4f((const float *)p + 4); }
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void from(const unsigned char *p, bool in) {
        u = in ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const float4 a = bf16x4_f32(make_uint2(u.x, u.y)), b = bf16x4_f32(make_uint2(u.z, u.w));
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// A thread's chunk i of a row: with VEC 8 neighbours from one or two vector
// loads, otherwise 8 elements NT apart (every load of a warp contiguous).
template <bool VEC> struct Chunk {
    // elements past the row's end read as zero and add nothing to its sums
    int base, dim, stride;
    __device__ __forceinline__ Chunk(int i, int lane, int nt, int dim_) : dim(dim_) {
        base = VEC ? (i * nt + lane) * 8 : i * nt * 8 + lane;
        stride = VEC ? 1 : nt;
    }
    __device__ __forceinline__ bool in(int j) const { return VEC ? base < dim : base + j * stride < dim; }
    __device__ __forceinline__ int at(int j) const { return base + j * stride; }
};

template <bool VEC, typename C> __device__ __forceinline__ void load_raw(const C &c, const float *p, Raw8<float> &r) {
    if (VEC) {
        if (c.in(0)) { r.a = load4f(p + c.base); r.b = load4f(p + c.base + 4); }
        else { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }
    } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c.in(j) ? p[c.at(j)] : 0.f;
        r.a = make_float4(v[0], v[1], v[2], v[3]);
        r.b = make_float4(v[4], v[5], v[6], v[7]);
    }
}
template <bool VEC, typename C>
__device__ __forceinline__ void load_raw(const C &c, const __nv_bfloat16 *p, Raw8<__nv_bfloat16> &r) {
    if (VEC) {
        r.u = c.in(0) ? *reinterpret_cast<const uint4 *>(p + c.base) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        unsigned v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = c.in(j) ? (unsigned)__bfloat16_as_ushort(p[c.at(j)]) : 0u;
        r.u = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
}
template <bool VEC, typename C> __device__ __forceinline__ void store8v(const C &c, float *p, const float (&v)[8]) {
    if (VEC) {
        if (c.in(0)) {
            store4f(p + c.base, make_float4(v[0], v[1], v[2], v[3]));
            store4f(p + c.base + 4, make_float4(v[4], v[5], v[6], v[7]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.in(j)) p[c.at(j)] = v[j];
    }
}
template <bool VEC, typename C>
__device__ __forceinline__ void store8v(const C &c, __nv_bfloat16 *p, const float (&v)[8]) {
    if (VEC) {
        if (c.in(0)) {
            __nv_bfloat162 h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4 *>(p + c.base) = *reinterpret_cast<const uint4 *>(h);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.in(j)) p[c.at(j)] = __float2bfloat16_rn(v[j]);
    }
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// Sum over the threads of a row; every thread gets it.  `buf` holds a value per
// warp, twice: successive sums take turns (`turn`), so that one barrier per sum
// is enough: a half is written again only after the other half's barrier.
template <bool WARP> __device__ __forceinline__ float2 row_sum2(float2 v, float2 (*buf)[32], int &turn) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (WARP) return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float2 *half = buf[turn];
    turn ^= 1;
    if (lane == 0) half[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 u = lane < warps ? half[lane] : make_float2(0.f, 0.f);
    u.x = warp_sum(u.x);
    u.y = warp_sum(u.y);
    return u;
}
template <bool WARP> __device__ __forceinline__ float row_sum(float v, float2 (*buf)[32], int &turn) {
    v = warp_sum(v);
    if (WARP) return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float2 *half = buf[turn];
    turn ^= 1;
    if (lane == 0) half[threadIdx.x >> 5].x = v;
    __syncthreads();
    return warp_sum(lane < warps ? half[lane].x : 0.f);
}

}  // namespace

// Blocks of MAXT threads at most, 512 threads on an SM and so 128 registers each.  Rows that need
// 1,024 threads leave 64 registers a thread: the forward kernel then reads the weights at every
// row (from L1) and does not load ahead (LEAN).
constexpr int sm_blocks(int maxt) { return maxt >= 512 ? 1 : 512 / maxt; }

template <typename TA, typename TR, int NV, int MAXT, bool WARP, bool VEC>
__global__ void __launch_bounds__(MAXT, sm_blocks(MAXT)) block_norm_kernel(NormArgs a) {
    __shared__ float2 buf[2][32];
    int turn = 0;
    using Ch = Chunk<VEC>;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const long long first = WARP ? blockIdx.x * (long long)kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const long long step = WARP ? gridDim.x * (long long)kWarpRows : gridDim.x;
    const float inv_dim = 1.0f / (float)a.dim;
    const bool channel_gate = a.gate && a.gate_cols > 1, row_gate = a.gate && a.gate_cols == 1;

    constexpr bool LEAN = MAXT == 1024;
    float w1[NV][8], w2[NV][8];
    auto weight = [&](const float *w, int i, float (&v)[8]) {
        Raw8<float> r;
        load_raw<VEC>(Ch(i, lane, nt, a.dim), w, r);
        r.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += a.offset;
    };
    if (!LEAN) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (a.w_post) weight(a.w_post, i, w1[i]);
            if (a.w_pre) weight(a.w_pre, i, w2[i]);
        }
    }
    Raw8<TA> rp[NV], rg[NV];
    Raw8<TR> rr[NV];
    float gate1 = 0.f;
    auto fetch = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Ch c(i, lane, nt, a.dim);
            if (a.block) load_raw<VEC>(c, (const TA *)a.block + row * a.ld_block, rp[i]);
            if (channel_gate) load_raw<VEC>(c, (const TA *)a.gate + row * a.ld_gate, rg[i]);
            load_raw<VEC>(c, (const TR *)a.residual + row * a.ld_res, rr[i]);
        }
        if (row_gate) gate1 = to_f32(((const TA *)a.gate)[row * a.ld_gate]);
    };
    if (!LEAN && first < a.rows) fetch(first);
    for (long long row = first; row < a.rows; row += step) {
        if (LEAN) fetch(row);
        float u[NV][8], p[NV][8], gt[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            rr[i].get(u[i]);
            if (a.block) rp[i].get(p[i]);
            if (channel_gate) rg[i].get(gt[i]);
        }
        const float g1 = gate1;
        if (!LEAN && row + step < a.rows) fetch(row + step);
        if (a.block) {
            float k = 1.0f;
            if (a.w_post) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(p[i][j], p[i][j], ss);
                ss = row_sum<WARP>(ss, buf, turn);
                k = 1.0f / sqrtf(fmaf(ss, inv_dim, a.eps));
                if (a.rstd_post && lane == 0) a.rstd_post[row] = k;
            }
            const float rs = a.scale * (row_gate ? sigmoid_f(g1) : 1.0f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (LEAN && a.w_post) weight(a.w_post, i, w1[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = a.w_post ? p[i][j] * k * w1[i][j] : p[i][j];
                    if (channel_gate) v *= sigmoid_for<TA>(gt[i][j]);
                    u[i][j] = fmaf(rs, v, u[i][j]);
                }
            }
            if (a.res_out) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    store8v<VEC>(Ch(i, lane, nt, a.dim), (TR *)a.res_out + row * a.ld_out, u[i]);
            }
        }
        if (a.w_pre) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(u[i][j], u[i][j], ss);
            ss = row_sum<WARP>(ss, buf, turn);
            const float k = 1.0f / sqrtf(fmaf(ss, inv_dim, a.eps));
            if (a.rstd_pre && lane == 0) a.rstd_pre[row] = k;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[8];
                if (LEAN) weight(a.w_pre, i, w2[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = u[i][j] * k * w2[i][j];
                store8v<VEC>(Ch(i, lane, nt, a.dim), (TA *)a.h + row * a.ld_h, v);
            }
        }
    }
}

// Shared memory for two rows' operands, 0 where that is more than an SM has.
template <typename TA, typename TR, int NV, bool VEC> constexpr int stage_bytes(int threads) {
    const int bytes = 2 * NV * (3 * (int)sizeof(Raw8<TA>) + 2 * (int)sizeof(Raw8<TR>)) * threads;
    return VEC && bytes <= 224 * 1024 ? bytes : 0;
}

// The gradients, from the kept r', rstd(p) and rstd(r'); p^ = p rstd(p), r^ = r' rstd(r'):
//   du    = d_r' + rstd(r') (dh w2 - r^ mean(dh w2 r^))        (d_r of the residual input)
//   dn    = s sigmoid(gate) du,  d_gate = s du n sigmoid' (summed over the row for a gate per row)
//   dp    = rstd(p) (dn w1 - p^ mean(dn w1 p^))
//   dw1   = sum over rows of dn p^,  dw2 = sum over rows of dh r^
// The weight gradients are summed in registers over a CTA's rows, then over the
// CTAs by norm_weight_grad_kernel, always in the same order.
template <typename TA, typename TR, int NV, int MAXT, bool WARP, bool VEC>
__global__ void __launch_bounds__(MAXT, sm_blocks(MAXT)) block_norm_bwd_kernel(NormArgs a) {
    __shared__ float2 buf[2][32];
    int turn = 0;
    using Ch = Chunk<VEC>;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const long long first = WARP ? blockIdx.x * (long long)kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const long long step = WARP ? gridDim.x * (long long)kWarpRows : gridDim.x;
    const float inv_dim = 1.0f / (float)a.dim;
    const bool channel_gate = a.gate && a.gate_cols > 1, row_gate = a.gate && a.gate_cols == 1;
    float dw1[NV][8], dw2[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw1[i][j] = dw2[i][j] = 0.f;

    // The five operands of the next row come into shared memory while this one is computed: every
    // thread copies and reads its own 16- or 32-byte pieces, so no barrier is needed.  (Rows whose
    // two stages do not fit, or of single elements, are loaded when their turn comes.)
    constexpr int EA = sizeof(Raw8<TA>), ER = sizeof(Raw8<TR>);
    constexpr bool AHEAD = stage_bytes<TA, TR, NV, VEC>(MAXT) > 0;
    extern __shared__ __align__(16) unsigned char stage[];
    // piece i of operand k (dh, block, gate, then r', d_r') in stage s
    auto piece = [&](int s, int k, int i) {
        return stage + ((s * NV + i) * (3 * EA + 2 * ER) + (k < 3 ? k * EA : 3 * EA + (k - 3) * ER)) * blockDim.x +
               threadIdx.x * (k < 3 ? EA : ER);
    };
    auto ahead = [&](long long row, int s) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Ch c(i, lane, nt, a.dim);
            if (row >= a.rows || !c.in(0)) continue;
            auto copy = [&](int k, const void *p, long long ld, int bytes) {
                const char *src = (const char *)p + (row * ld + c.base) * (bytes / 8);
#pragma unroll
                for (int q = 0; q < bytes; q += 16) cp_async16(piece(s, k, i) + q, src + q);
            };
            if (a.dh) { copy(0, a.dh, a.ld_dh, EA); copy(3, a.residual, a.ld_res, ER); }
            if (a.block) copy(1, a.block, a.ld_block, EA);
            if (channel_gate) copy(2, a.gate, a.ld_gate, EA);
            if (a.d_res_out) copy(4, a.d_res_out, a.ld_dout, ER);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (AHEAD) ahead(first, 0);
    int turn_row = 0;
    for (long long row = first; row < a.rows; row += step, turn_row ^= 1) {
        Raw8<TA> rp[NV], rg[NV], rh[NV];
        Raw8<TR> ru[NV], rd[NV];
        if (AHEAD) {
            ahead(row + step, turn_row ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Ch c(i, lane, nt, a.dim);
                if (a.dh) {
                    load_raw<VEC>(c, (const TA *)a.dh + row * a.ld_dh, rh[i]);
                    load_raw<VEC>(c, (const TR *)a.residual + row * a.ld_res, ru[i]);
                }
                if (a.d_res_out) load_raw<VEC>(c, (const TR *)a.d_res_out + row * a.ld_dout, rd[i]);
                if (a.block) load_raw<VEC>(c, (const TA *)a.block + row * a.ld_block, rp[i]);
                if (channel_gate) load_raw<VEC>(c, (const TA *)a.gate + row * a.ld_gate, rg[i]);
            }
        }
        float du[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (a.d_res_out) {
                if (AHEAD) rd[i].from(piece(turn_row, 4, i), Ch(i, lane, nt, a.dim).in(0));
                rd[i].get(du[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) du[i][j] = 0.f;
            }
        }
        if (a.dh) {
            const float k = a.k_pre[row];
            float g[NV][8], uh[NV][8], dot = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Ch c(i, lane, nt, a.dim);
                Raw8<float> rw;
                float w[8];
                load_raw<VEC>(c, a.w_pre, rw);
                rw.get(w);
                if (AHEAD) {
                    rh[i].from(piece(turn_row, 0, i), Ch(i, lane, nt, a.dim).in(0));
                    ru[i].from(piece(turn_row, 3, i), Ch(i, lane, nt, a.dim).in(0));
                }
                rh[i].get(g[i]);
                ru[i].get(uh[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uh[i][j] *= k;
                    dw2[i][j] = fmaf(g[i][j], uh[i][j], dw2[i][j]);
                    g[i][j] *= w[j] + a.offset;
                    dot = fmaf(g[i][j], uh[i][j], dot);
                }
            }
            const float m = row_sum<WARP>(dot, buf, turn) * inv_dim;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) du[i][j] = fmaf(k, g[i][j] - uh[i][j] * m, du[i][j]);
        }
        if (a.d_res) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                store8v<VEC>(Ch(i, lane, nt, a.dim), (TR *)a.d_res + row * a.ld_dres, du[i]);
        }
        if (a.block) {
            const float k = a.w_post ? a.k_post[row] : 1.0f;
            float s1 = 1.0f, q1 = 0.f;
            if (row_gate) sigmoid_pair<float>(to_f32(((const TA *)a.gate)[row * a.ld_gate]), s1, q1);
            float2 sums = make_float2(0.f, 0.f);      // sum of dn w1 p^, sum of the row gate's gradient
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const Ch c(i, lane, nt, a.dim);
                float ph[8], gt[8], w[8];
                if (AHEAD) {
                    rp[i].from(piece(turn_row, 1, i), Ch(i, lane, nt, a.dim).in(0));
                    if (channel_gate) rg[i].from(piece(turn_row, 2, i), Ch(i, lane, nt, a.dim).in(0));
                }
                rp[i].get(ph);
                if (channel_gate) rg[i].get(gt);
                if (a.w_post) {
                    Raw8<float> rw;
                    load_raw<VEC>(c, a.w_post, rw);
                    rw.get(w);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float wj = a.w_post ? w[j] + a.offset : 1.0f;
                    ph[j] *= k;
                    float sg = s1, rest = q1;
                    if (channel_gate) sigmoid_pair<TA>(gt[j], sg, rest);
                    const float dn = a.scale * du[i][j] * sg;
                    if (a.gate) {
                        gt[j] = dn * rest * ph[j] * wj;
                        sums.y += gt[j];
                    }
                    dw1[i][j] = fmaf(dn, ph[j], dw1[i][j]);
                    du[i][j] = dn * wj;               // du becomes the gradient of p^
                    sums.x = fmaf(du[i][j], ph[j], sums.x);
                }
                if (channel_gate && a.d_gate) store8v<VEC>(c, (TA *)a.d_gate + row * a.ld_dgate, gt);
            }
            if (a.w_post || row_gate) sums = row_sum2<WARP>(sums, buf, turn);
            if (row_gate && a.d_gate && lane == 0) ((TA *)a.d_gate)[row * a.ld_dgate] = from_f32<TA>(sums.y);
            if (a.d_block) {
                const float m = a.w_post ? sums.x * inv_dim : 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float ph[8], v[8];
                    if (AHEAD) rp[i].from(piece(turn_row, 1, i), Ch(i, lane, nt, a.dim).in(0));
                    rp[i].get(ph);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = a.w_post ? k * (du[i][j] - ph[j] * k * m) : du[i][j];
                    store8v<VEC>(Ch(i, lane, nt, a.dim), (TA *)a.d_block + row * a.ld_dblock, v);
                }
            }
        }
    }
    let_next_start();
    if (!a.ws) return;
    // this CTA's (or warp's) part of the weight gradients: [2][dim]
    const long long part = WARP ? blockIdx.x * (long long)kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    float *to = a.ws + part * 2 * a.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Ch c(i, lane, nt, a.dim);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.in(j)) {
                to[c.at(j)] = dw1[i][j];
                to[a.dim + c.at(j)] = dw2[i][j];
            }
    }
}

// dw[c] = sum over the parts, 32 columns of one weight per CTA: 32 threads down
// the parts for each column, then a sum over those 32.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float *ws, int parts, int dim,
                                                                float *dw_post, float *dw_pre) {
    __shared__ float s[32][33];
    await_previous();
    float *dw = blockIdx.y == 0 ? dw_post : dw_pre;
    if (!dw) return;
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
    float v = 0.f;
    if (col < dim)
        for (int k = r; k < parts; k += 32) v += ws[((long long)k * 2 + blockIdx.y) * dim + col];
    s[threadIdx.x & 31][r] = v;
    __syncthreads();
    v = warp_sum(s[r][threadIdx.x & 31]);
    if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + r < dim) dw[blockIdx.x * 32 + r] = v;
}

namespace {

// A warp owns a row of up to 512 elements, a CTA a longer one; a thread has 8 or 16 elements (with
// 8 alone the sums over a CTA's warps took a third of the instructions: 8,192 x 4,096 forward 63 us).
bool warp_rows(int dim) { return dim <= 512; }
int row_threads(int dim) { return warp_rows(dim) ? 32 * kWarpRows : ((dim + 15) / 16 + 31) / 32 * 32; }

// CTAs of the backward, and so the parts of the weight gradients.
int bwd_ctas(long long rows, int dim) {
    const int threads = row_threads(dim);
    const long long cap = (long long)sm_count() * (threads < 512 ? 512 / threads : 1);
    const long long want = warp_rows(dim) ? (rows + kWarpRows - 1) / kWarpRows : rows;
    return (int)(want < cap ? want : cap);
}

template <typename TA, typename TR, int NV, int MAXT, bool WARP, bool VEC>
cudaError_t run(const NormArgs &a, bool backward, cudaStream_t s) {
    const int threads = row_threads(a.dim);
    if (backward) {
        auto kern = block_norm_bwd_kernel<TA, TR, NV, MAXT, WARP, VEC>;
        const int smem = stage_bytes<TA, TR, NV, VEC>(MAXT) > 0 ? stage_bytes<TA, TR, NV, VEC>(threads) : 0;
        if (smem > 0) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        kern<<<bwd_ctas(a.rows, a.dim), threads, smem, s>>>(a);
    } else {
        const long long cap = (long long)sm_count() * (threads < 1024 ? 1024 / threads : 1);
        const long long want = WARP ? (a.rows + kWarpRows - 1) / kWarpRows : a.rows;
        block_norm_kernel<TA, TR, NV, MAXT, WARP, VEC><<<(unsigned)(want < cap ? want : cap), threads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename TA, typename TR, bool VEC> cudaError_t run_dim(const NormArgs &a, bool backward, cudaStream_t s) {
    if (a.dim <= 256) return run<TA, TR, 1, 32 * kWarpRows, true, VEC>(a, backward, s);
    if (warp_rows(a.dim)) return run<TA, TR, 2, 32 * kWarpRows, true, VEC>(a, backward, s);
    if (a.dim <= 4096) return run<TA, TR, 2, 256, false, VEC>(a, backward, s);
    if (a.dim <= 8192) return run<TA, TR, 2, 512, false, VEC>(a, backward, s);
    return run<TA, TR, 2, 1024, false, VEC>(a, backward, s);
}

template <bool VEC> cudaError_t run_types(const NormArgs &a, bool backward, cudaStream_t s) {
    if (!a.act_bf16) return run_dim<float, float, VEC>(a, backward, s);
    if (a.res_bf16) return run_dim<__nv_bfloat16, __nv_bfloat16, VEC>(a, backward, s);
    return run_dim<__nv_bfloat16, float, VEC>(a, backward, s);
}

}  // namespace

size_t norm_bwd_ws_bytes(long long rows, int dim) {
    return (size_t)bwd_ctas(rows, dim) * (warp_rows(dim) ? kWarpRows : 1) * 2 * dim * 4;
}

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s) {
    return a.vec ? run_types<true>(a, false, s) : run_types<false>(a, false, s);
}

cudaError_t launch_block_norm_backward(const NormArgs &a, cudaStream_t s) {
    if (a.rows > 0) {
        const cudaError_t e = a.vec ? run_types<true>(a, true, s) : run_types<false>(a, true, s);
        if (e != cudaSuccess) return e;
    }
    if (!a.dw_post && !a.dw_pre) return cudaSuccess;
    const int parts = a.rows > 0 ? bwd_ctas(a.rows, a.dim) * (warp_rows(a.dim) ? kWarpRows : 1) : 0;
    return launch_early(norm_weight_grad_kernel, dim3((a.dim + 31) / 32, 2), 1024, 0, s, (const float *)a.ws, parts, a.dim,
                        a.dw_post, a.dw_pre);
}

}  // namespace gdn
