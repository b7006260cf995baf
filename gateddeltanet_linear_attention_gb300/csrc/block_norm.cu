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
// row be issued before the sums of this one.  8,192 x 4,096 bf16 with a gate per
// channel: 59.5 us, 5.6 TB/s, 0.83 of a plain copy's rate.  Rows of single elements
// (odd widths, views off 16 bytes) are bound by their load and store instructions:
// 2^25 elements at 1,001 wide take 152 us, 2.2 TB/s.
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

// Eight values as four pairs for the packed multiply-adds.
template <typename R> __device__ __forceinline__ void get_pairs(const R &r, f32x2 (&v)[4]) {
    float f[8];
    r.get(f);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack2(f[2 * j], f[2 * j + 1]);
}
__device__ __forceinline__ f32x2 both(float x) { return pack2(x, x); }

// A thread's chunk i of a row: with VEC 8 neighbours from one or two vector
// loads, otherwise 8 elements 32 apart in its warp's NV x 256 (every load of a
// warp contiguous, at a constant distance from the one before).
template <bool VEC, int NV> struct Chunk {
    // elements past the row's end read as zero and add nothing to its sums
    static constexpr int stride = VEC ? 1 : 32;
    int base, dim;
    __device__ __forceinline__ Chunk(int i, int lane, int nt, int dim_) : dim(dim_) {
        base = VEC ? (i * nt + lane) * 8 : ((lane >> 5) * NV + i) * 256 + (lane & 31);
    }
    __device__ __forceinline__ bool in(int j) const { return VEC ? base < dim : base + j * stride < dim; }
    __device__ __forceinline__ int at(int j) const { return base + j * stride; }
    __device__ __forceinline__ bool whole() const { return in(7); }     // all 8 in the row: one test for them
};

template <bool VEC, typename C> __device__ __forceinline__ void load_raw(const C &c, const float *p, Raw8<float> &r) {
    if (VEC) {
        if (c.in(0)) { r.a = load4f(p + c.base); r.b = load4f(p + c.base + 4); }
        else { r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f); }
    } else {
        float v[8];
        if (c.whole()) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = p[c.at(j)];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = c.in(j) ? p[c.at(j)] : 0.f;
        }
        r.a = make_float4(v[0], v[1], v[2], v[3]);
        r.b = make_float4(v[4], v[5], v[6], v[7]);
    }
}
template <bool VEC, typename C>
__device__ __forceinline__ void load_raw(const C &c, const __nv_bfloat16 *p, Raw8<__nv_bfloat16> &r) {
    if (VEC) {
        r.u = c.in(0) ? *reinterpret_cast<const uint4 *>(p + c.base) : make_uint4(0u, 0u, 0u, 0u);
    } else {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
        unsigned v[8];
        if (c.whole()) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = q[c.at(j)];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = c.in(j) ? (unsigned)q[c.at(j)] : 0u;
        }
        r.u = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
}
template <bool VEC, typename C> __device__ __forceinline__ void store8v(const C &c, float *p, const float (&v)[8]) {
    if (VEC) {
        if (c.in(0)) {
            store4f(p + c.base, make_float4(v[0], v[1], v[2], v[3]));
            store4f(p + c.base + 4, make_float4(v[4], v[5], v[6], v[7]));
        }
    } else if (c.whole()) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[c.at(j)] = v[j];
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
    } else if (c.whole()) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[c.at(j)] = __float2bfloat16_rn(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.in(j)) p[c.at(j)] = __float2bfloat16_rn(v[j]);
    }
}

// The sigmoid of a gate of type TA in a result of type TR.  A 16-bit gate's in a 32-bit one: x times
// 16 bits of log2(e) is exact, and the rest of log2(e) a factor 1 - 4.9e-6 x behind the exponential, so the
// error does not grow with |x| (below 10 half steps up to 70; the factor stops changing where the
// exponential is nothing, so that a gate of +inf is 1).  2^25 elements with a gate per channel, 4,096 and
// 5,120 wide: 87 and 104 us, with the 16-bit results' sigmoid 87 and 103, with the accurate one 103 and 134.
template <typename TA, typename TR> __device__ __forceinline__ float gate_sigmoid(float x) { return sigmoid_for<TR>(x); }
template <> __device__ __forceinline__ float gate_sigmoid<__nv_bfloat16, float>(float x) {
    const float e = exp2_fast(-1.44268798828125f * x);
    return rcp_fast(1.0f + fmaf(e, -4.8884952e-6f * fminf(x, 128.f), e));
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// Sum over the threads of a row; every thread gets it.  `buf` holds a value per
// warp, twice: successive sums take turns (`turn`), so that one barrier per sum
// is enough: a half is written again only after the other half's barrier.
template <bool WARP> __device__ __forceinline__ float row_sum(float v, float (*buf)[32], int &turn) {
    v = warp_sum(v);
    if (WARP) return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float *half = buf[turn];
    turn ^= 1;
    if (lane == 0) half[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? half[lane] : 0.f);
}

}  // namespace

// Blocks of MAXT threads at most, in the forward kernel with the registers to keep the weights and
// to load a row ahead of the one that is computed (KEEP, AHEAD).
constexpr int sm_blocks(int maxt) { return maxt >= 512 ? 1 : 512 / maxt; }

template <typename TA, typename TR, int NV, int MAXT, bool WARP, bool VEC>
__global__ void __launch_bounds__(MAXT, sm_blocks(MAXT)) block_norm_kernel(NormArgs a) {
    __shared__ float buf[2][32];
    int turn = 0;
    using Ch = Chunk<VEC, NV>;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const long long first = WARP ? blockIdx.x * (long long)kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const long long step = WARP ? gridDim.x * (long long)kWarpRows : gridDim.x;
    const float inv_dim = 1.0f / (float)a.dim;
    const bool channel_gate = a.gate && a.gate_cols > 1, row_gate = a.gate && a.gate_cols == 1;

    constexpr bool AHEAD = VEC && MAXT < 1024, KEEP = AHEAD;
    float w1[NV][8], w2[NV][8];
    auto weight = [&](const float *w, int i, float (&v)[8]) {
        Raw8<float> r;
        load_raw<VEC>(Ch(i, lane, nt, a.dim), w, r);
        r.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += a.offset;
    };
    if (KEEP) {
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
    if (AHEAD && first < a.rows) fetch(first);
    for (long long row = first; row < a.rows; row += step) {
        if (!AHEAD) fetch(row);
        float u[NV][8], p[NV][8], gt[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            rr[i].get(u[i]);
            if (a.block) rp[i].get(p[i]);
            if (channel_gate) rg[i].get(gt[i]);
        }
        const float g1 = gate1;
        if (AHEAD && row + step < a.rows) fetch(row + step);
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
                if (!KEEP && a.w_post) weight(a.w_post, i, w1[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = a.w_post ? p[i][j] * k * w1[i][j] : p[i][j];
                    if (channel_gate) v *= gate_sigmoid<TA, TR>(gt[i][j]);
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
                if (!KEEP) weight(a.w_pre, i, w2[i]);
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
// 8,192 x 4,096 bf16 with a gate per channel: 117 us with the sum over CTAs (7 us alone), 4.6 TB/s.
// Half of the issue slots are used (61 instructions an element in packed arithmetic, 96 without:
// 132 us); 512 threads of 122 registers fill an SM, and two rows' chains of sums are too few to hide
// each other's barriers.  All sums of a row behind one barrier, with more arithmetic: 134 us.
// Rows wider than 8,192 spill (64 registers): 12,288 wide 325 us for 2^25 elements.
template <typename TA, typename TR, int NV, int MAXT, bool WARP, bool VEC>
__global__ void __launch_bounds__(MAXT, sm_blocks(MAXT)) block_norm_bwd_kernel(NormArgs a) {
    __shared__ float buf[2][32];
    int turn = 0;
    using Ch = Chunk<VEC, NV>;
    const int lane = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const long long first = WARP ? blockIdx.x * (long long)kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    const long long step = WARP ? gridDim.x * (long long)kWarpRows : gridDim.x;
    const float inv_dim = 1.0f / (float)a.dim;
    const bool channel_gate = a.gate && a.gate_cols > 1, row_gate = a.gate && a.gate_cols == 1;
    f32x2 dw1[NV][4], dw2[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw1[i][j] = dw2[i][j] = 0ull;
    // piece i of a weight with its offset, 1 where there is none
    auto weight = [&](const float *w, int i, f32x2 (&v)[4]) {
        if (w) {
            Raw8<float> r;
            load_raw<VEC>(Ch(i, lane, nt, a.dim), w, r);
            get_pairs(r, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = add2(v[j], both(a.offset));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = both(1.0f);
        }
    };
    auto store_act = [&](void *p, long long ld, long long row, int i, const f32x2 (&v)[4]) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 q = unpack2(v[j]);
            f[2 * j] = q.x;
            f[2 * j + 1] = q.y;
        }
        store8v<VEC>(Ch(i, lane, nt, a.dim), (TA *)p + row * ld, f);
    };

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
    // the next row's factors, loaded a row ahead
    float n1 = 1.0f, n2 = 0.f, ng = 0.f;
    auto factors = [&](long long row) {
        if (row >= a.rows) return;
        if (a.w_post) n1 = a.k_post[row];
        if (a.dh) n2 = a.k_pre[row];
        if (row_gate) ng = to_f32(((const TA *)a.gate)[row * a.ld_gate]);
    };
    factors(first);
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
        const float k1 = n1, k2 = n2;
        float s1 = 1.0f, q1 = 0.f;
        if (row_gate) sigmoid_pair(ng, s1, q1);
        factors(row + step);
        f32x2 du[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (a.d_res_out) {
                if (AHEAD) rd[i].from(piece(turn_row, 4, i), Ch(i, lane, nt, a.dim).in(0));
                get_pairs(rd[i], du[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) du[i][j] = 0ull;
            }
        }
        if (a.dh) {
            f32x2 g[NV][4], uh[NV][4], dot = 0ull;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                f32x2 w[4];
                weight(a.w_pre, i, w);
                if (AHEAD) {
                    rh[i].from(piece(turn_row, 0, i), Ch(i, lane, nt, a.dim).in(0));
                    ru[i].from(piece(turn_row, 3, i), Ch(i, lane, nt, a.dim).in(0));
                }
                get_pairs(rh[i], g[i]);
                get_pairs(ru[i], uh[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uh[i][j] = mul2(uh[i][j], both(k2));
                    dw2[i][j] = fma2(g[i][j], uh[i][j], dw2[i][j]);
                    g[i][j] = mul2(g[i][j], w[j]);
                    dot = fma2(g[i][j], uh[i][j], dot);
                }
            }
            const float2 sum = unpack2(dot);
            const float m = row_sum<WARP>(sum.x + sum.y, buf, turn) * inv_dim;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) du[i][j] = fma2(both(k2), fma2(both(-m), uh[i][j], g[i][j]), du[i][j]);
        }
        if (a.d_res) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 q = unpack2(du[i][j]);
                    f[2 * j] = q.x;
                    f[2 * j + 1] = q.y;
                }
                store8v<VEC>(Ch(i, lane, nt, a.dim), (TR *)a.d_res + row * a.ld_dres, f);
            }
        }
        if (a.block) {
            f32x2 dot = 0ull;                         // of dn w1 and p^
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                f32x2 ph[4], w[4], sg[4], rest[4];
                if (AHEAD) rp[i].from(piece(turn_row, 1, i), Ch(i, lane, nt, a.dim).in(0));
                get_pairs(rp[i], ph);
                weight(a.w_post, i, w);
                if (channel_gate) {
                    float x[8];
                    if (AHEAD) rg[i].from(piece(turn_row, 2, i), Ch(i, lane, nt, a.dim).in(0));
                    rg[i].get(x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (sizeof(TA) == 2) {
                            sigmoid_pairs_fast(x[2 * j], x[2 * j + 1], sg[j], rest[j]);
                        } else {
                            float s[2], q[2];
                            sigmoid_pair(x[2 * j], s[0], q[0]);
                            sigmoid_pair(x[2 * j + 1], s[1], q[1]);
                            sg[j] = pack2(s[0], s[1]);
                            rest[j] = pack2(q[0], q[1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) sg[j] = both(s1);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ph[j] = mul2(ph[j], both(k1));
                    const f32x2 dn = mul2(mul2(sg[j], both(a.scale)), du[i][j]);
                    dw1[i][j] = fma2(dn, ph[j], dw1[i][j]);
                    du[i][j] = mul2(dn, w[j]);        // du becomes the gradient of p^
                    dot = fma2(du[i][j], ph[j], dot);
                    if (channel_gate) rest[j] = mul2(rest[j], mul2(du[i][j], ph[j]));
                }
                if (channel_gate && a.d_gate) store_act(a.d_gate, a.ld_dgate, row, i, rest);
            }
            const float2 sum2 = unpack2(dot);
            float sum = sum2.x + sum2.y;
            if (a.w_post || row_gate) sum = row_sum<WARP>(sum, buf, turn);
            // (of a row's one gate: the same sum times 1 - sigmoid)
            if (row_gate && a.d_gate && lane == 0) ((TA *)a.d_gate)[row * a.ld_dgate] = from_f32<TA>(sum * q1);
            if (a.d_block) {
                const float m = a.w_post ? -k1 * k1 * sum * inv_dim : 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    f32x2 p[4];
                    if (AHEAD) rp[i].from(piece(turn_row, 1, i), Ch(i, lane, nt, a.dim).in(0));
                    get_pairs(rp[i], p);
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = fma2(both(m), p[j], mul2(both(k1), du[i][j]));
                    store_act(a.d_block, a.ld_dblock, row, i, p);
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
                const float2 p = unpack2(dw1[i][j / 2]), q = unpack2(dw2[i][j / 2]);
                to[c.at(j)] = j & 1 ? p.y : p.x;
                to[a.dim + c.at(j)] = j & 1 ? q.y : q.x;
            }
    }
}

// dw[c] = sum over the parts, 32 columns of one weight per CTA: 32 threads down
// the parts for each column, then a sum over those 32.  10 MB of parts (304 of 4,096
// columns): 7 us alone, bound by latency, launched while the parts are still written.
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

// A warp owns a row of up to 512 elements, a CTA a longer one; a thread has 8 or 16 elements, see
// fwd_dim and bwd_dim.
bool warp_rows(int dim) { return dim <= 512; }
int row_threads(int dim, int each) { return warp_rows(dim) ? 32 * kWarpRows : ((dim + each - 1) / each + 31) / 32 * 32; }
long long row_ctas(long long rows, int dim) { return warp_rows(dim) ? (rows + kWarpRows - 1) / kWarpRows : rows; }
// Backward CTAs that an SM's registers hold, 512 threads' worth.
int resident(int threads) { return threads < 512 ? 512 / threads : 1; }

template <typename TA, typename TR, int NV, int MAXT, bool WARP, bool VEC>
cudaError_t run_fwd(const NormArgs &a, cudaStream_t s) {
    const int threads = row_threads(a.dim, 8 * NV);
    const long long cap = (long long)sm_count() * (threads < 1024 ? 1024 / threads : 1);
    const long long want = row_ctas(a.rows, a.dim);
    block_norm_kernel<TA, TR, NV, MAXT, WARP, VEC><<<(unsigned)(want < cap ? want : cap), threads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename TA, typename TR, int NV, int MAXT, bool WARP, bool VEC>
cudaError_t run_bwd(const NormArgs &a, cudaStream_t s, int &ctas) {
    const int threads = row_threads(a.dim, 8 * NV);
    auto kern = block_norm_bwd_kernel<TA, TR, NV, MAXT, WARP, VEC>;
    const int smem = stage_bytes<TA, TR, NV, VEC>(MAXT) > 0 ? stage_bytes<TA, TR, NV, VEC>(threads) : 0;
    int per_sm = resident(threads);
    if (smem > 0) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const int fit = 228 * 1024 / (smem + 1280);    // (1,024 bytes that the system keeps, 256 of sums)
        per_sm = per_sm < fit ? per_sm : fit < 1 ? 1 : fit;
    }
    // no more than run at once: a CTA's parts of the weight gradients are written once
    const long long want = row_ctas(a.rows, a.dim), cap = (long long)sm_count() * per_sm;
    ctas = (int)(want < cap ? want : cap);
    kern<<<ctas, threads, smem, s>>>(a);
    return cudaGetLastError();
}

// Threads and elements of a thread by row width (times of 2^25 elements with a gate per channel,
// forward, fp32 unless stated).
// 16 elements: half as many sums over warps (bf16, 4,096 wide: 60 us, with 8 63 us).  With fp32
// operands the next row's loads then spill, and 8 elements are faster: 4,096 wide 127 us, with 16
// 149; 5,120 wide 118, with 16 198 (bf16: 110 and 84).  Rows of single elements keep 16 up to 4,096
// (2,500 wide 133 us, with 8 249).
template <typename TA, typename TR, bool VEC> cudaError_t fwd_dim(const NormArgs &a, cudaStream_t s) {
    constexpr bool kFew = sizeof(TA) == 4;
    if (a.dim <= 256) return run_fwd<TA, TR, 1, 32 * kWarpRows, true, VEC>(a, s);
    if (warp_rows(a.dim)) return run_fwd<TA, TR, 2, 32 * kWarpRows, true, VEC>(a, s);
    if constexpr (kFew && VEC) {
        if (a.dim <= 2048) return run_fwd<TA, TR, 1, 256, false, VEC>(a, s);
        if (a.dim <= 4096) return run_fwd<TA, TR, 1, 512, false, VEC>(a, s);
    } else {
        if (a.dim <= 4096) return run_fwd<TA, TR, 2, 256, false, VEC>(a, s);
    }
    if constexpr (kFew) {
        if (a.dim <= 5120) return run_fwd<TA, TR, 1, 640, false, VEC>(a, s);
        if (a.dim <= 8192) return run_fwd<TA, TR, 1, 1024, false, VEC>(a, s);
    } else {
        if (a.dim <= 8192) return run_fwd<TA, TR, 2, 512, false, VEC>(a, s);
    }
    return run_fwd<TA, TR, 2, 1024, false, VEC>(a, s);
}
// Backward: 16 elements but for rows of 4,097 to 5,120 (8 and 640 threads: 134 us in bf16, with 16
// and 320, 148; at 8,192 wide 138 and 126).
template <typename TA, typename TR, bool VEC> cudaError_t bwd_dim(const NormArgs &a, cudaStream_t s, int &ctas) {
    if (a.dim <= 256) return run_bwd<TA, TR, 1, 32 * kWarpRows, true, VEC>(a, s, ctas);
    if (warp_rows(a.dim)) return run_bwd<TA, TR, 2, 32 * kWarpRows, true, VEC>(a, s, ctas);
    if constexpr (sizeof(TA) == 4 && VEC) {
        if (a.dim > 2048 && a.dim <= 4096) return run_bwd<TA, TR, 1, 512, false, VEC>(a, s, ctas);
    }
    if (a.dim <= 4096) return run_bwd<TA, TR, 2, 256, false, VEC>(a, s, ctas);
    if (a.dim <= 5120) return run_bwd<TA, TR, 1, 640, false, VEC>(a, s, ctas);
    if (a.dim <= 8192) return run_bwd<TA, TR, 2, 512, false, VEC>(a, s, ctas);
    return run_bwd<TA, TR, 2, 1024, false, VEC>(a, s, ctas);
}
template <bool VEC> cudaError_t fwd_types(const NormArgs &a, cudaStream_t s) {
    if (!a.act_bf16) return fwd_dim<float, float, VEC>(a, s);
    if (a.res_bf16) return fwd_dim<__nv_bfloat16, __nv_bfloat16, VEC>(a, s);
    return fwd_dim<__nv_bfloat16, float, VEC>(a, s);
}
template <bool VEC> cudaError_t bwd_types(const NormArgs &a, cudaStream_t s, int &ctas) {
    if (!a.act_bf16) return bwd_dim<float, float, VEC>(a, s, ctas);
    if (a.res_bf16) return bwd_dim<__nv_bfloat16, __nv_bfloat16, VEC>(a, s, ctas);
    return bwd_dim<__nv_bfloat16, float, VEC>(a, s, ctas);
}

}  // namespace

size_t norm_bwd_ws_bytes(long long rows, int dim) {
    // the most CTAs of any type: those of 16 elements a thread
    const long long want = row_ctas(rows, dim), cap = (long long)sm_count() * resident(row_threads(dim, 16));
    return (size_t)(want < cap ? want : cap) * (warp_rows(dim) ? kWarpRows : 1) * 2 * dim * 4;
}

cudaError_t launch_block_norm(const NormArgs &a, cudaStream_t s) {
    return a.vec ? fwd_types<true>(a, s) : fwd_types<false>(a, s);
}

cudaError_t launch_block_norm_backward(const NormArgs &a, cudaStream_t s) {
    int ctas = 0;
    if (a.rows > 0) {
        const cudaError_t e = a.vec ? bwd_types<true>(a, s, ctas) : bwd_types<false>(a, s, ctas);
        if (e != cudaSuccess) return e;
    }
    if (!a.dw_post && !a.dw_pre) return cudaSuccess;
    const int parts = ctas * (warp_rows(a.dim) ? kWarpRows : 1);
    return launch_early(norm_weight_grad_kernel, dim3((a.dim + 31) / 32, 2), 1024, 0, s, (const float *)a.ws, parts, a.dim,
                        a.dw_post, a.dw_pre);
}

}  // namespace gdn
