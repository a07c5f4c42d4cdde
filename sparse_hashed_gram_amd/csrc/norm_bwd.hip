// Backward of the norms (include/norm.h), rows and, in parts, the sums over t
// that the parameters' gradients are made of.  xh is computed again from the row (no
// statistics are kept), so a row is read once and its gradient written once; the sums
// over t stay in registers over all rows of a block, then go through LDS to the block's
// part of the workspace, which one more kernel adds up in a fixed order (5 us).
//
// HBM bounds it at many rows: the norm of 49,152 x 768 takes 102 us of kernel (528 MB,
// 5.2 TB/s), the join with a gate an element 161 us (830 MB, 5.1 TB/s).  4,099 x 1,001 in
// fp32 with all gradients: 32 to 34 us (3.4 to 3.6 TB/s), 4 rows a block at a time and five
// turns of which the last has three rows.
#include <algorithm>

#include "norm_dev.hpp"

namespace rownorm {
namespace {

// q: what turns E into the gradient of the normalised B: gate (not a token's) times post_w
enum { kW, kQ, kScale, kPostW, kPostB, kVectors };

// xh and d -> the gradient in front of the norm over rho: d - [layer] mean(d) - xh mean(d xh).
template <int W, int P>
__device__ __forceinline__ void unnormalise(const float (&xh)[P][4], float (&d)[P][4], int layer, float inv_d,
                                            RowSum<W> &sum)
{
    float c1 = 0.0f, c0 = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c1 = __builtin_fmaf(d[p][k], xh[p][k], c1);
            c0 += d[p][k];
        }
    if (layer) {
        const float2 c = sum(c1, c0);
        c1 = c.x * inv_d;
        c0 = c.y * inv_d;
    } else {
        c1 = sum(c1) * inv_d;
        c0 = 0.0f;
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            d[p][k] = __builtin_fmaf(-xh[p][k], c1, d[p][k] - c0);
}

// A block's sums of a column: those of its rows, then to its part.
template <int W, int P>
__device__ __forceinline__ void put(float (&v)[P][4], const Place<W> &me, int D, float *to,
                                    float (*lds)[P * 256 * W])
{
    if constexpr (kRows<W> > 1) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<float4 *>(&lds[me.row][(p * 64 * W + me.lane) * 4]) =
                make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
        __syncthreads();
        for (int j = threadIdx.x; j < D; j += kThreads) {
            float s = lds[0][j];
#pragma unroll
            for (int i = 1; i < kRows<W>; ++i)
                s += lds[i][j];
            to[j] = s;
        }
        __syncthreads();
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = (p * 64 * W + me.lane) * 4;
            if (e < D)   // parts are padded to whole pieces
                *reinterpret_cast<float4 *>(to + e) = make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
        }
    }
}

template <int XE, int RE, int P, bool FULL, bool JOIN, bool EXTRA>
struct Row {
    Piece<RE> r1[P], d1[P], r[P];
    Piece<XE> dx[P], b[P], g[P];

    __device__ __forceinline__ void load(const Args &a, int64_t row, const int (&e)[P], const int (&n)[P])
    {
        const int64_t at = min(row, a.T - 1) * a.D;
        if (a.pre) {
            load_row<RE, P, FULL>(a.R1in + at * RE, e, n, r1);
            load_row<XE, P, FULL>(a.dX + at * XE, e, n, dx);
        }
        if constexpr (JOIN) {
            load_row<XE, P, FULL>(a.B + at * XE, e, n, b);
            if (a.G)
                load_row<XE, P, FULL>(a.G + at * XE, e, n, g);
        }
        if (a.dR1)
            load_row<RE, P, FULL>(a.dR1 + at * RE, e, n, d1);
        else
#pragma unroll
            for (int p = 0; p < P; ++p)
                d1[p].w = 0;
        if constexpr (JOIN && EXTRA)
            if (a.R)
                load_row<RE, P, FULL>(a.R + at * RE, e, n, r);
    }
};

template <int XE, int RE, int W, int P, bool FULL, bool JOIN, bool EXTRA>
__global__ __launch_bounds__(kThreads) void bwd_kernel(Args a)
{
    constexpr int N = JOIN ? kVectors : 1;
    __shared__ float2 red[2][8];
    __shared__ float params[W == 1 ? N : 1][P * 256];
    __shared__ float lds[kRows<W> > 1 ? kRows<W> : 1][P * 256 * W];
    const Place<W> me;
    const int lane = me.lane;
    RowSum<W> sum{red, me.row};
    ParamRows<W, P, N> par;
    par.lds = params;
    int e[P], n[P];
    float sum_pre[P][4] = {}, sum_post[P][4] = {}, sum_preb[P][4] = {}, sum_post0[P][4] = {}, sum_s[P][4] = {};
#pragma unroll
    for (int p = 0; p < P; ++p) {
        e[p] = (p * 64 * W + lane) * 4;
        n[p] = max(0, min(4, a.D - e[p]));
    }
    const int64_t step = (int64_t)gridDim.x * kRows<W>;
    int64_t row = (int64_t)blockIdx.x * kRows<W> + me.row, first = (int64_t)blockIdx.x * kRows<W>;
    Row<XE, RE, P, FULL, JOIN, EXTRA> next;
    next.load(a, row, e, n);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (W == 1 && me.row != i)   // a wavefront a vector
            continue;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float v[4];
            if (i == kW) {
                load_param(a.p.w, a.p.f32, 0, e[p], n[p], 1.0f, v);
            } else if (i == kScale) {
                load_param(a.p.scale, a.p.f32, a.p.scale_one, e[p], n[p], 1.0f, v);
            } else if (i == kPostB) {
                load_param(a.p.post_b, a.p.f32, 0, e[p], n[p], 0.0f, v);
            } else {
                load_param(a.p.post_w, a.p.f32, 0, e[p], n[p], 1.0f, v);
                if (i == kQ) {
                    float g[4];
                    load_param(a.G ? nullptr : a.p.gate, a.p.f32, a.p.gate_one, e[p], n[p], 1.0f, g);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[k] *= g[k];
                }
            }
            par.put(i, p, lane, v);
        }
    }
    if constexpr (W == 1)
        __syncthreads();
    // every wavefront of the block takes as many turns: one without a row takes the last
    // again, stores nothing and adds zeros
    for (; first < a.T; first += step, row += step) {
        const bool there = row < a.T;
        if (W == 1 && !there)
            break;
        const Row<XE, RE, P, FULL, JOIN, EXTRA> cur = next;
        next.load(a, row + step, e, n);
        const int64_t at = row * a.D;
        float d[P][4];   // E
        if (a.pre) {
            float x[P][4];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                unpack<RE>(cur.r1[p], x[p]);
                unpack<XE>(cur.dx[p], d[p]);
                if (W > 1 && !there)
                    d[p][0] = d[p][1] = d[p][2] = d[p][3] = 0.0f;
            }
            const float rho = normalise<W, P, FULL>(x, n, a.layer, a.inv_d, a.eps, sum);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float w[4];
                par.get(kW, p, lane, w);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sum_pre[p][k] = __builtin_fmaf(d[p][k], x[p][k], sum_pre[p][k]);
                    if constexpr (EXTRA)
                        sum_preb[p][k] += d[p][k];
                    d[p][k] *= w[k];
                }
            }
            unnormalise<W, P>(x, d, a.layer, a.inv_d, sum);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float r[4];
                unpack<RE>(cur.d1[p], r);
                if (W > 1 && !there)
                    r[0] = r[1] = r[2] = r[3] = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    d[p][k] = FULL || k < n[p] ? __builtin_fmaf(rho, d[p][k], r[k]) : 0.0f;
            }
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                unpack<RE>(cur.d1[p], d[p]);
                if (W > 1 && !there)
                    d[p][0] = d[p][1] = d[p][2] = d[p][3] = 0.0f;
            }
        }
        if constexpr (!JOIN) {
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (there)
                    store4<RE, FULL>(a.dR + at * RE + (uint32_t)(e[p] * RE), n[p], d[p]);
        } else {
            float v[P][4];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float o[4];
                if constexpr (EXTRA) {
                    if (a.R) {
                        unpack<RE>(cur.r[p], o);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sum_s[p][k] = __builtin_fmaf(d[p][k], o[k], sum_s[p][k]);
                    }
                }
                par.get(kScale, p, lane, o);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] *= d[p][k];
                if (there)
                    store4<RE, FULL>(a.dR + at * RE + (uint32_t)(e[p] * RE), n[p], o);
                unpack<XE>(cur.b[p], v[p]);
            }
            const float rho = a.post ? normalise<W, P, FULL>(v, n, a.layer, a.inv_d, a.eps, sum) : 1.0f;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (a.G) {
                    float g[4], dg[4], pw[4], pb[4];
                    unpack<XE>(cur.g[p], g);
                    par.get(kPostW, p, lane, pw);
                    par.get(kPostB, p, lane, pb);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float slope;
                        g[k] = sigmoid(g[k], slope);
                        dg[k] = d[p][k] * __builtin_fmaf(v[p][k], pw[k], pb[k]) * slope;
                        d[p][k] *= g[k];
                    }
                    if (a.dG && there)
                        store4<XE, FULL>(a.dG + at * XE + (uint32_t)(e[p] * XE), n[p], dg);
                }
                float q[4];
                par.get(kQ, p, lane, q);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sum_post[p][k] = __builtin_fmaf(d[p][k], v[p][k], sum_post[p][k]);
                    if constexpr (EXTRA)
                        sum_post0[p][k] += d[p][k];
                    d[p][k] *= q[k];
                }
            }
            if (a.post) {
                unnormalise<W, P>(v, d, a.layer, a.inv_d, sum);
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        d[p][k] *= rho;
            }
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (there)
                    store4<XE, FULL>(a.dB + at * XE + (uint32_t)(e[p] * XE), n[p], d[p]);
        }
    }
    const int ld = (a.D + 3) / 4 * 4;
    float *to = a.part + (int64_t)blockIdx.x * kSums * ld;
    put<W, P>(sum_pre, me, a.D, to + kSumPreW * ld, lds);
    if constexpr (JOIN)
        put<W, P>(sum_post, me, a.D, to + kSumPost1 * ld, lds);
    if constexpr (EXTRA) {
        put<W, P>(sum_preb, me, a.D, to + kSumPreB * ld, lds);
        if constexpr (JOIN) {
            put<W, P>(sum_post0, me, a.D, to + kSumPost0 * ld, lds);
            put<W, P>(sum_s, me, a.D, to + kSumScale * ld, lds);
        }
    }
}

template <int XE, int RE, int W, int P, bool FULL>
int launch_as(const Args &a, bool extra, hipStream_t s)
{
    // as many blocks as run at once: one a compute unit with the join's registers, two without
    // (512 for the join: 36.6 us instead of 31.8 at 4,099 x 1,001)
    const int grid = (int)std::min<int64_t>((a.T + kRows<W> - 1) / kRows<W>, a.dB ? 256 : kMaxBlocks);
    auto k = a.dB ? (extra ? bwd_kernel<XE, RE, W, P, FULL, true, true> : bwd_kernel<XE, RE, W, P, FULL, true, false>)
                  : (extra ? bwd_kernel<XE, RE, W, P, FULL, false, true> : bwd_kernel<XE, RE, W, P, FULL, false, false>);
    k<<<grid, kThreads, 0, s>>>(a);
    return grid;
}

template <int XE, int RE, int W, int P>
int launch(const Args &a, bool extra, hipStream_t s)
{
    return a.D == 256 * W * P ? launch_as<XE, RE, W, P, true>(a, extra, s) : launch_as<XE, RE, W, P, false>(a, extra, s);
}

template <int XE, int RE>
int by_width(const Args &a, bool extra, hipStream_t s)
{
    if (a.D <= 256)
        return launch<XE, RE, 1, 1>(a, extra, s);
    if (a.D <= 512)
        return launch<XE, RE, 1, 2>(a, extra, s);
    if (a.D <= 768)
        return launch<XE, RE, 1, 3>(a, extra, s);
    if (a.D <= 1024)
        return launch<XE, RE, 2, 2>(a, extra, s);
    if (a.D <= 2048)
        return launch<XE, RE, 4, 2>(a, extra, s);
    return launch<XE, RE, 8, 2>(a, extra, s);
}

}   // namespace

int launch_bwd(const Args &a, int x_dtype, int r_dtype, bool extra, hipStream_t s)
{
    if (x_dtype == NORM_DTYPE_F32)
        return by_width<4, 4>(a, extra, s);
    if (r_dtype == NORM_DTYPE_F32)
        return by_width<2, 4>(a, extra, s);
    return by_width<2, 2>(a, extra, s);
}

}   // namespace rownorm
