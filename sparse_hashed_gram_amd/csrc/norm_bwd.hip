// Backward of the norms (include/norm.h), rows and, in parts, the sums over t
// that the parameters' gradients are made of.
#include <algorithm>

#include "norm_dev.hpp"

namespace rownorm {
namespace {

// xh and d -> the gradient in front of the norm over rho: d - [layer] mean(d) - xh mean(d xh).
template <int W, int P>
__device__ __forceinline__ void unnormalise(const float (&xh)[P][4], float (&d)[P][4], const int (&n)[P], int layer,
                                            float inv_d, RowSum<W> &sum)
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

// A block's sums of a column: those of its rows' wavefronts, then to its part.
template <int W, int P>
__device__ __forceinline__ void put(float (&v)[P][4], const int (&e)[P], int D, float *to, float (*lds)[P * 256])
{
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    if constexpr (W == 1) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<float4 *>(&lds[wave][(p * 64 + lane) * 4]) = make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
        __syncthreads();
        for (int j = threadIdx.x; j < D; j += kThreads<W>)
            to[j] = (lds[0][j] + lds[1][j]) + (lds[2][j] + lds[3][j]);
        __syncthreads();
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (e[p] < D)   // parts are padded to whole pieces
                *reinterpret_cast<float4 *>(to + e[p]) = make_float4(v[p][0], v[p][1], v[p][2], v[p][3]);
    }
}

template <int XE, int RE, int W, int P, bool JOIN, bool EXTRA>
__global__ __launch_bounds__(kThreads<W>) void bwd_kernel(Args a)
{
    __shared__ float2 red[2][W];
    __shared__ float lds[W == 1 ? 4 : 1][P * 256];
    RowSum<W> sum{red};
    const int lane = W == 1 ? threadIdx.x % 64 : threadIdx.x;
    int e[P], n[P];
    // q: what turns E into the gradient of the normalised B: gate (not a token's) times post_w
    float w[P][4], q[P][4], pw[P][4], pb[P][4], s[P][4];
    float sum_pre[P][4] = {}, sum_post[P][4] = {}, sum_preb[P][4] = {}, sum_post0[P][4] = {}, sum_s[P][4] = {};
#pragma unroll
    for (int p = 0; p < P; ++p) {
        e[p] = (p * 64 * W + lane) * 4;
        n[p] = max(0, min(4, a.D - e[p]));
        load_param(a.p.w, a.p.f32, 0, e[p], n[p], 1.0f, w[p]);
        if constexpr (JOIN) {
            load_param(a.p.post_w, a.p.f32, 0, e[p], n[p], 1.0f, pw[p]);
            load_param(a.p.post_b, a.p.f32, 0, e[p], n[p], 0.0f, pb[p]);
            load_param(a.G ? nullptr : a.p.gate, a.p.f32, a.p.gate_one, e[p], n[p], 1.0f, q[p]);
            load_param(a.p.scale, a.p.f32, a.p.scale_one, e[p], n[p], 1.0f, s[p]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                q[p][k] *= pw[p][k];
        }
    }
    const int64_t step = (int64_t)gridDim.x * kRows<W>;
    for (int64_t row = (int64_t)blockIdx.x * kRows<W> + (W == 1 ? threadIdx.x / 64 : 0); row < a.T; row += step) {
        const int64_t at = row * a.D;
        float d[P][4];   // E
        if (a.pre) {
            float x[P][4], r[P][4];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                load4<RE>(a.R1in + (at + e[p]) * RE, n[p], x[p]);
                load4<XE>(a.dX + (at + e[p]) * XE, n[p], d[p]);
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (a.dR1)
                    load4<RE>(a.dR1 + (at + e[p]) * RE, n[p], r[p]);
                else
                    r[p][0] = r[p][1] = r[p][2] = r[p][3] = 0.0f;
            }
            const float rho = normalise<W, P>(x, n, a.layer, a.inv_d, a.eps, sum);
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sum_pre[p][k] = __builtin_fmaf(d[p][k], x[p][k], sum_pre[p][k]);
                    if constexpr (EXTRA)
                        sum_preb[p][k] += d[p][k];
                    d[p][k] *= w[p][k];
                }
            unnormalise<W, P>(x, d, n, a.layer, a.inv_d, sum);
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    d[p][k] = k < n[p] ? __builtin_fmaf(rho, d[p][k], r[p][k]) : 0.0f;
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p)
                load4<RE>(a.dR1 + (at + e[p]) * RE, n[p], d[p]);
        }
        if constexpr (!JOIN) {
#pragma unroll
            for (int p = 0; p < P; ++p)
                store4<RE>(a.dR + (at + e[p]) * RE, n[p], d[p]);
        } else {
            float v[P][4], t[P][4];
#pragma unroll
            for (int p = 0; p < P; ++p)
                load4<XE>(a.B + (at + e[p]) * XE, n[p], v[p]);
            if (a.G) {
#pragma unroll
                for (int p = 0; p < P; ++p)
                    load4<XE>(a.G + (at + e[p]) * XE, n[p], t[p]);
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float o[4];
                if constexpr (EXTRA) {
                    if (a.R) {
                        load4<RE>(a.R + (at + e[p]) * RE, n[p], o);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sum_s[p][k] = __builtin_fmaf(d[p][k], o[k], sum_s[p][k]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = d[p][k] * s[p][k];
                store4<RE>(a.dR + (at + e[p]) * RE, n[p], o);
            }
            const float rho = a.post ? normalise<W, P>(v, n, a.layer, a.inv_d, a.eps, sum) : 1.0f;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float dg[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (a.G) {
                        float slope;
                        const float gk = sigmoid(t[p][k], slope);
                        dg[k] = d[p][k] * __builtin_fmaf(v[p][k], pw[p][k], pb[p][k]) * slope;
                        d[p][k] *= gk;
                    }
                    sum_post[p][k] = __builtin_fmaf(d[p][k], v[p][k], sum_post[p][k]);
                    if constexpr (EXTRA)
                        sum_post0[p][k] += d[p][k];
                    d[p][k] *= q[p][k];
                }
                if (a.G && a.dG)
                    store4<XE>(a.dG + (at + e[p]) * XE, n[p], dg);
            }
            if (a.post) {
                unnormalise<W, P>(v, d, n, a.layer, a.inv_d, sum);
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        d[p][k] *= rho;
            }
#pragma unroll
            for (int p = 0; p < P; ++p)
                store4<XE>(a.dB + (at + e[p]) * XE, n[p], d[p]);
        }
    }
    const int ld = (a.D + 3) / 4 * 4;
    float *to = a.part + (int64_t)blockIdx.x * kSums * ld;
    put<W, P>(sum_pre, e, a.D, to + kSumPreW * ld, lds);
    if constexpr (JOIN)
        put<W, P>(sum_post, e, a.D, to + kSumPost1 * ld, lds);
    if constexpr (EXTRA) {
        put<W, P>(sum_preb, e, a.D, to + kSumPreB * ld, lds);
        if constexpr (JOIN) {
            put<W, P>(sum_post0, e, a.D, to + kSumPost0 * ld, lds);
            put<W, P>(sum_s, e, a.D, to + kSumScale * ld, lds);
        }
    }
}

template <int XE, int RE, int W, int P>
int launch(const Args &a, bool extra, hipStream_t s)
{
    const int grid = (int)std::min<int64_t>((a.T + kRows<W> - 1) / kRows<W>, kMaxBlocks);
    if (a.dB) {
        if (extra)
            bwd_kernel<XE, RE, W, P, true, true><<<grid, kThreads<W>, 0, s>>>(a);
        else
            bwd_kernel<XE, RE, W, P, true, false><<<grid, kThreads<W>, 0, s>>>(a);
    } else {
        if (extra)
            bwd_kernel<XE, RE, W, P, false, true><<<grid, kThreads<W>, 0, s>>>(a);
        else
            bwd_kernel<XE, RE, W, P, false, false><<<grid, kThreads<W>, 0, s>>>(a);
    }
    return grid;
}

template <int XE, int RE>
int by_width(const Args &a, bool extra, hipStream_t s)
{
    if (a.D <= 256)
        return launch<XE, RE, 1, 1>(a, extra, s);
    if (a.D <= 768)
        return launch<XE, RE, 1, 3>(a, extra, s);
    if (a.D <= 1024)
        return launch<XE, RE, 1, 4>(a, extra, s);
    if (a.D <= 2048)
        return launch<XE, RE, 2, 4>(a, extra, s);
    return launch<XE, RE, 4, 4>(a, extra, s);
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
