// Forward of the norms (include/norm.h): X = norm(R), and the join
// R1 = s R + g norm(B), X = norm(R1), in one pass over the rows.
#include <algorithm>

#include "norm_dev.hpp"

namespace rownorm {
namespace {

template <int XE, int RE, int W, int P, bool JOIN>
__global__ __launch_bounds__(kThreads<W>) void fwd_kernel(Args a)
{
    __shared__ float2 red[2][W];
    RowSum<W> sum{red};
    const int lane = W == 1 ? threadIdx.x % 64 : threadIdx.x;
    int e[P], n[P];
    float pw[P][4], pb[P][4], g[P][4], s[P][4], w[P][4], b[P][4];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        e[p] = (p * 64 * W + lane) * 4;
        n[p] = max(0, min(4, a.D - e[p]));
        load_param(a.p.w, a.p.f32, 0, e[p], n[p], 1.0f, w[p]);
        load_param(a.p.b, a.p.f32, 0, e[p], n[p], 0.0f, b[p]);
        if constexpr (JOIN) {
            load_param(a.p.post_w, a.p.f32, 0, e[p], n[p], 1.0f, pw[p]);
            load_param(a.p.post_b, a.p.f32, 0, e[p], n[p], 0.0f, pb[p]);
            load_param(a.G ? nullptr : a.p.gate, a.p.f32, a.p.gate_one, e[p], n[p], 1.0f, g[p]);
            load_param(a.p.scale, a.p.f32, a.p.scale_one, e[p], n[p], 1.0f, s[p]);
        }
    }
    const int64_t step = (int64_t)gridDim.x * kRows<W>;
    for (int64_t row = (int64_t)blockIdx.x * kRows<W> + (W == 1 ? threadIdx.x / 64 : 0); row < a.T; row += step) {
        const int64_t at = row * a.D;
        float r[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p)
            load4<RE>(a.R + (at + e[p]) * RE, n[p], r[p]);
        if constexpr (JOIN) {
            float v[P][4], t[P][4];
#pragma unroll
            for (int p = 0; p < P; ++p)
                load4<XE>(a.B + (at + e[p]) * XE, n[p], v[p]);
            if (a.G) {
#pragma unroll
                for (int p = 0; p < P; ++p)
                    load4<XE>(a.G + (at + e[p]) * XE, n[p], t[p]);
            }
            if (a.post) {
                normalise<W, P>(v, n, a.layer, a.inv_d, a.eps, sum);
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[p][k] = __builtin_fmaf(v[p][k], pw[p][k], pb[p][k]);
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float slope;
                    const float gk = a.G ? sigmoid(t[p][k], slope) : g[p][k];
                    r[p][k] = k < n[p] ? __builtin_fmaf(gk, v[p][k], s[p][k] * r[p][k]) : 0.0f;
                }
                store4<RE>(a.R1 + (at + e[p]) * RE, n[p], r[p]);
            }
            if (!a.pre)
                continue;
        }
        normalise<W, P>(r, n, a.layer, a.inv_d, a.eps, sum);
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                r[p][k] = __builtin_fmaf(r[p][k], w[p][k], b[p][k]);
            store4<XE>(a.X + (at + e[p]) * XE, n[p], r[p]);
        }
    }
}

template <int XE, int RE, int W, int P>
void launch(const Args &a, hipStream_t s)
{
    const unsigned grid = (unsigned)std::min<int64_t>((a.T + kRows<W> - 1) / kRows<W>, W == 1 ? 2048 : 4096);
    if (a.R1)
        fwd_kernel<XE, RE, W, P, true><<<grid, kThreads<W>, 0, s>>>(a);
    else
        fwd_kernel<XE, RE, W, P, false><<<grid, kThreads<W>, 0, s>>>(a);
}

template <int XE, int RE>
void by_width(const Args &a, hipStream_t s)
{
    if (a.D <= 256)
        launch<XE, RE, 1, 1>(a, s);
    else if (a.D <= 768)
        launch<XE, RE, 1, 3>(a, s);
    else if (a.D <= 1024)
        launch<XE, RE, 1, 4>(a, s);
    else if (a.D <= 2048)
        launch<XE, RE, 2, 4>(a, s);
    else
        launch<XE, RE, 4, 4>(a, s);
}

}   // namespace

void launch_fwd(const Args &a, int x_dtype, int r_dtype, hipStream_t s)
{
    if (x_dtype == NORM_DTYPE_F32)
        by_width<4, 4>(a, s);
    else if (r_dtype == NORM_DTYPE_F32)
        by_width<2, 4>(a, s);
    else
        by_width<2, 2>(a, s);
}

}   // namespace rownorm
