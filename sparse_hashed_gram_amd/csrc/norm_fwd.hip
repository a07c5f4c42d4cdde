// Forward of the norms (include/norm.h): X = norm(R), and the join
// R1 = s R + g norm(B), X = norm(R1), in one pass over the rows: a row lives in
// registers between its loads and its stores, the block's next rows are on their way
// meanwhile.  HBM bounds it: the join of 49,152 x 768 with a gate an element, bf16
// beside an fp32 stream, takes 100 us (528 MB, 5.3 TB/s; a copy reaches 5.0 to 5.2).
// One row takes 2.1 us of kernel and 7.7 with the call.
#include <algorithm>

#include "norm_dev.hpp"

namespace rownorm {
namespace {

enum { kW, kB, kPostW, kPostB, kGate, kScale, kVectors };

template <int XE, int RE, int P, bool FULL, bool JOIN>
struct Row {
    Piece<RE> r[P];
    Piece<XE> b[P], g[P];

    __device__ __forceinline__ void load(const Args &a, int64_t row, const int (&e)[P], const int (&n)[P])
    {
        const int64_t at = min(row, a.T - 1) * a.D;
        load_row<RE, P, FULL>(a.R + at * RE, e, n, r);
        if constexpr (JOIN) {
            load_row<XE, P, FULL>(a.B + at * XE, e, n, b);
            if (a.G)
                load_row<XE, P, FULL>(a.G + at * XE, e, n, g);
        }
    }
};

template <int XE, int RE, int W, int P, bool FULL, bool JOIN>
__device__ __forceinline__ void forward(const Args &a)
{
    constexpr int N = JOIN ? kVectors : kB + 1;
    __shared__ float2 red[2][8];
    __shared__ float params[W == 1 ? N : 1][P * 256];
    const Place<W> me;
    const int lane = me.lane;
    RowSum<W> sum{red, me.row};
    ParamRows<W, P, N> par;
    par.lds = params;
    int e[P], n[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        e[p] = (p * 64 * W + lane) * 4;
        n[p] = max(0, min(4, a.D - e[p]));
    }
    const int64_t step = (int64_t)gridDim.x * kRows<W>;
    int64_t row = (int64_t)blockIdx.x * kRows<W> + me.row, first = (int64_t)blockIdx.x * kRows<W>;
    Row<XE, RE, P, FULL, JOIN> next;
    next.load(a, row, e, n);
    const uint8_t *vec[kVectors] = {a.p.w, a.p.b, a.p.post_w, a.p.post_b, a.G ? nullptr : a.p.gate, a.p.scale};
    const float none[kVectors] = {1.0f, 0.0f, 1.0f, 0.0f, 1.0f, 1.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (W == 1 && me.row != i)   // a wavefront a vector
            continue;
        const int one = i == kGate ? a.p.gate_one : i == kScale ? a.p.scale_one : 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float v[4];
            load_param(vec[i], a.p.f32, one, e[p], n[p], none[i], v);
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
        const Row<XE, RE, P, FULL, JOIN> cur = next;
        next.load(a, row + step, e, n);
        const int64_t at = row * a.D;
        float r[P][4];
#pragma unroll
        for (int p = 0; p < P; ++p)
            unpack<RE>(cur.r[p], r[p]);
        if constexpr (JOIN) {
            float v[P][4];
#pragma unroll
            for (int p = 0; p < P; ++p)
                unpack<XE>(cur.b[p], v[p]);
            if (a.post) {
                normalise<W, P, FULL>(v, n, a.layer, a.inv_d, a.eps, sum);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    float pw[4], pb[4];
                    par.get(kPostW, p, lane, pw);
                    par.get(kPostB, p, lane, pb);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[p][k] = __builtin_fmaf(v[p][k], pw[k], pb[k]);
                }
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                float s[4], g[4];
                par.get(kScale, p, lane, s);
                if (a.G) {
                    unpack<XE>(cur.g[p], g);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float slope;
                        g[k] = sigmoid(g[k], slope);
                    }
                } else {
                    par.get(kGate, p, lane, g);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    r[p][k] = FULL || k < n[p] ? __builtin_fmaf(g[k], v[p][k], s[k] * r[p][k]) : 0.0f;
                if (there)
                    store4<RE, FULL>(a.R1 + at * RE + (uint32_t)(e[p] * RE), n[p], r[p]);
            }
            if (!a.pre)
                continue;
        }
        normalise<W, P, FULL>(r, n, a.layer, a.inv_d, a.eps, sum);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float w[4], b[4];
            par.get(kW, p, lane, w);
            par.get(kB, p, lane, b);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                r[p][k] = __builtin_fmaf(r[p][k], w[k], b[k]);
            if (there)
                store4<XE, FULL>(a.X + at * XE + (uint32_t)(e[p] * XE), n[p], r[p]);
        }
    }
}

// The norm alone runs four blocks a compute unit, eight wavefronts a SIMD, which is what
// the grid counts on.  Over 80 scalar registers only seven fit, whatever the compiler's
// occupancy says (20,000 x 1,500 bf16: 30.0 us instead of 23.0 with 82).
template <int XE, int RE, int W, int P, bool FULL>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_num_sgpr(80))) void fwd_kernel(Args a)
{
    forward<XE, RE, W, P, FULL, false>(a);
}

template <int XE, int RE, int W, int P, bool FULL>
__global__ __launch_bounds__(kThreads) void join_kernel(Args a)
{
    forward<XE, RE, W, P, FULL, true>(a);
}

template <int XE, int RE, int W, int P>
void launch(const Args &a, hipStream_t s)
{
    // as many blocks as run at once; rows in turns spare the rest their parameters' loads
    const unsigned grid = (unsigned)std::min<int64_t>((a.T + kRows<W> - 1) / kRows<W>, 1024);
    const bool full = a.D == 256 * W * P;
    auto k = a.R1 ? (full ? join_kernel<XE, RE, W, P, true> : join_kernel<XE, RE, W, P, false>)
                  : (full ? fwd_kernel<XE, RE, W, P, true> : fwd_kernel<XE, RE, W, P, false>);
    k<<<grid, kThreads, 0, s>>>(a);
}

template <int XE, int RE>
void by_width(const Args &a, hipStream_t s)
{
    if (a.D <= 256)
        launch<XE, RE, 1, 1>(a, s);
    else if (a.D <= 512)
        launch<XE, RE, 1, 2>(a, s);
    else if (a.D <= 768)
        launch<XE, RE, 1, 3>(a, s);
    else if (a.D <= 1024)
        launch<XE, RE, 2, 2>(a, s);
    else if (a.D <= 2048)
        launch<XE, RE, 4, 2>(a, s);
    else
        launch<XE, RE, 8, 2>(a, s);
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
