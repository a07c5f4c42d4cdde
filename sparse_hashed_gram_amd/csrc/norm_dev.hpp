// What norm_fwd.hip and norm_bwd.hip share: the pieces of a row that a lane
// holds, a row's sums and statistics, the parameters, and the choice of tile.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/norm.h"
#include "ngram_dev.hpp"

namespace rownorm {

// A lane holds P pieces of 4 neighbouring elements of a row, a piece of every
// lane beside the next lane's: whole 128-byte lines, and D = 768 is exactly 3
// pieces of one wavefront.  Rows of an odd width start at any element, so the
// 8- and 16-byte accesses claim no more than the elements' own alignment (global
// memory takes them unaligned).
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

template <int E>
__device__ __forceinline__ void load4(const uint8_t *p, int n, float (&v)[4])
{
    if constexpr (E == 2) {
        if (n >= 4) {
            const u32x2_a2 w = *reinterpret_cast<const u32x2_a2 *>(p);
            v[0] = ngram::bf16_lo(w[0]);
            v[1] = ngram::bf16_hi(w[0]);
            v[2] = ngram::bf16_lo(w[1]);
            v[3] = ngram::bf16_hi(w[1]);
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = k < n ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[k] << 16) : 0.0f;
    } else {
        if (n >= 4) {
            const f32x4_a4 w = *reinterpret_cast<const f32x4_a4 *>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = w[k];
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = k < n ? reinterpret_cast<const float *>(p)[k] : 0.0f;
    }
}

template <int E>
__device__ __forceinline__ void store4(uint8_t *p, int n, const float (&v)[4])
{
    if constexpr (E == 2) {
        if (n >= 4) {
            const u32x2_a2 w = {ngram::bf16_pack_rne(v[0], v[1]), ngram::bf16_pack_rne(v[2], v[3])};
            *reinterpret_cast<u32x2_a2 *>(p) = w;
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n)
                reinterpret_cast<uint16_t *>(p)[k] = (uint16_t)ngram::bf16_pack_rne(v[k], 0.0f);
    } else {
        if (n >= 4) {
            const f32x4_a4 w = {v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4_a4 *>(p) = w;
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n)
                reinterpret_cast<float *>(p)[k] = v[k];
    }
}

// W wavefronts to a row: up to 1,024 elements one wavefront, and four rows to a
// block of four; above, a block to a row.
template <int W>
constexpr int kRows = W == 1 ? 4 : 1;
template <int W>
constexpr int kThreads = W == 1 ? 256 : 64 * W;

// Sums over a row of `W` wavefronts, the same bits in every lane.  One barrier a
// sum: a wavefront can be one sum ahead of another, so two places do.
template <int W>
struct RowSum {
    float2 (*red)[W];
    int at = 0;

    __device__ __forceinline__ float2 operator()(float a, float b)
    {
        const float2 s = {ngram::wave_sum(a), ngram::wave_sum(b)};
        if constexpr (W == 1) {
            return s;
        } else {
            at ^= 1;
            if (threadIdx.x % 64 == 0)
                red[at][threadIdx.x / 64] = s;
            __syncthreads();
            float2 t = red[at][0];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                t.x += red[at][i].x;
                t.y += red[at][i].y;
            }
            return t;
        }
    }

    __device__ __forceinline__ float operator()(float a)
    {
        if constexpr (W == 1)
            return ngram::wave_sum(a);
        else
            return (*this)(a, 0.0f).x;
    }
};

// Turns v into xh in place; returns the factor rho that a gradient in front of
// the norm has.  The mean first, then the squares of what is left: no
// difference of large sums.  A row whose squares pass fp32's range (values over
// about 2^63) is scaled by 2^-80 before, and its eps no longer counts.  n[p]:
// elements of the row that piece p has, at most 4.
template <int W, int P>
__device__ __forceinline__ float normalise(float (&v)[P][4], const int (&n)[P], int layer, float inv_d, float eps,
                                           RowSum<W> &sum)
{
    float q = 0.0f, m = 0.0f, unit = 1.0f;
    auto squares = [&] {
        q = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                q = __builtin_fmaf(v[p][k], v[p][k], q);
    };
    auto total = [&] {
        m = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p)
            m += (v[p][0] + v[p][1]) + (v[p][2] + v[p][3]);
    };
    auto scale = [&](float by) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[p][k] *= by;
    };
    squares();
    if (layer) {
        total();
        const float2 s = sum(q, m);
        q = s.x;
        m = s.y;
    } else {
        q = sum(q);
    }
    if (!(q * inv_d < 1e38f)) {
        unit = 0x1p-80f;
        eps = 0.0f;
        scale(unit);
        squares();
        total();
        const float2 s = sum(q, m);
        q = s.x;
        m = s.y;
    }
    if (layer) {
        m *= inv_d;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[p][k] = k < n[p] ? v[p][k] - m : 0.0f;
        squares();
        q = sum(q);
    }
    const float rho = rsqrtf(__builtin_fmaf(q, inv_d, eps));
    scale(rho);
    return rho * unit;
}

// A parameter [D] (or one number, `one`) of fp32 or bf16 at element e; absent: `none`.
__device__ __forceinline__ void load_param(const uint8_t *p, int f32, int one, int e, int n, float none, float (&v)[4])
{
    if (!p) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = none;
    } else if (one) {
        const float x = f32 ? *reinterpret_cast<const float *>(p)
                            : __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t *>(p) << 16);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = x;
    } else if (f32) {
        load4<4>(p + (int64_t)e * 4, n, v);
    } else {
        load4<2>(p + (int64_t)e * 2, n, v);
    }
}

// sigmoid(x), and its derivative e / (1 + e)^2 with e = exp(-|x|): no difference
// of numbers near 1.
__device__ __forceinline__ float sigmoid(float x, float &slope)
{
    const float e = __expf(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e);
    slope = e * r * r;
    return x >= 0.0f ? r : e * r;
}

struct Params {
    const uint8_t *post_w, *post_b, *gate, *scale, *w, *b;
    int f32, gate_one, scale_one;
};

// One call of a forward (R1 = NULL, B = NULL: the norm alone) or a backward.
struct Args {
    const uint8_t *R, *B, *G, *R1in, *dX, *dR1;
    uint8_t *R1, *X, *dR, *dB, *dG;
    float *part;
    Params p;
    int64_t T;
    int D, layer, post, pre;
    float eps, inv_d;
};

// The backward's sums over t: places in a block's part of the workspace.
constexpr int kSumPreW = 0, kSumPost1 = 1, kSumPreB = 2, kSumPost0 = 3, kSumScale = 4, kSums = 5;
constexpr int kMaxBlocks = 512;   // parts; a block of the backward takes rows in turns
inline int padded(int D) { return (D + 3) / 4 * 4; }

struct GradArgs {
    const float *part;
    float *cols;   // [2][padded D]: column sums of a scalar gate's and scale's gradients
    Params p;
    void *dpost_w, *dpost_b, *dgate, *dscale, *dw, *db;
    int D, parts, f32, accum, post, gate_token;
};

void launch_fwd(const Args &a, int x_dtype, int r_dtype, hipStream_t s);
// Enqueues the backward's rows; the number of parts that it leaves in a.part.
// extra: other sums than kSumPreW and kSumPost1 are wanted.
int launch_bwd(const Args &a, int x_dtype, int r_dtype, bool extra, hipStream_t s);

}   // namespace rownorm
