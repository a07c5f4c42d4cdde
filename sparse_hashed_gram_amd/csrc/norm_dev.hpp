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
// memory takes them unaligned).  Pieces stay packed until they are needed, so that
// the next row's can be on their way while one row is worked on.
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int E>
struct Piece {
    f32x4 w;
};
template <>
struct Piece<2> {
    u32x2 w;
};

// n: elements of the row that the piece has; FULL: it has 4.
template <int E, bool FULL>
__device__ __forceinline__ Piece<E> load4(const uint8_t *p, int n)
{
    Piece<E> r;
    if constexpr (E == 2) {
        if (FULL || n >= 4) {
            r.w = *reinterpret_cast<const u32x2_a2 *>(p);
        } else {
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = k < n ? reinterpret_cast<const uint16_t *>(p)[k] : 0;
            r.w = u32x2{v[0] | v[1] << 16, v[2] | v[3] << 16};
        }
    } else {
        if (FULL || n >= 4) {
            r.w = *reinterpret_cast<const f32x4_a4 *>(p);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                r.w[k] = k < n ? reinterpret_cast<const float *>(p)[k] : 0.0f;
        }
    }
    return r;
}

template <int E>
__device__ __forceinline__ void unpack(const Piece<E> &r, float (&v)[4])
{
    if constexpr (E == 2) {
        v[0] = ngram::bf16_lo(r.w[0]);
        v[1] = ngram::bf16_hi(r.w[0]);
        v[2] = ngram::bf16_lo(r.w[1]);
        v[3] = ngram::bf16_hi(r.w[1]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = r.w[k];
    }
}

template <int E, bool FULL>
__device__ __forceinline__ void store4(uint8_t *p, int n, const float (&v)[4])
{
    if constexpr (E == 2) {
        if (FULL || n >= 4) {
            const u32x2_a2 w = {ngram::bf16_pack_rne(v[0], v[1]), ngram::bf16_pack_rne(v[2], v[3])};
            *reinterpret_cast<u32x2_a2 *>(p) = w;
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n)
                reinterpret_cast<uint16_t *>(p)[k] = (uint16_t)ngram::bf16_pack_rne(v[k], 0.0f);
    } else {
        if (FULL || n >= 4) {
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

// A row's pieces of one lane, at element e[p] of the row at `row`.
template <int E, int P, bool FULL>
__device__ __forceinline__ void load_row(const uint8_t *row, const int (&e)[P], const int (&n)[P], Piece<E> (&v)[P])
{
#pragma unroll
    for (int p = 0; p < P; ++p)
        v[p] = load4<E, FULL>(row + (uint32_t)(e[p] * E), n[p]);
}

// W wavefronts to a row, eight wavefronts to a block.
constexpr int kThreads = 512;
template <int W>
constexpr int kRows = 8 / W;

// Where a thread stands: its wavefront's row among the block's, and its lane among
// the row's.
template <int W>
struct Place {
    int row, lane;
    __device__ __forceinline__ Place()
    {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        row = wave / W;
        lane = wave % W * 64 + threadIdx.x % 64;
    }
};

// Sums over a row of W wavefronts, the same bits in every lane.  With W over 1 every
// wavefront of the block takes part, with one barrier a sum: a wavefront can be one
// sum ahead of another, so two places do.  any(): whether q of any row of the block
// is not below the limit (of its own row, with W = 1): what all wavefronts that meet at
// a barrier agree on.
template <int W>
struct RowSum {
    float2 (*red)[8];
    int row;
    int at = 0;

    __device__ __forceinline__ float2 of(int r) const
    {
        float2 t = red[at][r * W];
#pragma unroll
        for (int i = 1; i < W; ++i) {
            t.x += red[at][r * W + i].x;
            t.y += red[at][r * W + i].y;
        }
        return t;
    }
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
            return of(row);
        }
    }
    __device__ __forceinline__ float operator()(float a)
    {
        if constexpr (W == 1)
            return ngram::wave_sum(a);
        else
            return (*this)(a, 0.0f).x;
    }
    __device__ __forceinline__ bool any(float q, float limit) const
    {
        if constexpr (W == 1) {
            return !(q < limit);
        } else {
            bool over = false;
#pragma unroll
            for (int r = 0; r < kRows<W>; ++r)
                over = over || !(of(r).x < limit);
            return over;
        }
    }
};

// Turns v into xh in place; returns the factor rho that a gradient in front of
// the norm has.  The mean first, then the squares of what is left: no
// difference of large sums.  A row whose squares pass fp32's range (values over
// about 2^63) is scaled by 2^-80 before, and its eps no longer counts, unless all its
// values are the same and there is a mean to take away.  n[p]: elements of the row that
// piece p has, at most 4.
template <int W, int P, bool FULL>
__device__ __forceinline__ float normalise(float (&v)[P][4], const int (&n)[P], int layer, float inv_d, float eps,
                                           RowSum<W> &sum)
{
    float q = 0.0f, m = 0.0f, unit = 1.0f;
    const float given = eps;
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
    const float limit = 0x1p126f;
    squares();
    if (layer) {
        total();
        const float2 s = sum(q, m);
        q = s.x;
        m = s.y;
    } else {
        q = sum(q);
    }
    if (sum.any(q, limit)) {
        if (!(q < limit)) {
            unit = 0x1p-80f;
            eps = 0.0f;
            scale(unit);
        }
        if (layer) {   // from the first element on: a row of one value is exactly 0
            float x = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v[0][0])));
            if constexpr (W > 1)
                x = sum((int)threadIdx.x == sum.row * W * 64 ? x : 0.0f);
            if (!(q < limit)) {
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[p][k] = FULL || k < n[p] ? v[p][k] - x : 0.0f;
            }
        }
        squares();
        total();
        const float2 s = sum(q, m);
        q = s.x < INFINITY ? s.x : NAN;   // of an infinity: rho 0 would make its row zeros
        m = s.y;
        if (layer && q == 0.0f) {   // then nothing but eps counts
            eps = given;
            unit = 1.0f;
        }
    }
    if (layer) {
        m *= inv_d;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[p][k] = FULL || k < n[p] ? v[p][k] - m : 0.0f;
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
        unpack<4>(load4<4, false>(p + (int64_t)e * 4, n), v);
    } else {
        unpack<2>(load4<2, false>(p + (int64_t)e * 2, n), v);
    }
}

// N parameter vectors of a block's rows.  Where the block's wavefronts have a row
// each, they share a copy in LDS (60 registers fewer in the backward, so twelve
// wavefronts to a compute unit instead of eight); where a row is a block's, each lane
// holds its own elements.
template <int W, int P, int N>
struct ParamRows {
    float (*lds)[P * 256];
    float own[W == 1 ? 1 : N][P][4];

    __device__ __forceinline__ void put(int i, int p, int lane, const float (&v)[4])
    {
        if constexpr (W == 1)
            *reinterpret_cast<float4 *>(&lds[i][(p * 64 + lane) * 4]) = make_float4(v[0], v[1], v[2], v[3]);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k)
                own[i][p][k] = v[k];
    }
    __device__ __forceinline__ void get(int i, int p, int lane, float (&v)[4]) const
    {
        if constexpr (W == 1) {
            const float4 x = *reinterpret_cast<const float4 *>(&lds[i][(p * 64 + lane) * 4]);
            v[0] = x.x;
            v[1] = x.y;
            v[2] = x.z;
            v[3] = x.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = own[i][p][k];
        }
    }
};

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
