// What the kernels of the gated linear recurrence share: the gates, loads and
// stores of a lane's channels, and a call's arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/recur.h"
#include "ngram_dev.hpp"

namespace recur {

// A block takes a chunk of WAVES * STEPS positions, STEPS to a wavefront (13 to 20 in the
// forward: the same times).
constexpr int kWaves = 4, kFwdSteps = 16, kBwdSteps = 8;
constexpr int kManyWaves = 16;   // where that makes one chunk of the whole call
static_assert(kWaves * kBwdSteps == RECUR_CHUNK, "a saved state in front of every backward chunk");
constexpr int kTicketWords = 64;   // from one column's ticket to the next
constexpr int kGroup = 16;   // chunks between two states that are passed on

struct Args {
    const uint8_t *x, *r, *i, *dy;
    int64_t ldx, ldr, ldi;   // bytes
    const float *lam, *h0, *dhT;
    const int32_t *offsets;
    uint8_t *y, *dx, *dr, *di;
    int64_t lddx, lddr, lddi;   // bytes
    float *hT, *saved, *dlam, *dh0;
    int64_t T, n;
    int D, accum, per, columns;   // channels of a lane; columns: blocks side by side
    int chunks;              // in a column
    bool alone;              // one chunk: nobody waits
    float c;
    // workspace
    uint32_t *tickets;  // [columns], kTicketWords apart
    uint64_t *sums;     // [chunks][columns][V][64]: a chunk's (A, H)
    uint64_t *states;   // [chunks / kGroup + 1][columns][V][64]: the state in front of a group
    int64_t words;      // of both
    float *part;        // [chunks][D]: the backward's sums for dlam
};

constexpr float kLog2e = 1.44269504f;

// s(v).
__device__ __forceinline__ float sigmoid(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -kLog2e));
}

// s(v) and 1 - s(v), neither a difference of numbers near 1.
__device__ __forceinline__ void sigmoid(float v, float &s, float &rest)
{
    const float e = __builtin_amdgcn_exp2f(fabsf(v) * -kLog2e), q = __builtin_amdgcn_rcpf(1.0f + e), p = e * q;
    s = v >= 0.0f ? q : p;
    rest = v >= 0.0f ? p : q;
}

// exp(z) - 1 for z <= 0 near 0: the series to z^7, which above kSeries leaves out less
// than 2^-25 of the value.
constexpr float kSeries = -0.35f;
__device__ __forceinline__ float expm1_near(float z)
{
    float p = __builtin_fmaf(z, 1.0f / 5040, 1.0f / 720);
    p = __builtin_fmaf(z, p, 1.0f / 120);
    p = __builtin_fmaf(z, p, 1.0f / 24);
    p = __builtin_fmaf(z, p, 1.0f / 6);
    p = __builtin_fmaf(z, p, 0.5f);
    return __builtin_fmaf(z * z, p, z);
}

// -c sp(lam), sp(lam) = max(lam, 0) + log(1 + w) with w = exp(-|lam|), and log(1 + w)
// = 2 atanh(s), s = w / (2 + w) at most 1/3: its series to s^15 leaves out less than
// 2^-26 of the value.
__device__ __forceinline__ float decay(float lam, float c)
{
    const float w = __builtin_amdgcn_exp2f(fabsf(lam) * -kLog2e), s = w * __builtin_amdgcn_rcpf(2.0f + w), q = s * s;
    float p = __builtin_fmaf(q, 1.0f / 15, 1.0f / 13);
    p = __builtin_fmaf(q, p, 1.0f / 11);
    p = __builtin_fmaf(q, p, 1.0f / 9);
    p = __builtin_fmaf(q, p, 1.0f / 7);
    p = __builtin_fmaf(q, p, 1.0f / 5);
    p = __builtin_fmaf(q, p, 1.0f / 3);
    p = __builtin_fmaf(q, p, 1.0f);
    return -c * __builtin_fmaf(2.0f * s, p, fmaxf(lam, 0.0f));
}

// a b, rounded by itself and not fused into a sum: an accumulated gradient is then
// what was there plus the gradient that a call without accumulation gives.
__device__ __forceinline__ float alone(float a, float b)
{
#pragma clang fp contract(off)
    return a * b;
}

// The value is computed where this stands.  Otherwise the compiler moves a product
// down to the branch that uses it, and its factors stay in registers until then (256
// registers and spills instead of 168 in the backward).
__device__ __forceinline__ void here(float &v) { asm volatile("" : "+v"(v)); }

// a = exp(z), e = a - 1 and m = sqrt(1 - a^2) = sqrt(-e (2 + e)).  Near 1 the series gives
// e, and a = 1 + e; from kSeries on exp gives a, which is below 0.71 there, and e = a - 1:
// each of them keeps its relative precision, however fast or slow the decay.  (1 + e on
// both sides would leave a an absolute error of 2^-24, and make it 0 from z = -17.5 on.)
__device__ __forceinline__ void decay_near(float z, float &a, float &e)
{
    e = expm1_near(z);
    a = 1.0f + e;
}
// The same of any z <= 0, after decay_near.
__device__ __forceinline__ void decay_any(float z, float &a, float &e)
{
    const float x = __builtin_amdgcn_exp2f(z * kLog2e);
    const bool near = z > kSeries;
    a = near ? a : x;
    e = near ? e : x - 1.0f;
}
__device__ __forceinline__ float rest_of(float e) { return __builtin_amdgcn_sqrtf(-e * (2.0f + e)); }

// ALL: z is known to be above kSeries, which saves a quarter of the gates' instructions.
template <bool ALL>
__device__ __forceinline__ void decays(float z, float &a, float &m)
{
    float e;
    decay_near(z, a, e);
    if constexpr (!ALL)
        decay_any(z, a, e);
    m = rest_of(e);
}

// V channels side by side as floats.  Rows start at any element: the access
// claims no more than the elements' own alignment (global memory takes it).
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef float f32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));

template <int E, int V>
struct Raw;
template <>
struct Raw<2, 1> {
    uint16_t w;
};
template <>
struct Raw<2, 2> {
    uint32_t w;
};
template <>
struct Raw<4, 1> {
    float w;
};
template <>
struct Raw<4, 2> {
    f32x2_a4 w;
};

template <int E, int V>
__device__ __forceinline__ Raw<E, V> load(const uint8_t *p)
{
    Raw<E, V> r;
    if constexpr (E == 2 && V == 2)
        r.w = *reinterpret_cast<const u32_a2 *>(p);
    else
        r.w = *reinterpret_cast<const decltype(r.w) *>(p);
    return r;
}

template <int E, int V>
__device__ __forceinline__ void unpack(const Raw<E, V> &r, float (&v)[V])
{
    if constexpr (E == 2 && V == 2) {
        v[0] = ngram::bf16_lo(r.w);
        v[1] = ngram::bf16_hi(r.w);
    } else if constexpr (E == 2) {
        v[0] = __uint_as_float((uint32_t)r.w << 16);
    } else if constexpr (V == 2) {
        v[0] = r.w[0];
        v[1] = r.w[1];
    } else {
        v[0] = r.w;
    }
}

template <int E, int V>
__device__ __forceinline__ void store(uint8_t *p, const float (&v)[V])
{
    if constexpr (E == 2 && V == 2)
        *reinterpret_cast<u32_a2 *>(p) = ngram::bf16_pack_rne(v[0], v[1]);
    else if constexpr (E == 2)
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)ngram::bf16_pack_rne(v[0], 0.0f);
    else if constexpr (V == 2)
        *reinterpret_cast<f32x2_a4 *>(p) = f32x2_a4{v[0], v[1]};
    else
        *reinterpret_cast<float *>(p) = v[0];
}

// A stretch of positions takes the state h in front of it to A h + H, or, where a
// sequence begins in it, to H: A is -1 then (a product of a's is never negative),
// so that an infinity or NaN of the sequence before does not come through a 0 A.
struct Span1 {
    float A, H;
};

__device__ __forceinline__ float through(const Span1 &s, float h) { return s.A < 0.0f ? s.H : __builtin_fmaf(s.A, h, s.H); }

// First p, then q.
__device__ __forceinline__ Span1 join(const Span1 &p, const Span1 &q)
{
    Span1 r;
    r.A = q.A < 0.0f || p.A < 0.0f ? -1.0f : p.A * q.A;
    r.H = through(q, p.H);
    return r;
}

// Words of the workspace that one block writes and others wait for: a value that
// says by itself that it is there (kNone is not), so no other memory has to be
// ordered with it.
constexpr uint64_t kNone = ~0ull;

__device__ __forceinline__ uint64_t word(const Span1 &s)
{
    const uint32_t A = s.A != s.A ? 0x7FC00000u : __float_as_uint(s.A);
    return (uint64_t)__float_as_uint(s.H) << 32 | A;
}
__device__ __forceinline__ Span1 span(uint64_t w)
{
    return Span1{__uint_as_float((uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}
__device__ __forceinline__ void publish(uint64_t *p, uint64_t w)
{
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t peek(const uint64_t *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}   // namespace recur
