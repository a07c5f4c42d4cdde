// What the kernels of the gated linear recurrence share: the gates, loads and
// stores of a lane's channels, and a call's arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/recur.h"
#include "ngram_dev.hpp"

namespace recur {

struct Args {
    const uint8_t *x, *r, *i, *dy;
    int64_t ldx, ldr, ldi;   // bytes
    const float *lam, *h0, *dhT;
    const int32_t *offsets;
    uint8_t *y, *dx, *dr, *di;
    int64_t lddx, lddr, lddi;   // bytes
    float *hT, *saved, *dlam, *dh0;
    int64_t T, n;
    int D, accum;
    float c;
};

// s(v) and 1 - s(v), neither a difference of numbers near 1.
__device__ __forceinline__ void sigmoid(float v, float &s, float &rest)
{
    const float e = __expf(-fabsf(v)), q = __builtin_amdgcn_rcpf(1.0f + e), p = e * q;
    s = v >= 0.0f ? q : p;
    rest = v >= 0.0f ? p : q;
}

// exp(z) - 1 for z <= 0: the series to z^7 above -0.35 (what it leaves out is
// below 2^-25 of the value), else through exp, which is below 0.71 there.
__device__ __forceinline__ float expm1_neg(float z)
{
    float p = __builtin_fmaf(z, 1.0f / 5040, 1.0f / 720);
    p = __builtin_fmaf(z, p, 1.0f / 120);
    p = __builtin_fmaf(z, p, 1.0f / 24);
    p = __builtin_fmaf(z, p, 1.0f / 6);
    p = __builtin_fmaf(z, p, 0.5f);
    p = __builtin_fmaf(z * z, p, z);
    return z > -0.35f ? p : __expf(z) - 1.0f;
}

// -c sp(lam), and s(lam).
__device__ __forceinline__ float decay(float lam, float c) { return -c * (fmaxf(lam, 0.0f) + log1pf(expf(-fabsf(lam)))); }

// a b, rounded by itself and not fused into a sum: an accumulated gradient is then
// what was there plus the gradient that a call without accumulation gives.
__device__ __forceinline__ float alone(float a, float b)
{
#pragma clang fp contract(off)
    return a * b;
}

struct Gates {
    float a, m, g, g_rest, rho, rho_rest;
};

// a = 1 + e and 1 - a^2 = -e (2 + e) with e = exp(z) - 1, so that both keep their
// relative precision where a is near 1.
__device__ __forceinline__ Gates gates(float r, float i, float k)
{
    Gates t;
    sigmoid(r, t.rho, t.rho_rest);
    sigmoid(i, t.g, t.g_rest);
    const float e = expm1_neg(k * t.rho);
    t.a = 1.0f + e;
    t.m = __builtin_amdgcn_sqrtf(-e * (2.0f + e));
    return t;
}

template <int E>
__device__ __forceinline__ float load1(const uint8_t *p)
{
    if constexpr (E == 2)
        return __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t *>(p) << 16);
    else
        return *reinterpret_cast<const float *>(p);
}

template <int E>
__device__ __forceinline__ void store1(uint8_t *p, float v)
{
    if constexpr (E == 2)
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)ngram::bf16_pack_rne(v, 0.0f);
    else
        *reinterpret_cast<float *>(p) = v;
}

}   // namespace recur
