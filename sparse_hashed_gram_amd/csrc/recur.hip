// The gated linear recurrence (include/recur.h): a lane a channel, position by
// position.
#include <algorithm>
#include <initializer_list>

#include "recur_dev.hpp"
#include "spans.hpp"

namespace recur {
namespace {

using spans::meet;
using spans::Span;

constexpr uint64_t kAlign = 256;
constexpr int kChunk = RECUR_CHUNK;

// Sequence k's rows, inside [0, T).
__device__ __forceinline__ void sequence(const Args &a, int64_t k, int64_t &from, int64_t &to)
{
    from = a.offsets ? a.offsets[k] : 0;
    to = a.offsets ? a.offsets[k + 1] : a.T;
    from = max((int64_t)0, min(from, a.T));
    to = max((int64_t)0, min(to, a.T));
}

template <int E>
__global__ __launch_bounds__(64) void fwd_kernel(Args a)
{
    const int j = blockIdx.x * 64 + threadIdx.x;
    if (j >= a.D)
        return;
    const float k = decay(a.lam[j], a.c);
    for (int64_t s = 0; s < a.n; ++s) {
        int64_t from, to;
        sequence(a, s, from, to);
        float h = a.h0 ? a.h0[s * a.D + j] : 0.0f;
        for (int64_t t = from; t < to; ++t) {
            if (a.saved && t % kChunk == 0)
                a.saved[t / kChunk * a.D + j] = h;
            const Gates v = gates(load1<E>(a.r + t * a.ldr + (int64_t)j * E), load1<E>(a.i + t * a.ldi + (int64_t)j * E), k);
            h = __builtin_fmaf(v.a, h, v.m * v.g * load1<E>(a.x + t * a.ldx + (int64_t)j * E));
            store1<E>(a.y + (t * a.D + j) * E, h);
        }
        if (a.hT)
            a.hT[s * a.D + j] = h;
    }
}

template <int E>
__global__ __launch_bounds__(64) void bwd_kernel(Args a)
{
    __shared__ float before[kChunk][64];   // h_{t-1} of a chunk's positions
    const int j = blockIdx.x * 64 + threadIdx.x;
    if (j >= a.D)
        return;
    const float k = decay(a.lam[j], a.c);
    float dk = 0.0f;
    for (int64_t s = a.n; s-- > 0;) {
        int64_t from, to;
        sequence(a, s, from, to);
        float in = a.dhT ? a.dhT[s * a.D + j] : 0.0f;   // a_{t+1} G_{t+1}
        for (int64_t end = to; end > from;) {
            const int64_t begin = std::max(from, (end - 1) / kChunk * kChunk);
            float h = begin == from ? (a.h0 ? a.h0[s * a.D + j] : 0.0f) : a.saved[begin / kChunk * a.D + j];
            for (int64_t t = begin; t < end; ++t) {
                before[t - begin][threadIdx.x] = h;
                const Gates v = gates(load1<E>(a.r + t * a.ldr + (int64_t)j * E), load1<E>(a.i + t * a.ldi + (int64_t)j * E), k);
                h = __builtin_fmaf(v.a, h, v.m * v.g * load1<E>(a.x + t * a.ldx + (int64_t)j * E));
            }
            for (int64_t t = end; t-- > begin;) {
                const Gates v = gates(load1<E>(a.r + t * a.ldr + (int64_t)j * E), load1<E>(a.i + t * a.ldi + (int64_t)j * E), k);
                const float x = load1<E>(a.x + t * a.ldx + (int64_t)j * E);
                const float G = load1<E>(a.dy + (t * a.D + j) * E) + in;
                in = v.a * G;
                const float mg = v.m * v.g, over = v.m > 0.0f ? v.a * v.a / v.m : 0.0f;
                const float dz = in * before[t - begin][threadIdx.x] - G * v.g * x * over;
                store1<E>(a.dx + t * a.lddx + (int64_t)j * E, G * mg);
                store1<E>(a.di + t * a.lddi + (int64_t)j * E, G * mg * x * v.g_rest);
                store1<E>(a.dr + t * a.lddr + (int64_t)j * E, k * dz * v.rho * v.rho_rest);
                dk = __builtin_fmaf(v.rho, dz, dk);
            }
            end = begin;
        }
        if (a.dh0)
            a.dh0[s * a.D + j] = in;
    }
    float s, rest;
    sigmoid(a.lam[j], s, rest);
    const float v = alone(-a.c * s, dk);
    a.dlam[j] = a.accum ? a.dlam[j] + v : v;
}

// A wavefront a row and 64 channels.  Rows of one slot form a chain: its first
// row takes them all, in order.
template <int E>
__global__ __launch_bounds__(64) void step_kernel(Args a, float *state, int64_t states, const int32_t *slots)
{
    const int j = blockIdx.x * 64 + threadIdx.x;
    const int64_t row = blockIdx.y;
    const int64_t slot = slots ? slots[row] : row;
    if (slot < 0 || slot >= states) {
        if (j < a.D)
            store1<E>(a.y + (row * a.D + j) * E, 0.0f);
        return;
    }
    if (slots) {
        for (int64_t k = 0; k < row; ++k)
            if (slots[k] == slot)
                return;
    }
    if (j >= a.D)
        return;
    const float k = decay(a.lam[j], a.c);
    float h = state[slot * a.D + j];
    for (int64_t t = row; t < (slots ? a.n : row + 1); ++t) {
        if (slots && slots[t] != slot)
            continue;
        const Gates v = gates(load1<E>(a.r + t * a.ldr + (int64_t)j * E), load1<E>(a.i + t * a.ldi + (int64_t)j * E), k);
        h = __builtin_fmaf(v.a, h, v.m * v.g * load1<E>(a.x + t * a.ldx + (int64_t)j * E));
        store1<E>(a.y + (t * a.D + j) * E, h);
    }
    state[slot * a.D + j] = h;
}

uint64_t size_of(int dtype) { return dtype == RECUR_DTYPE_F32 ? 4 : 2; }

int check_config(const recur_config *c)
{
    if (!c)
        return RECUR_ENULL;
    const bool ok = c->dim >= 1 && c->dim <= 16384 && (c->dtype == RECUR_DTYPE_F32 || c->dtype == RECUR_DTYPE_BF16) &&
                    c->c > 0.0f && c->c <= 64.0f && (c->options & ~RECUR_OPT_ACCUM) == 0 && c->max_tokens >= 1 &&
                    c->max_tokens <= (int64_t(1) << 24);
    return ok ? RECUR_OK : RECUR_ECONFIG;
}

int64_t chunks(int64_t T) { return (T + kChunk - 1) / kChunk; }

uint64_t ws_need(const recur_config *, int) { return kAlign; }

struct Buf {
    Span s;
    uint64_t elt;
    bool needed;
};

int check(std::initializer_list<Buf> ins, std::initializer_list<Buf> outs, const Span &ws)
{
    for (const auto *l : {&ins, &outs})
        for (const Buf &b : *l) {
            if (b.needed && !b.s.p && b.s.len && b.s.rows)
                return RECUR_ENULL;
            if ((uintptr_t)b.s.p % b.elt)
                return RECUR_EALIGN;
        }
    const Buf *o = outs.begin();
    for (size_t i = 0; i < outs.size(); ++i) {
        for (const Buf &b : ins)
            if (meet(o[i].s, b.s))
                return RECUR_EARG;
        for (size_t k = 0; k < i; ++k)
            if (meet(o[i].s, o[k].s))
                return RECUR_EARG;
        if (meet(o[i].s, ws))
            return RECUR_EARG;
    }
    for (const Buf &b : ins)
        if (meet(ws, b.s))
            return RECUR_EARG;
    return RECUR_OK;
}

bool bad_ld(const recur_config *c, int64_t ld) { return ld < c->dim || ld > INT32_MAX; }

Buf columns(const recur_config *c, const void *p, int64_t ld, int64_t T)
{
    const uint64_t e = size_of(c->dtype);
    return Buf{Span{p, (uint64_t)c->dim * e, (uint64_t)T, (uint64_t)ld * e}, e, true};
}
Buf rows_of(const recur_config *c, const void *p, int64_t T)
{
    const uint64_t e = size_of(c->dtype);
    return Buf{Span{p, (uint64_t)T * c->dim * e}, e, true};
}
Buf states_of(const recur_config *c, const void *p, int64_t n, bool needed = false)
{
    return Buf{Span{p, (uint64_t)n * c->dim * 4}, 4, needed};
}

int check_call(const recur_config *cfg, int pass, const void *ws, uint64_t ws_bytes, const recur_inputs *in,
               const int32_t *offsets, int64_t n, int64_t T)
{
    const int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!in || !ws)
        return RECUR_ENULL;
    if ((uintptr_t)ws % kAlign || (uintptr_t)offsets % 4)
        return RECUR_EALIGN;
    if (T < 0 || T > cfg->max_tokens || n < 0 || n > (int64_t(1) << 24) || (!offsets && n != 1) ||
        bad_ld(cfg, in->ldx) || bad_ld(cfg, in->ldr) || bad_ld(cfg, in->ldi) || ws_bytes < ws_need(cfg, pass))
        return RECUR_ESIZE;
    return RECUR_OK;
}

Args base(const recur_config *c, const recur_inputs *in, const float *lam, int64_t T)
{
    const int64_t e = (int64_t)size_of(c->dtype);
    Args a{};
    a.x = (const uint8_t *)in->x;
    a.r = (const uint8_t *)in->r;
    a.i = (const uint8_t *)in->i;
    a.ldx = in->ldx * e;
    a.ldr = in->ldr * e;
    a.ldi = in->ldi * e;
    a.lam = lam;
    a.T = T;
    a.D = c->dim;
    a.c = c->c;
    a.accum = (c->options & RECUR_OPT_ACCUM) != 0;
    return a;
}

int done() { return hipGetLastError() == hipSuccess ? RECUR_OK : RECUR_EHIP; }

}   // namespace
}   // namespace recur

using namespace recur;

extern "C" {

int recur_abi_version(void) { return RECUR_ABI_VERSION; }

const char *recur_status_string(int status)
{
    switch (status) {
    case RECUR_OK: return "ok";
    case RECUR_ENULL: return "a required pointer is NULL";
    case RECUR_EALIGN: return "a pointer is misaligned";
    case RECUR_ECONFIG: return "invalid config";
    case RECUR_ESIZE: return "size out of range or workspace too small";
    case RECUR_EARG: return "buffers overlap, or an unknown pass";
    case RECUR_EHIP: return "HIP runtime error";
    default: return "unknown status";
    }
}

int recur_config_check(const recur_config *cfg) { return check_config(cfg); }

int recur_workspace_bytes(const recur_config *cfg, int pass, uint64_t *bytes)
{
    const int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!bytes)
        return RECUR_ENULL;
    if (pass != RECUR_PASS_FWD && pass != RECUR_PASS_BWD)
        return RECUR_EARG;
    *bytes = ws_need(cfg, pass);
    return RECUR_OK;
}

int recur_saved_bytes(const recur_config *cfg, int64_t T, uint64_t *bytes)
{
    const int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!bytes)
        return RECUR_ENULL;
    if (T < 0 || T > cfg->max_tokens)
        return RECUR_ESIZE;
    *bytes = (uint64_t)chunks(T) * cfg->dim * 4;
    return RECUR_OK;
}

int recur_fwd(const recur_config *cfg, void *ws, uint64_t ws_bytes, const recur_inputs *in, const float *lam,
              const int32_t *offsets, int64_t n, const float *h0, int64_t T, void *y, float *hT, float *saved,
              void *stream)
{
    int rc = check_call(cfg, RECUR_PASS_FWD, ws, ws_bytes, in, offsets, n, T);
    if (rc)
        return rc;
    if ((rc = check({columns(cfg, in->x, in->ldx, T), columns(cfg, in->r, in->ldr, T), columns(cfg, in->i, in->ldi, T),
                     states_of(cfg, lam, 1, true), Buf{Span{offsets, offsets ? 4 * ((uint64_t)n + 1) : 0}, 4, false},
                     states_of(cfg, h0, n)},
                    {rows_of(cfg, y, T), states_of(cfg, hT, n), states_of(cfg, saved, chunks(T))}, Span{ws, ws_bytes})))
        return rc;
    if (n == 0 || (T == 0 && !hT))
        return RECUR_OK;
    Args a = base(cfg, in, lam, T);
    a.offsets = offsets;
    a.n = n;
    a.h0 = h0;
    a.y = (uint8_t *)y;
    a.hT = hT;
    a.saved = saved;
    const unsigned grid = (cfg->dim + 63) / 64;
    (cfg->dtype == RECUR_DTYPE_F32 ? fwd_kernel<4> : fwd_kernel<2>)<<<grid, 64, 0, (hipStream_t)stream>>>(a);
    return done();
}

int recur_bwd(const recur_config *cfg, void *ws, uint64_t ws_bytes, const recur_inputs *in, const float *lam,
              const int32_t *offsets, int64_t n, const float *h0, const float *saved, const void *dy,
              const float *dhT, int64_t T, const recur_grads *out, float *dlam, float *dh0, void *stream)
{
    int rc = check_call(cfg, RECUR_PASS_BWD, ws, ws_bytes, in, offsets, n, T);
    if (rc)
        return rc;
    if (!out)
        return RECUR_ENULL;
    if (bad_ld(cfg, out->lddx) || bad_ld(cfg, out->lddr) || bad_ld(cfg, out->lddi))
        return RECUR_ESIZE;
    if ((rc = check({columns(cfg, in->x, in->ldx, T), columns(cfg, in->r, in->ldr, T), columns(cfg, in->i, in->ldi, T),
                     states_of(cfg, lam, 1, true), Buf{Span{offsets, offsets ? 4 * ((uint64_t)n + 1) : 0}, 4, false},
                     states_of(cfg, h0, n), states_of(cfg, saved, chunks(T), true), rows_of(cfg, dy, T),
                     states_of(cfg, dhT, n)},
                    {columns(cfg, out->dx, out->lddx, T), columns(cfg, out->dr, out->lddr, T),
                     columns(cfg, out->di, out->lddi, T), states_of(cfg, dlam, 1, true), states_of(cfg, dh0, n)},
                    Span{ws, ws_bytes})))
        return rc;
    Args a = base(cfg, in, lam, T);
    a.offsets = offsets;
    a.n = n;
    a.h0 = h0;
    a.saved = const_cast<float *>(saved);
    a.dy = (const uint8_t *)dy;
    a.dhT = dhT;
    const int64_t e = (int64_t)size_of(cfg->dtype);
    a.dx = (uint8_t *)out->dx;
    a.dr = (uint8_t *)out->dr;
    a.di = (uint8_t *)out->di;
    a.lddx = out->lddx * e;
    a.lddr = out->lddr * e;
    a.lddi = out->lddi * e;
    a.dlam = dlam;
    a.dh0 = dh0;
    const unsigned grid = (cfg->dim + 63) / 64;
    (cfg->dtype == RECUR_DTYPE_F32 ? bwd_kernel<4> : bwd_kernel<2>)<<<grid, 64, 0, (hipStream_t)stream>>>(a);
    return done();
}

int recur_step(const recur_config *cfg, const recur_inputs *in, const float *lam, float *state, int64_t states,
               const int32_t *slots, int64_t n, void *y, void *stream)
{
    int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!in)
        return RECUR_ENULL;
    if (n < 0 || n > (int64_t(1) << 20) || states < 0 || states > INT32_MAX || (!slots && states < n) ||
        bad_ld(cfg, in->ldx) || bad_ld(cfg, in->ldr) || bad_ld(cfg, in->ldi))
        return RECUR_ESIZE;
    if ((rc = check({columns(cfg, in->x, in->ldx, n), columns(cfg, in->r, in->ldr, n), columns(cfg, in->i, in->ldi, n),
                     states_of(cfg, lam, 1, true), Buf{Span{slots, slots ? 4 * (uint64_t)n : 0}, 4, false}},
                    {rows_of(cfg, y, n), states_of(cfg, state, states, true)}, Span{nullptr, 0})))
        return rc;
    if (n == 0)
        return RECUR_OK;
    Args a = base(cfg, in, lam, n);
    a.y = (uint8_t *)y;
    a.n = n;
    const dim3 grid((cfg->dim + 63) / 64, (unsigned)n);
    (cfg->dtype == RECUR_DTYPE_F32 ? step_kernel<4> : step_kernel<2>)<<<grid, 64, 0, (hipStream_t)stream>>>(
        a, state, states, slots);
    return done();
}

}   // extern "C"
