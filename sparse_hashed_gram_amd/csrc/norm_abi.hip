// Entry points of include/norm.h, and the last step of the backward: the
// parameters' gradients from the blocks' parts.
#include <initializer_list>

#include "norm_dev.hpp"
#include "spans.hpp"

namespace rownorm {
namespace {

using spans::meet;
using spans::Span;

constexpr uint64_t kAlign = 256;

// v, added to what is there if `accum`, rounded once.
__device__ __forceinline__ void put_grad(void *to, int j, int f32, int accum, float v)
{
    if (f32) {
        float *p = reinterpret_cast<float *>(to) + j;
        *p = accum ? *p + v : v;
    } else {
        uint16_t *p = reinterpret_cast<uint16_t *>(to) + j;
        const float old = accum ? __uint_as_float((uint32_t)*p << 16) : 0.0f;
        *p = (uint16_t)ngram::bf16_pack_rne(old + v, 0.0f);
    }
}

// a b, rounded by itself and not fused into the sum of an accumulated gradient.
__device__ __forceinline__ float alone(float a, float b)
{
#pragma clang fp contract(off)
    return a * b;
}

__device__ __forceinline__ float param_at(const uint8_t *p, int f32, int one, int j, float none)
{
    if (!p)
        return none;
    if (one)
        j = 0;
    return f32 ? reinterpret_cast<const float *>(p)[j]
               : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[j] << 16);
}

// Column sums over the parts, in a fixed order: 16 columns a block, 64 threads to
// a column.  blockIdx.y: the norm in front, the norm and gate behind, the scale.
__global__ __launch_bounds__(1024) void grad_kernel(GradArgs a)
{
    __shared__ float lds[2][16][16];
    const int c = threadIdx.x % 16, g = threadIdx.x / 16, j = blockIdx.x * 16 + c;
    const int ld = (a.D + 3) / 4 * 4, what = blockIdx.y;
    const int first = what == 0 ? kSumPreW : what == 1 ? kSumPost1 : kSumScale;
    const int second = what == 0 ? (a.db ? kSumPreB : -1)
                     : what == 1 ? (a.dpost_b || (a.dgate && a.p.post_b) ? kSumPost0 : -1) : -1;
    float x = 0.0f, y = 0.0f;   // without a second sum, y is the first again and not looked at
    if (j < a.D) {
        const float *p = a.part + (int64_t)g * kSums * ld + j + first * ld;
        const int apart = second >= 0 ? (second - first) * ld : 0;
#pragma unroll 8
        for (int i = g; i < a.parts; i += 64, p += 64 * kSums * ld) {
            x += p[0];
            y += p[apart];
        }
    }
    x += __shfl_xor(x, 16);
    y += __shfl_xor(y, 16);
    x += __shfl_xor(x, 32);
    y += __shfl_xor(y, 32);
    if (g % 4 == 0) {
        lds[0][g / 4][c] = x;
        lds[1][g / 4][c] = y;
    }
    __syncthreads();
    if (g != 0 || j >= a.D)
        return;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
        x += lds[0][i][c];
        y += lds[1][i][c];
    }
    if (what == 0) {
        if (a.dw)
            put_grad(a.dw, j, a.f32, a.accum, x);
        if (a.db)
            put_grad(a.db, j, a.f32, a.accum, y);
    } else if (what == 1) {
        // x = sum E nh, y = sum E (a token's gate is in them already)
        const float gate = a.gate_token ? 1.0f : param_at(a.p.gate, a.p.f32, a.p.gate_one, j, 1.0f);
        if (a.dpost_w)
            put_grad(a.dpost_w, j, a.f32, a.accum, alone(gate, x));
        if (a.dpost_b)
            put_grad(a.dpost_b, j, a.f32, a.accum, alone(gate, y));
        if (a.dgate) {
            float v = x;
            if (a.post)
                v = alone(v, param_at(a.p.post_w, a.p.f32, 0, j, 1.0f));
            if (a.post && a.p.post_b)
                v += alone(param_at(a.p.post_b, a.p.f32, 0, j, 0.0f), y);
            if (a.p.gate_one)
                a.cols[j] = v;
            else
                put_grad(a.dgate, j, a.f32, a.accum, v);
        }
    } else {
        if (a.p.scale_one)
            a.cols[ld + j] = x;
        else
            put_grad(a.dscale, j, a.f32, a.accum, x);
    }
}

// A scalar's gradient from its column sums.  blockIdx.x: gate, scale.
__global__ __launch_bounds__(256) void scalar_kernel(GradArgs a)
{
    __shared__ float lds[4];
    const bool gate = blockIdx.x == 0;
    void *to = gate ? a.dgate : a.dscale;
    if (!to || !(gate ? a.p.gate_one : a.p.scale_one))
        return;
    const float *v = a.cols + (gate ? 0 : (a.D + 3) / 4 * 4);
    float s = 0.0f;
    for (int j = threadIdx.x; j < a.D; j += 256)
        s += v[j];
    s = ngram::wave_sum(s);
    if (threadIdx.x % 64 == 0)
        lds[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        put_grad(to, 0, a.f32, a.accum, (lds[0] + lds[1]) + (lds[2] + lds[3]));
}

uint64_t align_up(uint64_t n) { return (n + kAlign - 1) / kAlign * kAlign; }
uint64_t part_bytes(int D) { return align_up((uint64_t)kMaxBlocks * kSums * padded(D) * 4); }
uint64_t ws_need(int D) { return part_bytes(D) + align_up((uint64_t)2 * padded(D) * 4); }

uint64_t size_of(int dtype) { return dtype == NORM_DTYPE_F32 ? 4 : 2; }

// A buffer of a call: where, its bytes, its elements' size, and whether it has
// to be there.
struct Buf {
    const void *p;
    uint64_t bytes;
    uint64_t elt;
    bool needed;
};

// ins x outs may not meet, but outs[0] may be `in_place`, whole.
int check(std::initializer_list<Buf> ins, std::initializer_list<Buf> outs, const void *in_place, const Span &ws)
{
    for (const auto *l : {&ins, &outs})
        for (const Buf &b : *l) {
            if (b.needed && b.bytes && !b.p)
                return NORM_ENULL;
            if ((uintptr_t)b.p % b.elt)
                return NORM_EALIGN;
        }
    const Buf *o = outs.begin();
    for (size_t i = 0; i < outs.size(); ++i) {
        const Span out{o[i].p, o[i].bytes};
        for (const Buf &b : ins)
            if (!(i == 0 && b.p == in_place && b.p == out.p) && meet(out, Span{b.p, b.bytes}))
                return NORM_EARG;
        for (size_t k = 0; k < i; ++k)
            if (meet(out, Span{o[k].p, o[k].bytes}))
                return NORM_EARG;
        if (meet(out, ws))
            return NORM_EARG;
    }
    for (const Buf &b : ins)
        if (meet(ws, Span{b.p, b.bytes}))
            return NORM_EARG;
    return NORM_OK;
}

int check_ws(const norm_config *cfg, const void *ws, uint64_t ws_bytes)
{
    if (!ws)
        return NORM_ENULL;
    if ((uintptr_t)ws % kAlign)
        return NORM_EALIGN;
    return ws_bytes < ws_need(cfg->dim) ? NORM_ESIZE : NORM_OK;
}

int check_config(const norm_config *c)
{
    if (!c)
        return NORM_ENULL;
    auto type = [](int t) { return t == NORM_DTYPE_F32 || t == NORM_DTYPE_BF16; };
    const bool ok = c->dim >= 1 && c->dim <= 4096 && (c->kind == NORM_KIND_RMS || c->kind == NORM_KIND_LAYER) &&
                    type(c->x_dtype) && type(c->r_dtype) && type(c->p_dtype) && type(c->dp_dtype) &&
                    !(c->x_dtype == NORM_DTYPE_F32 && c->r_dtype != NORM_DTYPE_F32) && c->gate >= NORM_BY_NONE &&
                    c->gate <= NORM_BY_TOKEN && c->scale >= NORM_BY_NONE && c->scale <= NORM_BY_VECTOR &&
                    (c->options & ~(NORM_OPT_PRE | NORM_OPT_POST | NORM_OPT_ACCUM)) == 0 && c->eps >= 1e-12f &&
                    c->eps <= 1.0f;
    return ok ? NORM_OK : NORM_ECONFIG;
}

bool bad_rows(int64_t T) { return T < 0 || T > INT32_MAX; }

Args base(const norm_config *c, int64_t T)
{
    Args a{};
    a.T = T;
    a.D = c->dim;
    a.layer = c->kind == NORM_KIND_LAYER;
    a.pre = 1;
    a.eps = c->eps;
    a.inv_d = 1.0f / (float)c->dim;
    a.p.f32 = c->p_dtype == NORM_DTYPE_F32;
    a.p.gate_one = c->gate == NORM_BY_SCALAR;
    a.p.scale_one = c->scale == NORM_BY_SCALAR;
    return a;
}

int done() { return hipGetLastError() == hipSuccess ? NORM_OK : NORM_EHIP; }

const uint8_t *in(const void *p) { return (const uint8_t *)p; }
uint8_t *out(void *p) { return (uint8_t *)p; }

uint64_t count_of(int by, int dim) { return by == NORM_BY_SCALAR ? 1 : by == NORM_BY_VECTOR ? dim : 0; }

int gradients(const norm_config *c, const Args &a, const norm_grads &g, int parts, float *cols, bool join, hipStream_t s)
{
    GradArgs d{};
    d.part = a.part;
    d.cols = cols;
    d.p = a.p;
    d.dw = a.pre ? g.dw : nullptr;
    d.db = a.pre ? g.db : nullptr;
    if (join) {
        d.gate_token = c->gate == NORM_BY_TOKEN;
        d.post = a.post;
        d.dpost_w = a.post ? g.dpost_w : nullptr;
        d.dpost_b = a.post ? g.dpost_b : nullptr;
        d.dgate = c->gate == NORM_BY_SCALAR || c->gate == NORM_BY_VECTOR ? g.dgate : nullptr;
        d.dscale = c->scale != NORM_BY_NONE ? g.dscale : nullptr;
    }
    d.D = c->dim;
    d.parts = parts;
    d.f32 = c->dp_dtype == NORM_DTYPE_F32;
    d.accum = (c->options & NORM_OPT_ACCUM) != 0;
    const bool post = d.dpost_w || d.dpost_b || d.dgate;
    if (!d.dw && !d.db && !post && !d.dscale)
        return done();
    const dim3 grid((c->dim + 15) / 16, d.dscale ? 3 : post ? 2 : 1);
    grad_kernel<<<grid, 1024, 0, s>>>(d);
    if ((d.dgate && d.p.gate_one) || (d.dscale && d.p.scale_one))
        scalar_kernel<<<2, 256, 0, s>>>(d);
    return done();
}

}   // namespace
}   // namespace rownorm

using namespace rownorm;

extern "C" {

int norm_abi_version(void) { return NORM_ABI_VERSION; }

const char *norm_status_string(int status)
{
    switch (status) {
    case NORM_OK: return "ok";
    case NORM_ENULL: return "a required pointer is NULL";
    case NORM_EALIGN: return "a pointer is misaligned";
    case NORM_ECONFIG: return "invalid config";
    case NORM_ESIZE: return "size out of range or workspace too small";
    case NORM_EARG: return "buffers overlap";
    case NORM_EHIP: return "HIP runtime error";
    default: return "unknown status";
    }
}

int norm_config_check(const norm_config *cfg) { return check_config(cfg); }

int norm_workspace_bytes(const norm_config *cfg, uint64_t *bytes)
{
    const int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!bytes)
        return NORM_ENULL;
    *bytes = ws_need(cfg->dim);
    return NORM_OK;
}

int norm_fwd(const norm_config *cfg, const void *R, const void *w, const void *b, int64_t T, void *X, void *stream)
{
    int rc = check_config(cfg);
    if (rc)
        return rc;
    if (bad_rows(T))
        return NORM_ESIZE;
    const uint64_t re = size_of(cfg->r_dtype), xe = size_of(cfg->x_dtype), pe = size_of(cfg->p_dtype), D = cfg->dim;
    const uint64_t n = (uint64_t)T * D;
    if ((rc = check({{R, n * re, re, true}, {w, D * pe, pe, false}, {b, D * pe, pe, false}}, {{X, n * xe, xe, true}},
                    nullptr, Span{nullptr, 0})))
        return rc;
    if (T == 0)
        return NORM_OK;
    Args a = base(cfg, T);
    a.R = in(R);
    a.X = out(X);
    a.p.w = in(w);
    a.p.b = in(b);
    launch_fwd(a, cfg->x_dtype, cfg->r_dtype, (hipStream_t)stream);
    return done();
}

int norm_bwd(const norm_config *cfg, void *ws, uint64_t ws_bytes, const void *R, const void *dX, const void *dR1,
             const void *w, int64_t T, void *dR, void *dw, void *db, void *stream)
{
    int rc = check_config(cfg);
    if (rc)
        return rc;
    if (bad_rows(T))
        return NORM_ESIZE;
    if ((rc = check_ws(cfg, ws, ws_bytes)))
        return rc;
    const uint64_t re = size_of(cfg->r_dtype), xe = size_of(cfg->x_dtype), pe = size_of(cfg->p_dtype);
    const uint64_t ge = size_of(cfg->dp_dtype), D = cfg->dim, n = (uint64_t)T * D;
    if ((rc = check({{R, n * re, re, true}, {dX, n * xe, xe, true}, {dR1, n * re, re, false}, {w, D * pe, pe, false}},
                    {{dR, n * re, re, true}, {dw, D * ge, ge, false}, {db, D * ge, ge, false}}, dR1, Span{ws, ws_bytes})))
        return rc;
    if (T == 0 && (cfg->options & NORM_OPT_ACCUM))
        return NORM_OK;
    Args a = base(cfg, T);
    a.R1in = in(R);
    a.dX = in(dX);
    a.dR1 = in(dR1);
    a.dR = out(dR);
    a.p.w = in(w);
    a.part = (float *)ws;
    hipStream_t s = (hipStream_t)stream;
    const int parts = T ? launch_bwd(a, cfg->x_dtype, cfg->r_dtype, db != nullptr, s) : 0;
    return gradients(cfg, a, norm_grads{nullptr, nullptr, nullptr, nullptr, dw, db}, parts, nullptr, false, s);
}

int norm_join_fwd(const norm_config *cfg, const void *R, const void *B, const norm_params *p, int64_t T, void *R1,
                  void *X, void *stream)
{
    int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!p)
        return NORM_ENULL;
    if (bad_rows(T))
        return NORM_ESIZE;
    const bool pre = cfg->options & NORM_OPT_PRE, post = cfg->options & NORM_OPT_POST, token = cfg->gate == NORM_BY_TOKEN;
    const uint64_t re = size_of(cfg->r_dtype), xe = size_of(cfg->x_dtype), pe = size_of(cfg->p_dtype), D = cfg->dim;
    const uint64_t n = (uint64_t)T * D, gates = count_of(cfg->gate, cfg->dim) * pe;
    if ((rc = check({{R, n * re, re, true},
                     {B, n * xe, xe, true},
                     {p->post_w, post ? D * pe : 0, pe, false},
                     {p->post_b, post ? D * pe : 0, pe, false},
                     {p->gate, token ? n * xe : gates, token ? xe : pe, cfg->gate != NORM_BY_NONE},
                     {p->scale, count_of(cfg->scale, cfg->dim) * pe, pe, cfg->scale != NORM_BY_NONE},
                     {p->w, pre ? D * pe : 0, pe, false},
                     {p->b, pre ? D * pe : 0, pe, false}},
                    {{R1, n * re, re, true}, {X, pre ? n * xe : 0, xe, pre}}, R, Span{nullptr, 0})))
        return rc;
    if (T == 0)
        return NORM_OK;
    Args a = base(cfg, T);
    a.R = in(R);
    a.B = in(B);
    a.G = token ? in(p->gate) : nullptr;
    a.R1 = out(R1);
    a.X = out(X);
    a.post = post;
    a.pre = pre;
    a.p.post_w = post ? in(p->post_w) : nullptr;
    a.p.post_b = post ? in(p->post_b) : nullptr;
    a.p.gate = cfg->gate == NORM_BY_NONE || token ? nullptr : in(p->gate);
    a.p.scale = cfg->scale == NORM_BY_NONE ? nullptr : in(p->scale);
    a.p.w = pre ? in(p->w) : nullptr;
    a.p.b = pre ? in(p->b) : nullptr;
    launch_fwd(a, cfg->x_dtype, cfg->r_dtype, (hipStream_t)stream);
    return done();
}

int norm_join_bwd(const norm_config *cfg, void *ws, uint64_t ws_bytes, const void *R, const void *B, const void *R1,
                  const void *dX, const void *dR1, const norm_params *p, int64_t T, void *dR, void *dB,
                  const norm_grads *g, void *stream)
{
    int rc = check_config(cfg);
    if (rc)
        return rc;
    if (!p || !g)
        return NORM_ENULL;
    if (bad_rows(T))
        return NORM_ESIZE;
    if ((rc = check_ws(cfg, ws, ws_bytes)))
        return rc;
    const bool pre = cfg->options & NORM_OPT_PRE, post = cfg->options & NORM_OPT_POST, token = cfg->gate == NORM_BY_TOKEN;
    const uint64_t re = size_of(cfg->r_dtype), xe = size_of(cfg->x_dtype), pe = size_of(cfg->p_dtype);
    const uint64_t ge = size_of(cfg->dp_dtype), D = cfg->dim, n = (uint64_t)T * D;
    const uint64_t gates = count_of(cfg->gate, cfg->dim), scales = count_of(cfg->scale, cfg->dim);
    const bool need_r = cfg->scale != NORM_BY_NONE && g->dscale;
    if ((rc = check({{R, need_r ? n * re : 0, re, need_r},
                     {B, n * xe, xe, true},
                     {R1, pre ? n * re : 0, re, pre},
                     {dX, pre ? n * xe : 0, xe, pre},
                     {dR1, n * re, re, !pre},
                     {p->post_w, post ? D * pe : 0, pe, false},
                     {p->post_b, post ? D * pe : 0, pe, false},
                     {p->gate, token ? n * xe : gates * pe, token ? xe : pe, cfg->gate != NORM_BY_NONE},
                     {p->scale, scales * pe, pe, cfg->scale != NORM_BY_NONE},
                     {p->w, pre ? D * pe : 0, pe, false}},
                    {{dR, n * re, re, true},
                     {dB, n * xe, xe, true},
                     {g->dpost_w, post ? D * ge : 0, ge, false},
                     {g->dpost_b, post ? D * ge : 0, ge, false},
                     {g->dgate, token ? n * xe : gates * ge, token ? xe : ge, false},
                     {g->dscale, scales * ge, ge, false},
                     {g->dw, pre ? D * ge : 0, ge, false},
                     {g->db, pre ? D * ge : 0, ge, false}},
                    dR1, Span{ws, ws_bytes})))
        return rc;
    if (T == 0 && (cfg->options & NORM_OPT_ACCUM))
        return NORM_OK;
    Args a = base(cfg, T);
    a.R = need_r ? in(R) : nullptr;
    a.B = in(B);
    a.G = token ? in(p->gate) : nullptr;
    a.R1in = in(R1);
    a.dX = in(dX);
    a.dR1 = in(dR1);
    a.dR = out(dR);
    a.dB = out(dB);
    a.dG = token ? out(g->dgate) : nullptr;
    a.post = post;
    a.pre = pre;
    a.p.post_w = post ? in(p->post_w) : nullptr;
    a.p.post_b = post ? in(p->post_b) : nullptr;
    a.p.gate = cfg->gate == NORM_BY_NONE || token ? nullptr : in(p->gate);
    a.p.scale = cfg->scale == NORM_BY_NONE ? nullptr : in(p->scale);
    a.p.w = pre ? in(p->w) : nullptr;
    a.part = (float *)ws;
    const bool gate_sums = gates && g->dgate;
    const bool extra = (pre && g->db) || (post && (g->dpost_b || (gate_sums && p->post_b))) || need_r;
    hipStream_t s = (hipStream_t)stream;
    const int parts = T ? launch_bwd(a, cfg->x_dtype, cfg->r_dtype, extra, s) : 0;
    float *cols = (float *)((uint8_t *)ws + part_bytes(cfg->dim));
    return gradients(cfg, a, *g, parts, cols, true, s);
}

}   // extern "C"
