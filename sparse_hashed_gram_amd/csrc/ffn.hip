// Gated feed-forward block on gfx950, forward and backward (the formulas and
// the rounding points are in include/ffn.h).
//
//   up_kernel     H = a(X Wg^T) * (X Wu^T)                  -> workspace, bf16
//   rows_kernel   Y = (res +) drop(H Wd^T); dX = dG Wg + dU Wu (one contraction over 2 F)
//   grad_kernel   G, U again, dH = dY' Wd -> dG, dU, H       -> workspace, bf16
//   dw_kernel     dWg, dWu, dWd in one launch, k = T, in parts where the tiles alone
//                 do not fill the chip; dw_reduce_kernel adds the parts in order
//
// Every product is a block tile of mfma_tile.hpp.  Weights are read as they
// lie: where k runs over a weight's rows (dH, dX) or over positions (the weights'
// gradients) the operand is k-major and comes through the LDS transpose read,
// so nothing is transposed in memory.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ffn.h"
#include "mfma_tile.hpp"
#include "ngram_dev.hpp"
#include "philox.hpp"

namespace {

using namespace tile;

constexpr int kD = 768;
constexpr int kMaxParts = 8;     // parts of k of the weights' gradients
constexpr uint64_t kAlign = 256;
constexpr uint32_t kCUs = 256, kXcds = 8;

inline int64_t rup(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// ------------------------------------------------------------- block order

// The hardware hands consecutive workgroups to the 8 XCDs in turn.  Each XCD
// gets a contiguous range of tiles, walked in groups of 8 tiles of positions
// (all weight tiles of a group before the next group), so the blocks that are
// resident on an XCD share their operands in its L2.
constexpr uint32_t kGroup = 8;

__host__ __device__ inline uint32_t grid_blocks(uint32_t tiles) { return kXcds * ((tiles + kXcds - 1) / kXcds); }

// rows: tiles of positions, cols: tiles of the other side
__device__ inline bool tile_of(uint32_t rows, uint32_t cols, uint32_t &rt, uint32_t &ct)
{
    const uint32_t total = rows * cols, per = (total + kXcds - 1) / kXcds;
    const uint32_t t = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
    if (blockIdx.x / kXcds >= per || t >= total)
        return false;
    const uint32_t span = kGroup * cols, g = t / span, first = g * kGroup;
    const uint32_t gm = rows - first < kGroup ? rows - first : kGroup;
    const uint32_t r = t - g * span;
    rt = first + r % gm;
    ct = r / gm;
    return true;
}

// ---------------------------------------------------------------- epilogue

// Writes a wavefront's 32 MB x 32 block out as rows: val(mb, e) is the value at
// m = 32 mb + 8 (e / 4) + 4 (lane / 32) + e % 4, n = lane % 32, and
// out(n, m, v) takes 8 consecutive m of one n.  Through the wavefront's own piece of
// LDS in fp32 (rows padded by 16 bytes: no bank conflicts), so whole rows leave
// in 16-byte stores and each lane of the last step holds one mask group.
template <int MB>
struct Rows {
    static constexpr int LD = 32 * MB + 4;
    static constexpr uint32_t BYTES = 32 * LD * 4;   // per wavefront

    template <typename V, typename O>
    static __device__ __forceinline__ void write(float *lds, V val, O out)
    {
        const int lane = threadIdx.x & 63;
        float *p = lds + (lane & 31) * LD + 4 * (lane >> 5);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *(float4 *)(p + 32 * mb + 8 * q) =
                    make_float4(val(mb, 4 * q), val(mb, 4 * q + 1), val(mb, 4 * q + 2), val(mb, 4 * q + 3));
        __builtin_amdgcn_wave_barrier();
        constexpr int PER = 4 * MB;   // lanes per row
        constexpr int STEP = 64 / PER;
#pragma unroll
        for (int i = 0; i < 32 / STEP; ++i) {
            const int n = i * STEP + lane / PER, m = 8 * (lane % PER);
            const float4 a = *(const float4 *)(lds + n * LD + m), b = *(const float4 *)(lds + n * LD + m + 4);
            float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            out(n, m, v);
        }
        __builtin_amdgcn_wave_barrier();
    }
};

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    using ngram::bf16_pack_rne;
    return make_uint4(bf16_pack_rne(v[0], v[1]), bf16_pack_rne(v[2], v[3]), bf16_pack_rne(v[4], v[5]),
                      bf16_pack_rne(v[6], v[7]));
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = ngram::bf16_lo(u[k]);
        v[2 * k + 1] = ngram::bf16_hi(u[k]);
    }
}

// 8 elements at index i of an fp32 or bf16 array
__device__ __forceinline__ void load_as(const void *p, bool f32, int64_t i, float (&v)[8])
{
    if (f32) {
        const float4 *q = reinterpret_cast<const float4 *>((const float *)p + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4 *>((const uint16_t *)p + i), v);
    }
}

__device__ __forceinline__ void store_as(void *p, bool f32, int64_t i, const float (&v)[8])
{
    if (f32) {
        float4 *q = reinterpret_cast<float4 *>((float *)p + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>((uint16_t *)p + i) = pack8(v);
    }
}

// -------------------------------------------------------------- activation

constexpr float kG1 = 0.7978845608028654f, kG3 = 0.044715f;   // sqrt(2 / pi)

// 1 / (1 + exp(-x)): exp overflows to inf for x below -88 and gives 0, as it should
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + __expf(-x)); }

// a(g) and, if D, a'(g).  GELU: (1 + tanh z) / 2 = sigmoid(2 z).
template <int ACT, bool D>
__device__ __forceinline__ float act(float g, float &d)
{
    if constexpr (ACT == FFN_ACT_SILU) {
        const float s = sigmoid(g), a = g * s;
        if (D)
            d = s + a * (1.0f - s);
        return a;
    } else if constexpr (ACT == FFN_ACT_GELU) {
        const float c = __builtin_amdgcn_fmed3f(g, -1e4f, 1e4f);   // far past both ends; c^2 stays finite
        const float g2 = c * c, s = sigmoid(2.0f * kG1 * c * (1.0f + kG3 * g2)), a = g * s;
        if (D)
            d = s + a * (1.0f - s) * (2.0f * kG1) * (1.0f + 3.0f * kG3 * g2);
        return a;
    } else {
        const float r = g < 0.0f ? 0.0f : g;   // a NaN stays one
        if (D)
            d = 2.0f * r;
        return r * r;
    }
}

// ------------------------------------------------------------------ kernels

// Tiles: WM x WN matrix-core tiles of 32 x 32 per wavefront, 2 x 2 wavefronts.
constexpr int kWM = 2, kWN = 2, kGM = 2, kGN = 2, kNS = 2, kThreads = 64 * kGM * kGN;
constexpr int kBM = 32 * kWM * kGM, kBN = 32 * kWN * kGN;

struct Args {
    const uint16_t *X, *Wg, *Wu, *Wd, *dY;
    uint16_t *S;             // workspace: forward H [T][Fp]; backward [T][3 Fp] dG | dU | H
    int64_t T, F, Fp;
    uint32_t tiles_t, tiles_o;
    const void *res;
    void *out;
    int32_t out_f32;
    drop::Mask mask;
};

__device__ __forceinline__ Operand rows_of(const uint16_t *p, int64_t ld, int64_t first, int64_t count, int64_t k)
{
    return Operand{{p, p}, ld, first, count, INT64_MAX, k, 0};
}

constexpr uint32_t cmax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int MB>
constexpr uint32_t smem_for(uint32_t main)
{
    return cmax(main, kGM * kGN * Rows<MB>::BYTES);
}

// H tile of kBN positions x kBM / 2 hidden units: each wavefront holds its
// units' gate sums in the first half of its m-blocks and the up sums in the
// second, so both meet in one lane.
template <int ACT>
__global__ __launch_bounds__(kThreads) void up_kernel(Args a)
{
    using T0 = Tile<false, false, kWM, kWN, kGM, kGN, kNS>;
    constexpr int HB = kWM / 2;
    __shared__ __align__(16) uint8_t sm[smem_for<HB>(T0::SMEM)];
    uint32_t tt, ot;
    if (!tile_of(a.tiles_t, a.tiles_o, tt, ot))
        return;
    const int64_t n0 = (int64_t)tt * kBN, f0 = (int64_t)ot * (kBM / 2);
    f32x16 acc[kWM][kWN];
    clear(acc);
    const Operand A{{a.Wg, a.Wu}, kD, f0, a.F, INT64_MAX, kD, 32 * HB};
    product<false, false, kWM, kWN, kGM, kGN, kNS>(A, rows_of(a.X, kD, n0, a.T, kD), kD, sm, acc);
    const int w = threadIdx.x >> 6, wm = w / kGN, wn = w % kGN;
    float *lds = reinterpret_cast<float *>(sm + w * Rows<HB>::BYTES);
    const int64_t fw = f0 + wm * 32 * HB;
#pragma unroll
    for (int nb = 0; nb < kWN; ++nb) {
        const int64_t tw = n0 + (wn * kWN + nb) * 32;
        Rows<HB>::write(
            lds,
            [&](int mb, int e) {
                float d;
                return act<ACT, false>(acc[mb][nb][e], d) * acc[mb + HB][nb][e];
            },
            [&](int n, int m, const float (&v)[8]) {
                const int64_t t = tw + n, f = fw + m;
                if (t < a.T && f < a.F)
                    *reinterpret_cast<uint4 *>(a.S + t * a.Fp + f) = pack8(v);
            });
    }
}

// A [T][768] result: DX false: Y = (res +) drop(H Wd^T); true: dX = [dG | dU] [Wg; Wu].
template <bool DX>
__global__ __launch_bounds__(kThreads) void rows_kernel(Args a)
{
    using T0 = Tile<DX, false, kWM, kWN, kGM, kGN, kNS>;
    __shared__ __align__(16) uint8_t sm[smem_for<kWM>(T0::SMEM)];
    uint32_t tt, ot;
    if (!tile_of(a.tiles_t, a.tiles_o, tt, ot))
        return;
    const int64_t n0 = (int64_t)tt * kBN, d0 = (int64_t)ot * kBM;
    f32x16 acc[kWM][kWN];
    clear(acc);
    if constexpr (DX) {
        const Operand A{{a.Wg, a.Wu}, kD, d0, kD, a.Fp, a.F, 0};
        const Operand B{{a.S, a.S}, 3 * a.Fp, n0, a.T, a.Fp, a.F, 0};
        product<true, false, kWM, kWN, kGM, kGN, kNS>(A, B, 2 * a.Fp, sm, acc);
    } else {
        product<false, false, kWM, kWN, kGM, kGN, kNS>(rows_of(a.Wd, a.F, d0, kD, a.F),
                                                       rows_of(a.S, a.Fp, n0, a.T, a.F), a.Fp, sm, acc);
    }
    const int w = threadIdx.x >> 6, wm = w / kGN, wn = w % kGN;
    float *lds = reinterpret_cast<float *>(sm + w * Rows<kWM>::BYTES);
    const drop::Key key = drop::key_of(a.mask);
#pragma unroll
    for (int nb = 0; nb < kWN; ++nb) {
        const int64_t tw = n0 + (wn * kWN + nb) * 32, dw = d0 + wm * 32 * kWM;
        Rows<kWM>::write(
            lds, [&](int mb, int e) { return acc[mb][nb][e]; },
            [&](int n, int m, float (&v)[8]) {
                const int64_t t = tw + n, i = t * kD + dw + m;
                if (t >= a.T)
                    return;
                if (!DX && a.mask.thr != 0) {
                    const uint4 bits = drop::bits_of(key, (uint64_t)i / 8);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = drop::dropped(v[e], bits, e, a.mask.thr, a.mask.scale);
                }
                if (!DX && a.res) {
                    float r[8];
                    load_as(a.res, a.out_f32, i, r);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] += r[e];
                }
                store_as(a.out, a.out_f32, i, v);
            });
    }
}

// dG, dU and H of kBN positions x kBM / 2 hidden units: the gate and up sums
// again as in up_kernel, then dH of the same tile.
template <int ACT>
__global__ __launch_bounds__(kThreads) void grad_kernel(Args a)
{
    constexpr int HB = kWM / 2;
    using T0 = Tile<false, false, kWM, kWN, kGM, kGN, kNS>;
    using T1 = Tile<true, false, HB, kWN, kGM, kGN, kNS>;
    __shared__ __align__(16) uint8_t sm[smem_for<HB>(cmax(T0::SMEM, T1::SMEM))];
    uint32_t tt, ot;
    if (!tile_of(a.tiles_t, a.tiles_o, tt, ot))
        return;
    const int64_t n0 = (int64_t)tt * kBN, f0 = (int64_t)ot * (kBM / 2);
    f32x16 acc[kWM][kWN], dh[HB][kWN];
    clear(acc);
    clear(dh);
    const Operand A{{a.Wg, a.Wu}, kD, f0, a.F, INT64_MAX, kD, 32 * HB};
    product<false, false, kWM, kWN, kGM, kGN, kNS>(A, rows_of(a.X, kD, n0, a.T, kD), kD, sm, acc);
    product<true, false, HB, kWN, kGM, kGN, kNS>(rows_of(a.Wd, a.F, f0, a.F, kD),
                                                 rows_of(a.dY, kD, n0, a.T, kD), kD, sm, dh);
    const int w = threadIdx.x >> 6, wm = w / kGN, wn = w % kGN;
    float *lds = reinterpret_cast<float *>(sm + w * Rows<HB>::BYTES);
    const int64_t fw = f0 + wm * 32 * HB;
#pragma unroll
    for (int nb = 0; nb < kWN; ++nb) {
        const int64_t tw = n0 + (wn * kWN + nb) * 32;
        auto put = [&](int which) {
            return [&, which](int n, int m, const float (&v)[8]) {
                const int64_t t = tw + n, f = fw + m;
                if (t < a.T && f < a.F)
                    *reinterpret_cast<uint4 *>(a.S + t * 3 * a.Fp + which * a.Fp + f) = pack8(v);
            };
        };
        // H, then dU over the gate sums' place, dG over the up sums'
        Rows<HB>::write(
            lds,
            [&](int mb, int e) {
                const float g = acc[mb][nb][e], u = acc[mb + HB][nb][e], h = a.mask.scale * dh[mb][nb][e];
                float d;
                const float s = act<ACT, true>(g, d);
                acc[mb][nb][e] = h * s;
                acc[mb + HB][nb][e] = h * u * d;
                return s * u;
            },
            put(2));
        Rows<HB>::write(lds, [&](int mb, int e) { return acc[mb][nb][e]; }, put(1));
        Rows<HB>::write(lds, [&](int mb, int e) { return acc[mb + HB][nb][e]; }, put(0));
    }
}

struct DwArgs {
    const uint16_t *X, *dY, *S;
    int64_t T, F, Fp;
    uint32_t tiles_f2, tiles_d;     // dWg and dWu: tiles of 2 Fp rows x 768
    uint32_t tiles_e, tiles_h;      // dWd: tiles of 768 rows x F
    int32_t parts;
    float *part;                    // [parts][2 Fp 768 + 768 Fp] where parts > 1
    void *dWg, *dWu, *dWd;
    int32_t dw_f32, accum;
    float scale;                    // of dY' (the mask alone is in dY)
};

__device__ __forceinline__ void put_dw(const DwArgs &a, void *dst, int64_t i, float scale, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] *= scale;
    if (a.accum) {
        float o[8];
        load_as(dst, a.dw_f32, i, o);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += o[e];
    }
    store_as(dst, a.dw_f32, i, v);
}

// One tile of one part of k: rows n of the result with m contiguous.
//   dWg | dWu: n = f of 2 Fp (B = dG | dU), m = d (A = X)
//   dWd:       n = d (B = dY'),             m = f (A = H)
__global__ __launch_bounds__(kThreads) void dw_kernel(DwArgs a)
{
    using T0 = Tile<true, true, kWM, kWN, kGM, kGN, kNS>;
    __shared__ __align__(16) uint8_t sm[smem_for<kWM>(T0::SMEM)];
    const uint32_t first = a.tiles_f2 * a.tiles_d, tiles = first + a.tiles_e * a.tiles_h;
    uint32_t part, ti;
    {
        // parts outermost: the blocks that run together share their rows of k
        const uint32_t total = tiles * (uint32_t)a.parts, per = (total + kXcds - 1) / kXcds;
        const uint32_t t = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
        if (blockIdx.x / kXcds >= per || t >= total)
            return;
        part = t / tiles;
        ti = t % tiles;
    }
    const bool down = ti >= first;
    int64_t n0, m0;
    if (!down) {
        n0 = (int64_t)(ti / a.tiles_d) * kBN;
        m0 = (int64_t)(ti % a.tiles_d) * kBM;
    } else {
        ti -= first;
        m0 = (int64_t)(ti / a.tiles_e) * kBM;
        n0 = (int64_t)(ti % a.tiles_e) * kBN;
    }
    const int64_t nk = (a.T + kBK - 1) / kBK, k0 = part * nk / a.parts * kBK, k1 = (part + 1) * nk / a.parts * kBK;
    const int64_t ls = 3 * a.Fp, valid = (a.T < k1 ? a.T : k1) - k0;
    const Operand A = down ? rows_of(a.S + 2 * a.Fp + k0 * ls, ls, m0, a.F, valid)
                           : rows_of(a.X + k0 * kD, kD, m0, kD, valid);
    const Operand B = down ? rows_of(a.dY + k0 * kD, kD, n0, kD, valid)
                           : rows_of(a.S + k0 * ls, ls, n0, 2 * a.Fp, valid);
    f32x16 acc[kWM][kWN];
    clear(acc);
    product<true, true, kWM, kWN, kGM, kGN, kNS>(A, B, k1 - k0, sm, acc);
    const int w = threadIdx.x >> 6, wm = w / kGN, wn = w % kGN;
    float *lds = reinterpret_cast<float *>(sm + w * Rows<kWM>::BYTES);
    float *pp = a.parts > 1 ? a.part + part * (3 * a.Fp * kD) : nullptr;
#pragma unroll
    for (int nb = 0; nb < kWN; ++nb) {
        const int64_t nw = n0 + (wn * kWN + nb) * 32, mw = m0 + wm * 32 * kWM;
        Rows<kWM>::write(
            lds, [&](int mb, int e) { return acc[mb][nb][e]; },
            [&](int nn, int mm, float (&v)[8]) {
                const int64_t n = nw + nn, m = mw + mm;
                if (!down) {
                    const bool up = n >= a.Fp;
                    const int64_t f = up ? n - a.Fp : n;
                    if (f >= a.F || n >= 2 * a.Fp)
                        return;
                    if (pp)
                        store_as(pp, true, n * kD + m, v);
                    else
                        put_dw(a, up ? a.dWu : a.dWg, f * kD + m, 1.0f, v);
                } else if (m < a.F) {
                    if (pp)
                        store_as(pp + 2 * a.Fp * kD, true, n * a.Fp + m, v);
                    else
                        put_dw(a, a.dWd, n * a.F + m, a.scale, v);
                }
            });
    }
}

// The parts of k, added in order; blockIdx.y: dWg, dWu, dWd.  parts = 0 gives
// zeros (no positions).
__global__ __launch_bounds__(256) void dw_reduce_kernel(DwArgs a)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;   // element of [F][768] or [768][F]
    if (i >= a.F * kD)
        return;
    const int which = blockIdx.y;
    int64_t at = which * a.Fp * kD + i;
    if (which == 2)
        at = 2 * a.Fp * kD + i / a.F * a.Fp + i % a.F;
    float v[8] = {};
    for (int p = 0; p < a.parts; ++p) {
        float x[8];
        load_as(a.part + p * (3 * a.Fp * kD), true, at, x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += x[e];
    }
    put_dw(a, which == 0 ? a.dWg : which == 1 ? a.dWu : a.dWd, i, which == 2 ? a.scale : 1.0f, v);
}

// dY' as the products take it: bf16, dropped places 0, unscaled.
__global__ __launch_bounds__(256) void dy_kernel(const void *dY, int f32, drop::Mask m, int64_t groups, uint16_t *out)
{
    const drop::Key key = drop::key_of(m);
    for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < groups; g += (int64_t)gridDim.x * 256) {
        float v[8];
        load_as(dY, f32, g * 8, v);
        if (m.thr != 0) {
            const uint4 w = drop::bits_of(key, (uint64_t)g);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = drop::kept(w, e, m.thr) ? v[e] : 0.0f;
        }
        *reinterpret_cast<uint4 *>(out + g * 8) = pack8(v);
    }
}

// ------------------------------------------------------------------- host

struct Layout {
    int64_t Fp;
    uint64_t S, dY, part, total;
};

Layout layout(const ffn_config *c, int pass)
{
    Layout L{};
    L.Fp = rup(c->hidden, kBK);
    uint64_t o = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t at = o;
        o += (bytes + kAlign - 1) / kAlign * kAlign;
        return at;
    };
    L.S = take(2ull * c->max_tokens * L.Fp * (pass == FFN_PASS_BWD ? 3 : 1));
    if (pass == FFN_PASS_BWD) {
        L.dY = take(2ull * c->max_tokens * kD);
        L.part = take(4ull * kMaxParts * 3 * L.Fp * kD);
    }
    L.total = o;
    return L;
}

int check_cfg(const ffn_config *c)
{
    if (!c)
        return FFN_ENULL;
    if (c->dim != kD || c->hidden < 8 || c->hidden > 65536 || c->hidden % 8 != 0 || c->act < FFN_ACT_SILU ||
        c->act > FFN_ACT_RELU2 || (c->y_dtype != FFN_DTYPE_F32 && c->y_dtype != FFN_DTYPE_BF16) ||
        (c->dw_dtype != FFN_DTYPE_F32 && c->dw_dtype != FFN_DTYPE_BF16) || (c->options & ~FFN_OPT_ACCUM) != 0 ||
        c->max_tokens < 1 || c->max_tokens > (1 << 24))
        return FFN_ECONFIG;
    return FFN_OK;
}

struct Span {
    const void *p;
    uint64_t n;
};

bool meet(const Span &a, const Span &b)
{
    return a.p && b.p && (uintptr_t)a.p < (uintptr_t)b.p + b.n && (uintptr_t)b.p < (uintptr_t)a.p + a.n;
}

int done() { return hipGetLastError() == hipSuccess ? FFN_OK : FFN_EHIP; }

uint32_t blocks(int64_t n, int64_t b) { return (uint32_t)((n + b - 1) / b); }

drop::Mask no_drop()
{
    drop::Mask m{};
    m.scale = 1.0f;
    return m;
}

// Share of the resident slots busy over all rounds of nb blocks.
double round_fill(uint32_t nb, uint32_t slots)
{
    const uint32_t rounds = (nb + slots - 1) / slots;
    return rounds ? (double)nb / ((double)rounds * slots) : 1.0;
}

}   // namespace

extern "C" {

int ffn_abi_version(void) { return FFN_ABI_VERSION; }

const char *ffn_status_string(int status)
{
    switch (status) {
    case FFN_OK: return "ok";
    case FFN_ENULL: return "a required pointer is NULL";
    case FFN_EALIGN: return "a pointer is misaligned";
    case FFN_ECONFIG: return "invalid config";
    case FFN_ESIZE: return "size out of range";
    case FFN_EARG: return "argument out of range";
    case FFN_EHIP: return "HIP runtime error";
    default: return "unknown status";
    }
}

int ffn_config_check(const ffn_config *cfg) { return check_cfg(cfg) ? FFN_ECONFIG : FFN_OK; }

int ffn_workspace_bytes(const ffn_config *cfg, int pass, uint64_t *bytes)
{
    const int rc = check_cfg(cfg);
    if (rc)
        return rc;
    if (!bytes)
        return FFN_ENULL;
    if (pass != FFN_PASS_FWD && pass != FFN_PASS_BWD)
        return FFN_EARG;
    *bytes = layout(cfg, pass).total;
    return FFN_OK;
}

// The checks that both passes share; `outs` must not meet `ins`, the
// workspace or each other (but res, outs[0] of the forward: whole).
static int check_call(const ffn_config *cfg, int pass, void *ws, uint64_t ws_bytes, int64_t T, const drop_spec *drop,
                      const Span *ins, int n_in, const Span *outs, int n_out, const void *res)
{
    int rc = check_cfg(cfg);
    if (rc)
        return rc;
    if (T < 0 || T > cfg->max_tokens)
        return FFN_ESIZE;
    if (drop && (rc = drop::check_spec(drop)))
        return rc;
    if (!ws)
        return FFN_ENULL;
    for (int i = 0; i < n_in; ++i)
        if (!ins[i].p && ins[i].n)
            return FFN_ENULL;
    for (int i = 0; i < n_out; ++i)
        if (!outs[i].p && outs[i].n)
            return FFN_ENULL;
    if ((uintptr_t)ws % kAlign || (uintptr_t)res % 16)
        return FFN_EALIGN;
    for (int i = 0; i < n_in; ++i)
        if ((uintptr_t)ins[i].p % 16)
            return FFN_EALIGN;
    for (int i = 0; i < n_out; ++i)
        if ((uintptr_t)outs[i].p % 16)
            return FFN_EALIGN;
    if (ws_bytes < layout(cfg, pass).total)
        return FFN_ESIZE;
    const Span work{ws, ws_bytes};
    const Span r{res, outs[0].n};
    for (int i = 0; i < n_out; ++i) {
        for (int k = 0; k < n_in; ++k)
            if (meet(outs[i], ins[k]))
                return FFN_EARG;
        for (int k = 0; k < i; ++k)
            if (meet(outs[i], outs[k]))
                return FFN_EARG;
        if (meet(outs[i], work))
            return FFN_EARG;
    }
    for (int k = 0; k < n_in; ++k)
        if (meet(ins[k], work))
            return FFN_EARG;
    if (meet(r, work) || (res && res != outs[0].p && meet(r, outs[0])))
        return FFN_EARG;
    return FFN_OK;
}

int ffn_fwd(const ffn_config *cfg, void *ws, uint64_t ws_bytes, const void *X, const void *Wg, const void *Wu,
            const void *Wd, const void *res, const drop_spec *drop, int64_t T, void *Y, void *stream)
{
    if (!cfg)
        return FFN_ENULL;
    const uint64_t w = 2ull * kD * (uint64_t)(cfg->hidden > 0 ? cfg->hidden : 0), t = T > 0 ? T : 0;
    const Span ins[] = {{X, 2 * t * kD}, {Wg, w}, {Wu, w}, {Wd, w}};
    const Span outs[] = {{Y, (cfg->y_dtype == FFN_DTYPE_F32 ? 4 : 2) * t * kD}};
    const int rc = check_call(cfg, FFN_PASS_FWD, ws, ws_bytes, T, drop, ins, 4, outs, 1, res);
    if (rc || T == 0)
        return rc;
    const Layout L = layout(cfg, FFN_PASS_FWD);
    Args a{};
    a.X = (const uint16_t *)X;
    a.Wg = (const uint16_t *)Wg;
    a.Wu = (const uint16_t *)Wu;
    a.Wd = (const uint16_t *)Wd;
    a.S = (uint16_t *)((uint8_t *)ws + L.S);
    a.T = T;
    a.F = cfg->hidden;
    a.Fp = L.Fp;
    a.mask = drop ? drop::mask_of(*drop) : no_drop();
    a.res = res;
    a.out = Y;
    a.out_f32 = cfg->y_dtype == FFN_DTYPE_F32;
    hipStream_t s = (hipStream_t)stream;
    a.tiles_t = blocks(T, kBN);
    a.tiles_o = blocks(a.F, kBM / 2);
    auto up = cfg->act == FFN_ACT_SILU ? up_kernel<FFN_ACT_SILU>
              : cfg->act == FFN_ACT_GELU ? up_kernel<FFN_ACT_GELU> : up_kernel<FFN_ACT_RELU2>;
    up<<<grid_blocks(a.tiles_t * a.tiles_o), kThreads, 0, s>>>(a);
    a.tiles_o = kD / kBM;
    rows_kernel<false><<<grid_blocks(a.tiles_t * a.tiles_o), kThreads, 0, s>>>(a);
    return done();
}

int ffn_bwd(const ffn_config *cfg, void *ws, uint64_t ws_bytes, const void *X, const void *Wg, const void *Wu,
            const void *Wd, const void *dY, const drop_spec *drop, int64_t T, void *dX, void *dWg, void *dWu,
            void *dWd, void *stream)
{
    if (!cfg)
        return FFN_ENULL;
    const uint64_t n = (uint64_t)kD * (uint64_t)(cfg->hidden > 0 ? cfg->hidden : 0), t = T > 0 ? T : 0;
    const uint64_t ye = cfg->y_dtype == FFN_DTYPE_F32 ? 4 : 2, we = cfg->dw_dtype == FFN_DTYPE_F32 ? 4 : 2;
    const Span ins[] = {{X, 2 * t * kD}, {Wg, 2 * n}, {Wu, 2 * n}, {Wd, 2 * n}, {dY, ye * t * kD}};
    const Span outs[] = {{dX, ye * t * kD}, {dWg, we * n}, {dWu, we * n}, {dWd, we * n}};
    const int rc = check_call(cfg, FFN_PASS_BWD, ws, ws_bytes, T, drop, ins, 5, outs, 4, nullptr);
    if (rc)
        return rc;
    const Layout L = layout(cfg, FFN_PASS_BWD);
    hipStream_t s = (hipStream_t)stream;
    DwArgs d{};
    d.T = T;
    d.F = cfg->hidden;
    d.Fp = L.Fp;
    d.dWg = dWg;
    d.dWu = dWu;
    d.dWd = dWd;
    d.dw_f32 = cfg->dw_dtype == FFN_DTYPE_F32;
    d.accum = cfg->options & FFN_OPT_ACCUM;
    const dim3 rgrid(blocks(d.F * kD, 8 * 256), 3);
    if (T == 0) {
        if (d.accum)
            return FFN_OK;
        dw_reduce_kernel<<<rgrid, 256, 0, s>>>(d);   // no parts: zeros
        return done();
    }
    Args a{};
    a.X = (const uint16_t *)X;
    a.Wg = (const uint16_t *)Wg;
    a.Wu = (const uint16_t *)Wu;
    a.Wd = (const uint16_t *)Wd;
    a.dY = (const uint16_t *)dY;
    a.S = (uint16_t *)((uint8_t *)ws + L.S);
    a.T = T;
    a.F = cfg->hidden;
    a.Fp = L.Fp;
    a.mask = drop ? drop::mask_of(*drop) : no_drop();
    a.out = dX;
    a.out_f32 = cfg->y_dtype == FFN_DTYPE_F32;
    if (a.out_f32 || a.mask.thr != 0) {
        uint16_t *m = (uint16_t *)((uint8_t *)ws + L.dY);
        const int64_t groups = T * (kD / 8);
        dy_kernel<<<blocks(groups, 256), 256, 0, s>>>(dY, a.out_f32, a.mask, groups, m);
        a.dY = m;
    }
    a.tiles_t = blocks(T, kBN);
    a.tiles_o = blocks(a.F, kBM / 2);
    auto grad = cfg->act == FFN_ACT_SILU ? grad_kernel<FFN_ACT_SILU>
                : cfg->act == FFN_ACT_GELU ? grad_kernel<FFN_ACT_GELU> : grad_kernel<FFN_ACT_RELU2>;
    grad<<<grid_blocks(a.tiles_t * a.tiles_o), kThreads, 0, s>>>(a);
    a.tiles_o = kD / kBM;
    rows_kernel<true><<<grid_blocks(a.tiles_t * a.tiles_o), kThreads, 0, s>>>(a);

    d.X = a.X;
    d.dY = a.dY;
    d.S = a.S;
    d.scale = a.mask.scale;
    d.tiles_f2 = blocks(2 * d.Fp, kBN);
    d.tiles_d = kD / kBM;
    d.tiles_e = kD / kBN;
    d.tiles_h = blocks(d.F, kBM);
    const uint32_t tiles = d.tiles_f2 * d.tiles_d + d.tiles_e * d.tiles_h;
    // parts of k by the fill of the rounds of resident blocks (two per CU);
    // parts cost their reduction, about 3 %
    int parts = 1;
    double best = 0.0;
    const int64_t nk = blocks(T, kBK);
    for (int p = 1; p <= kMaxParts && p <= nk; ++p) {
        const double score = round_fill(tiles * p, 2 * kCUs) * (p > 1 ? 0.97 : 1.0);
        if (score > best + 1e-9) {
            best = score;
            parts = p;
        }
    }
    d.parts = parts;
    d.part = (float *)((uint8_t *)ws + L.part);
    dw_kernel<<<grid_blocks(tiles * (uint32_t)parts), kThreads, 0, s>>>(d);
    if (parts > 1)
        dw_reduce_kernel<<<rgrid, 256, 0, s>>>(d);
    return done();
}

}   // extern "C"
