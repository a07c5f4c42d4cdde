// Gated feed-forward block on gfx950, forward and backward (the formulas and
// the rounding points are in include/ffn.h).
//
//   up_kernel     H = a(X Wg^T) * (X Wu^T)                  -> workspace, bf16
//   rows_kernel   Y = (res +) drop(H Wd^T); dX = dG Wg + dU Wu (one contraction over 2 F)
//   grad_kernel   G, U again, dH = dY' Wd -> dG, dU, H       -> workspace, bf16
//   hidden8_kernel  up_kernel's or grad_kernel's results on 256 x 256 tiles, for many positions
//   dw_kernel     dWg, dWu, dWd in one launch, k = T, in parts where the tiles alone
//                 do not fill the chip; dw_reduce_kernel adds the parts in order
//   tail_kernel   dX and dWg, dWu, dWd in one launch, for few positions
//   up_few_kernel, down_few_kernel  the forward of up to 64 positions
//   dy_kernel     dY' where dY is fp32 or was dropped: a masked copy in bf16
//
// Every product is a block tile of mfma_tile.hpp.  Weights are read as they
// lie: where k runs over a weight's rows (dH, dX) or over positions (the weights'
// gradients) the operand is k-major and comes through the LDS transpose read,
// so nothing is transposed in memory.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/ffn.h"
#include "ffn_plan.hpp"
#include "mfma_tile.hpp"
#include "ngram_dev.hpp"
#include "philox.hpp"

namespace {

using namespace tile;
using namespace ffn_plan;

constexpr uint64_t kAlign = 256;

// ------------------------------------------------------------- block order

// The hardware hands consecutive workgroups to the 8 XCDs in turn.  Each XCD
// gets a contiguous range of tiles, walked in groups of 8 tiles of positions
// (all weight tiles of a group before the next group), so the blocks that are
// resident on an XCD share their operands in its L2.  49,152 x 2048, groups of 1 /
// 4 / 8 / 16: H 293 / 257 / 257 / 259 us, gradients of the hidden units 543 / 500 /
// 496 / 542, Y 151 / 149 / 141 / 144, dX 302 / 302 / 300 / 315.
constexpr uint32_t kGroup = 8;

// rows: tiles of positions, cols: tiles of the other side; block: the block's
// number, blockIdx.x or, where a block takes several tiles, that plus turns of the grid
__device__ inline bool tile_of(uint32_t block, uint32_t rows, uint32_t cols, uint32_t &rt, uint32_t &ct)
{
    const uint32_t total = rows * cols, per = (total + kXcds - 1) / kXcds;
    const uint32_t t = (block % kXcds) * per + block / kXcds;
    if (block / kXcds >= per || t >= total)
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

// The same for values that leave as bf16, in 4 KB of LDS per wavefront: rows of
// 64 bf16, 8 chunks of 16 bytes, chunk c of row n at c ^ (n & 7).  out(n, m, w)
// takes 8 consecutive m of one n, packed.
struct RowsBf16 {
    static constexpr uint32_t BYTES = 4096;

    template <typename V, typename O>
    static __device__ __forceinline__ void write(uint8_t *lds, V val, O out)
    {
        const int lane = fresh_tid() & 63, n = lane & 31;
        uint8_t *p = lds + n * 128 + 8 * (lane >> 5);
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint2 w;
                w.x = ngram::bf16_pack_rne(val(mb, 4 * q), val(mb, 4 * q + 1));
                w.y = ngram::bf16_pack_rne(val(mb, 4 * q + 2), val(mb, 4 * q + 3));
                *(uint2 *)(p + 16 * ((4 * mb + q) ^ (n & 7))) = w;
                __builtin_amdgcn_sched_barrier(0);   // few values in flight: the accumulators leave few registers
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + lane / 8, c = lane % 8;
            out(r, 8 * c, *(const uint4 *)(lds + r * 128 + 16 * (c ^ (r & 7))));
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

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8]);

// What rounding v to bf16 (r) left, itself in bf16: together 16 bits of it.
__device__ __forceinline__ float left_over(float v, float r) { return isinf(r) ? 0.0f : v - r; }

// The sum of products of rounded values and of what the rounding left (sums of
// their own): an infinity among the other operands times a left-over of 0 or of
// the other sign must not undo the infinity that it gave with the value itself.
__device__ __forceinline__ float with_left(float sum, float left) { return isfinite(sum) ? sum + left : sum; }

template <int WM, int WN>
__device__ __forceinline__ void add_left(f32x16 (&sum)[WM][WN], const f32x16 (&left)[WM][WN])
{
#pragma unroll
    for (int mb = 0; mb < WM; ++mb)
#pragma unroll
        for (int nb = 0; nb < WN; ++nb)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                sum[mb][nb][e] = with_left(sum[mb][nb][e], left[mb][nb][e]);
}

__device__ __forceinline__ uint4 pack8_left(const float (&v)[8], const uint4 &rounded)
{
    float r[8];
    unpack8(rounded, r);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        r[e] = left_over(v[e], r[e]);
    return pack8(r);
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

// Block tiles of BM x BN: GM x GN wavefronts of WM x WN matrix-core tiles of 32 x 32.
template <int WM_, int WN_, int GM_, int GN_>
struct Shape {
    static constexpr int WM = WM_, WN = WN_, GM = GM_, GN = GN_, NW = GM * GN, THREADS = 64 * NW;
    static constexpr int BM = 32 * WM * GM, BN = 32 * WN * GN;

    template <bool AK, bool BK, int M>
    static constexpr uint32_t smem()
    {
        return Tile<AK, BK, M, WN, GM, GN>::SMEM;
    }

    template <bool AK, bool BK, int M>
    static __device__ __forceinline__ void run(const Operand &A, const Operand &B, int64_t k0, int64_t K,
                                               uint8_t *sm, f32x16 (&acc)[M][WN])
    {
        product<AK, BK, M, WN, GM, GN>(A, B, (int32_t)k0, (int32_t)K, sm, acc);
    }
};
using Half = Shape<2, 1, 2, 2>;     // 128 x 64, 4 wavefronts, three blocks per CU
using Small = Shape<2, 2, 2, 2>;    // 128 x 128, 4 wavefronts, two blocks per CU
using Mid = Shape<2, 3, 2, 2>;      // 128 x 192, 4 wavefronts, two blocks per CU (81,920 bytes of LDS each)
using Square = Shape<4, 2, 2, 4>;   // 256 x 256, 8 wavefronts

template <class S>
constexpr bool is(Size t) { return S::BM == t.bm && S::BN == t.bn; }
static_assert(is<Half>(kHalf) && is<Small>(kSmall) && is<Mid>(kMid) && is<Square>(kSquare) && kStep == kBK, "ffn_plan.hpp's tiles");

struct Args {
    const uint16_t *X, *Wg, *Wu, *Wd, *dY;
    uint16_t *S;             // workspace: forward H [T][Fp]; backward [T][3 Fp] dG | dU | H
    int64_t T, F, Fp;
    uint32_t tiles_t, tiles_o;
    const void *res;
    void *out;
    int32_t out_f32;
    int32_t parts;           // parts of k of a [T][768] result
    float *part;             // [parts][T][768] where parts > 1
    uint16_t *lo;            // of wide_rows: what S's rounding left, laid out as S; else NULL
    drop::Mask mask;
};

__device__ __forceinline__ Operand rows_of(const uint16_t *p, int64_t ld, int64_t first, int64_t count, int64_t k)
{
    return Operand{{p, p}, ld, first, count, INT32_MAX, (int32_t)k, 0};
}

constexpr uint32_t cmax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <class S, int MB>
constexpr uint32_t smem_for(uint32_t main)
{
    return cmax(main, S::NW * Rows<MB>::BYTES);
}

// H tile of BN positions x BM / 2 hidden units: each wavefront holds its
// units' gate sums in the first half of its m-blocks and the up sums in the
// second, so both meet in one lane.
template <class S, int ACT>
__global__ __launch_bounds__(S::THREADS) void up_kernel(Args a)
{
    constexpr int HB = S::WM / 2;
    __shared__ __align__(16) uint8_t sm[smem_for<S, HB>(S::template smem<false, false, S::WM>())];
    uint32_t tt, ot;
    if (!tile_of(blockIdx.x, a.tiles_t, a.tiles_o, tt, ot))
        return;
    const int64_t n0 = (int64_t)tt * S::BN, f0 = (int64_t)ot * (S::BM / 2);
    f32x16 acc[S::WM][S::WN];
    clear(acc);
    const Operand A{{a.Wg, a.Wu}, kD, f0, a.F, INT32_MAX, kD, 32 * HB};
    S::template run<false, false, S::WM>(A, rows_of(a.X, kD, n0, a.T, kD), 0, kD, sm, acc);
    const int w = threadIdx.x >> 6, wm = w / S::GN, wn = w % S::GN;
    float *lds = reinterpret_cast<float *>(sm + w * Rows<HB>::BYTES);
    const int64_t fw = f0 + wm * 32 * HB;
#pragma unroll
    for (int nb = 0; nb < S::WN; ++nb) {
        const int64_t tw = n0 + (wn * S::WN + nb) * 32;
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

// dropout, residual, rounding: 8 results of element i on of Y or dX
template <bool DX>
__device__ __forceinline__ void put_rows(const Args &a, const drop::Key &key, int64_t i, float (&v)[8])
{
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
}

// A [T][768] result: DX false: Y = (res +) drop(H Wd^T); true: dX = [dG | dU] [Wg; Wu].
// With parts of k, each block's sums go to the workspace and rows_reduce_kernel ends the pass.
// 49,152 x 2048: Y 146 us (1.06 PFLOP/s), with dropout and a residual 176 us
// (its 75 MB more, read or not 32 rows ahead: 174 us); dX 303 us (1.02 PFLOP/s).
template <class S, bool DX>
constexpr uint32_t kRowsLds = smem_for<S, S::WM>(S::template smem<DX, false, S::WM>());

// WIDE (see wide_rows): S's left-overs as well.
template <class S, bool DX, bool WIDE>
__device__ __forceinline__ void rows_tile(const Args &a, uint32_t block, uint8_t *sm)
{
    uint32_t tt, ot;
    if (!tile_of(block, a.tiles_t, a.tiles_o * (uint32_t)a.parts, tt, ot))
        return;
    const uint32_t part = ot / a.tiles_o;
    ot -= part * a.tiles_o;
    const int64_t n0 = (int64_t)tt * S::BN, d0 = (int64_t)ot * S::BM;
    const int64_t nk = (DX ? 2 * a.Fp : a.Fp) / kBK, k0 = part * nk / a.parts * kBK, k1 = (part + 1) * nk / a.parts * kBK;
    f32x16 acc[S::WM][S::WN];
    clear(acc);
    if constexpr (DX) {
        const Operand A{{a.Wg, a.Wu}, kD, d0, kD, (int32_t)a.Fp, (int32_t)a.F, 0};
        auto from = [&](const uint16_t *src) {
            return Operand{{src, src}, 3 * a.Fp, n0, a.T, (int32_t)a.Fp, (int32_t)a.F, 0};
        };
        S::template run<true, false, S::WM>(A, from(a.S), k0, k1 - k0, sm, acc);
        if constexpr (WIDE) {
            f32x16 left[S::WM][S::WN];
            clear(left);
            S::template run<true, false, S::WM>(A, from(a.lo), k0, k1 - k0, sm, left);
            add_left(acc, left);
        }
    } else {
        S::template run<false, false, S::WM>(rows_of(a.Wd, a.F, d0, kD, a.F), rows_of(a.S, a.Fp, n0, a.T, a.F), k0,
                                             k1 - k0, sm, acc);
    }
    const int w = threadIdx.x >> 6, wm = w / S::GN, wn = w % S::GN;
    float *lds = reinterpret_cast<float *>(sm + w * Rows<S::WM>::BYTES);
    const drop::Key key = drop::key_of(a.mask);
    float *pp = a.parts > 1 ? a.part + part * (a.T * kD) : nullptr;
#pragma unroll
    for (int nb = 0; nb < S::WN; ++nb) {
        const int64_t tw = n0 + (wn * S::WN + nb) * 32, dw = d0 + wm * 32 * S::WM;
        Rows<S::WM>::write(
            lds, [&](int mb, int e) { return acc[mb][nb][e]; },
            [&](int n, int m, float (&v)[8]) {
                const int64_t t = tw + n, i = t * kD + dw + m;
                if (t >= a.T)
                    return;
                if (pp)
                    store_as(pp, true, i, v);
                else
                    put_rows<DX>(a, key, i, v);
            });
    }
}

template <class S, bool DX>
__global__ __launch_bounds__(S::THREADS) void rows_kernel(Args a)
{
    __shared__ __align__(16) uint8_t sm[kRowsLds<S, DX>];
    rows_tile<S, DX, false>(a, blockIdx.x, sm);
}

// v += the parts' 8 values at i, in order; eight parts' loads at a time are in flight.
__device__ __forceinline__ void add_parts(const float *part, int64_t size, int parts, int64_t i, float (&v)[8])
{
    for (int p = 0; p < parts; p += 8) {
        float x[8][8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (p + q < parts)
                load_as(part + (p + q) * size, true, i, x[q]);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (p + q < parts) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] += x[q][e];
            }
    }
}

// The parts of k, added in order, then the same end as rows_kernel's.
template <bool DX>
__global__ __launch_bounds__(256) void rows_reduce_kernel(Args a)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= a.T * kD)
        return;
    float v[8] = {};
    add_parts(a.part, a.T * kD, a.parts, i, v);
    put_rows<DX>(a, drop::key_of(a.mask), i, v);
}

// dG, dU and H of BN positions x BM / 2 hidden units: the gate and up sums
// again as in up_kernel, and dH of the same tile.  Half tiles take both
// products' steps together (257 x 1000: 11.0 -> 9.9 us, the whole backward 29.2 ->
// 26.1); the larger ones, bound by more than a step's chain, one after the other,
// in the LDS of one.
template <class S, int ACT>
__global__ __launch_bounds__(S::THREADS) void grad_kernel(Args a)
{
    constexpr int HB = S::WM / 2;
    constexpr bool TOGETHER = S::WN == 1;
    using P = Pair<false, true, false, S::WM, HB, S::WN, S::GM, S::GN>;
    __shared__ __align__(16) uint8_t sm[smem_for<S, HB>(
        TOGETHER ? P::SMEM : cmax(S::template smem<false, false, S::WM>(), S::template smem<true, false, HB>()))];
    uint32_t tt, ot;
    if (!tile_of(blockIdx.x, a.tiles_t, a.tiles_o, tt, ot))
        return;
    const int64_t n0 = (int64_t)tt * S::BN, f0 = (int64_t)ot * (S::BM / 2);
    f32x16 acc[S::WM][S::WN], dh[HB][S::WN];
    clear(acc);
    const Operand A{{a.Wg, a.Wu}, kD, f0, a.F, INT32_MAX, kD, 32 * HB};
    const Operand X = rows_of(a.X, kD, n0, a.T, kD), Wd = rows_of(a.Wd, a.F, f0, a.F, kD), dY = rows_of(a.dY, kD, n0, a.T, kD);
    if constexpr (TOGETHER) {
        clear(dh);
        P::run(A, X, Wd, dY, kD, sm, acc, dh);
    } else {
        S::template run<false, false, S::WM>(A, X, 0, kD, sm, acc);
        clear(dh);
        S::template run<true, false, HB>(Wd, dY, 0, kD, sm, dh);
    }
    const int w = threadIdx.x >> 6, wm = w / S::GN, wn = w % S::GN;
    float *lds = reinterpret_cast<float *>(sm + w * Rows<HB>::BYTES);
    const int64_t fw = f0 + wm * 32 * HB;
#pragma unroll
    for (int nb = 0; nb < S::WN; ++nb) {
        const int64_t tw = n0 + (wn * S::WN + nb) * 32;
        auto put = [&](int which) {
            return [&, which](int n, int m, const float (&v)[8]) {
                const int64_t t = tw + n, f = fw + m;
                if (t < a.T && f < a.F) {
                    const int64_t i = t * 3 * a.Fp + which * a.Fp + f;
                    const uint4 r = pack8(v);
                    *reinterpret_cast<uint4 *>(a.S + i) = r;
                    if (a.lo)
                        *reinterpret_cast<uint4 *>(a.lo + i) = pack8_left(v, r);
                }
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

// ------------------------------------------- many tiles on eight wavefronts
//
// up_kernel and grad_kernel on Square tiles, one block per CU that takes tiles
// in turns.  With 12 steps of k a tile, what is around the steps counts: while
// a product's last step runs, the first stage of the next product (dH's, or the
// next tile's) is loaded already, and a tile's results leave through LDS of
// their own (the two stages and 8 x 4 KB make up the CU's 160 KB) while the
// next tile begins.  One launch of a block per tile measured 277 us for H of
// 49,152 x 2048 and 580 us for the gradients (on 256 x 192 tiles; 600 with
// spills on 256 x 256); this 263 us (1.18 PFLOP/s) and 503 us (0.92 PFLOP/s),
// of which storing 604 MB is about 80 us.  Storing H between the two products
// (fewer bytes at a time) cost more registers than there are: 625 us.
constexpr int kLds = 160 * 1024;

using G8 = Square;
using LX = Loader<false, G8::BN, G8::NW>;        // rows of X and of dY'
using LW = Loader<false, G8::BM, G8::NW>;        // rows of Wg and Wu, in turns of 64
using LD = Loader<true, G8::BM / 2, G8::NW>;     // columns of Wd
using FX = Reader<false, G8::BN, G8::WN>;
using FW = Reader<false, G8::BM, G8::WM>;
using FD = Reader<true, G8::BM / 2, G8::WM / 2>;
constexpr uint32_t kStage8 = LX::BYTES + LW::BYTES;
static_assert(2 * kStage8 + G8::NW * RowsBf16::BYTES == kLds && G8::WM == 4 && LD::BYTES <= LW::BYTES, "the CU's LDS");

// A product's operands: the position side, which the two products share, and the weights'.
template <class LA, class FA, int WM>
struct View {
    LA &la;
    LX &lb;
    const FA &ra;
    const FX &rb;

    __device__ __forceinline__ void issue(lds_u8 *stage)
    {
        lb.issue(stage);
        la.issue(stage + LX::BYTES);
    }

    __device__ __forceinline__ void read(const lds_u8 *stage, int kk, bf16x8 (&x)[WM], bf16x8 (&y)[G8::WN]) const
    {
#pragma unroll
        for (int mb = 0; mb < WM; ++mb)
            x[mb] = ra.get(stage, mb, kk);
#pragma unroll
        for (int nb = 0; nb < G8::WN; ++nb)
            y[nb] = rb.get(stage, nb, kk);
    }
};

// A tile's first position and unit, moved back where it would reach past the
// last: every tile is whole, so the lanes' offsets never change and the next
// tile costs scalar work only.  (Needs T and F of at least a tile.  What two
// tiles share, both compute and write, bit for bit the same.)
struct TileAt {
    int64_t n0, f0;
    bool ok;
};

__device__ __forceinline__ TileAt next_tile(const Args &a, uint32_t block)
{
    TileAt p;
    uint32_t tt = 0, ot = 0;
    p.ok = tile_of(block, a.tiles_t, a.tiles_o, tt, ot);
    p.n0 = min((int64_t)tt * G8::BN, a.T - G8::BN);
    p.f0 = min((int64_t)ot * (G8::BM / 2), a.F - G8::BM / 2);
    return p;
}

__device__ __forceinline__ Operand gate_up(const Args &a, const TileAt &p)
{
    return Operand{{a.Wg, a.Wu}, kD, p.f0, a.F, INT32_MAX, kD, 16 * G8::WM};
}

__device__ __forceinline__ Operand positions(const Args &a, const uint16_t *src, const TileAt &p)
{
    return rows_of(src, kD, p.n0, a.T, kD);
}

// BWD false: H; true: dG, dU and H.
template <int ACT, bool BWD>
__global__ __launch_bounds__(G8::THREADS) void hidden8_kernel(Args a)
{
    __shared__ __align__(16) uint8_t sm[kLds];
    uint32_t block = blockIdx.x;
    TileAt p = next_tile(a, block);
    if (!p.ok)
        return;
    lds_u8 *s0, *s1;
    places(sm, kStage8, s0, s1);
    const int w = wave_id(), wm = w / G8::GN, wn = w % G8::GN;
    LX lx;
    LW lw;
    LD ld;
    FX fx;
    FW fw;
    FD fd;
    lx.set_lanes(positions(a, a.X, p));
    lw.set_lanes(gate_up(a, p));
    fx.init(0, wn * 32 * G8::WN);
    fw.init(LX::BYTES, wm * 32 * G8::WM);
    if constexpr (BWD) {
        ld.set_lanes(rows_of(a.Wd, a.F, p.f0, a.F, kD));
        fd.init(LX::BYTES, wm * 16 * G8::WM);
    }
    View<LW, FW, G8::WM> gu{lw, lx, fw, fx};
    View<LD, FD, G8::WM / 2> du{ld, lx, fd, fx};
    auto begin = [&](const TileAt &q, lds_u8 *stage) {
        lx.set_base(positions(a, a.X, q), 0);
        lw.set_base(gate_up(a, q), 0);
        gu.issue(stage);
    };
    begin(p, s0);
    wait_vmcnt<0>();
    barrier_nofence();
    uint8_t *lds = sm + 2 * kStage8 + w * RowsBf16::BYTES;
    while (p.ok) {
        f32x16 acc[G8::WM][G8::WN], dh[G8::WM / 2][G8::WN];
        clear(acc);
        block += gridDim.x;
        const TileAt q = next_tile(a, block);
        chain8(gu, kD / kBK, s0, s1, acc, [&](lds_u8 *stage) {
            if constexpr (BWD) {
                lx.set_base(positions(a, a.dY, p), 0);
                ld.set_base(rows_of(a.Wd, a.F, p.f0, a.F, kD), 0);
                du.issue(stage);
            } else if (q.ok) {
                begin(q, stage);
            }
        });
        if constexpr (BWD) {
            clear(dh);
            chain8(du, kD / kBK, s0, s1, dh, [&](lds_u8 *stage) {
                if (q.ok)
                    begin(q, stage);
            });
        }
        const int64_t ls = (BWD ? 3 : 1) * a.Fp;
        uint16_t *const at = a.S + (p.n0 + wn * 32 * G8::WN) * ls + p.f0 + wm * 64;
#pragma unroll
        for (int nb = 0; nb < G8::WN; ++nb) {
            auto put = [&](int64_t which) {
                return [&, which](int n, int m, const uint4 &v) {
                    *reinterpret_cast<uint4 *>(at + (32 * nb + n) * ls + which * a.Fp + m) = v;
                };
            };
            if constexpr (BWD) {
                RowsBf16::write(
                    lds,
                    [&](int mb, int e) {
                        const float g = acc[mb][nb][e], up = acc[mb + 2][nb][e], h = a.mask.scale * dh[mb][nb][e];
                        float d;
                        const float s = act<ACT, true>(g, d);
                        acc[mb][nb][e] = h * s;
                        acc[mb + 2][nb][e] = h * up * d;
                        return s * up;
                    },
                    put(2));
                RowsBf16::write(lds, [&](int mb, int e) { return acc[mb][nb][e]; }, put(1));
                RowsBf16::write(lds, [&](int mb, int e) { return acc[mb + 2][nb][e]; }, put(0));
            } else {
                RowsBf16::write(
                    lds,
                    [&](int mb, int e) {
                        float d;
                        return act<ACT, false>(acc[mb][nb][e], d) * acc[mb + 2][nb][e];
                    },
                    put(0));
            }
        }
        p = q;
    }
}

// ---------------------------------------------------------------- few rows

// Up to 64 positions: the weights' bytes bound the pass, and the latency of
// one round of loads most of it.  No LDS stages and no k loop over barriers:
// every wavefront loads its share of k straight into matrix-core fragments
// (16 weight rows x 16 positions x 32 values of k each), all loads in flight at
// once, and the wavefronts' sums meet in LDS.  F = 2048: T = 1 7.9 us (8.5 with
// two bf16 values of H) against 14.5 through the tiles, T = 16 10 against 15, T =
// 32 12.7 against 15.5.  The down product has 48 blocks whatever F, so F and T F are bounded: the two
// meet near T F = 96 Ki (16 x 6144 19 against 19 us, 24 x 4096 16 against 16,
// 32 x 4096 18 against 16) and, for one position, between F = 8192 (16.5
// against 20) and 16,384 (29 against 26).  From 33 positions on, four tiles of
// positions: 33 x 424 8.8 against 13.4, 64 x 1000 12.3 against 14.0, but 64 x 2048 17.7
// against 16.1, so T F is 64 Ki at most there.
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

constexpr int kFewWaves = 4;
constexpr int kFewDown = 8;   // wavefronts of a down block

// H of 16 hidden units, NT tiles of 16 positions; a wavefront takes a quarter of k.
template <int ACT, int NT, bool WIDE>
__global__ __launch_bounds__(64 * kFewWaves) void up_few_kernel(Args a)
{
    constexpr int STEPS = kD / (32 * kFewWaves);   // 6
    __shared__ __align__(16) f32x4 red[kFewWaves][2][NT][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15;
    const int64_t f0 = (int64_t)blockIdx.x * 16, f = f0 + r < a.F ? f0 + r : a.F - 1;
    const int k = w * (kD / kFewWaves) + 8 * (lane >> 4);
    const uint16_t *pg = a.Wg + f * kD + k, *pu = a.Wu + f * kD + k;
    bf16x8 g[STEPS], u[STEPS];
    f32x4 ag[NT] = {}, au[NT] = {};
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        g[s] = *reinterpret_cast<const bf16x8 *>(pg + 32 * s);
        u[s] = *reinterpret_cast<const bf16x8 *>(pu + 32 * s);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int64_t t = 16 * n + r < a.T ? 16 * n + r : a.T - 1;
        const uint16_t *px = a.X + t * kD + k;
        bf16x8 x[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            x[s] = *reinterpret_cast<const bf16x8 *>(px + 32 * s);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            ag[n] = mfma16(g[s], x[s], ag[n]);
            au[n] = mfma16(u[s], x[s], au[n]);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        red[w][0][n][lane] = ag[n];
        red[w][1][n][lane] = au[n];
    }
    __syncthreads();
    if (w >= NT)
        return;
    f32x4 sg = red[0][0][w][lane], su = red[0][1][w][lane];
#pragma unroll
    for (int p = 1; p < kFewWaves; ++p) {
        sg += red[p][0][w][lane];
        su += red[p][1][w][lane];
    }
    // lane: position 16 w + lane % 16, units 4 (lane / 16) .. + 3
    const int64_t t = 16 * w + r, ff = f0 + 4 * (lane >> 4);
    if (t < a.T && ff < a.F) {
        float h[4], d;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = act<ACT, false>(sg[e], d) * su[e];
        uint2 o, l;
        o.x = ngram::bf16_pack_rne(h[0], h[1]);
        o.y = ngram::bf16_pack_rne(h[2], h[3]);
        *reinterpret_cast<uint2 *>(a.S + t * a.Fp + ff) = o;
        if constexpr (WIDE) {
            l.x = ngram::bf16_pack_rne(left_over(h[0], ngram::bf16_lo(o.x)), left_over(h[1], ngram::bf16_hi(o.x)));
            l.y = ngram::bf16_pack_rne(left_over(h[2], ngram::bf16_lo(o.y)), left_over(h[3], ngram::bf16_hi(o.y)));
            *reinterpret_cast<uint2 *>(a.lo + t * a.Fp + ff) = l;
        }
    }
}

// Y of 16 outputs; a wavefront takes every eighth step of 32 values of k.
template <int NT, bool WIDE>
__global__ __launch_bounds__(64 * kFewDown) void down_few_kernel(Args a)
{
    constexpr int U = 4;   // steps in flight
    __shared__ __align__(16) f32x4 red[kFewDown][NT][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r = lane & 15;
    const int64_t d0 = (int64_t)blockIdx.x * 16;
    const uint16_t *pw = a.Wd + (d0 + r) * a.F;
    int64_t ph[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        ph[n] = (16 * n + r < a.T ? 16 * n + r : a.T - 1) * a.Fp;
    f32x4 acc[NT] = {}, left[NT] = {};
    const bf16x8 zero = {};
    for (int64_t k0 = (int64_t)w * 32 + 8 * (lane >> 4); k0 - 8 * (lane >> 4) < a.F; k0 += U * kFewDown * 32) {
        bf16x8 x[U], h[U][NT], l[U][NT];
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const int64_t k = k0 + s * (kFewDown * 32);
            const bool in = k < a.F;
            x[s] = in ? *reinterpret_cast<const bf16x8 *>(pw + k) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                h[s][n] = in ? *reinterpret_cast<const bf16x8 *>(a.S + ph[n] + k) : zero;
                if constexpr (WIDE)
                    l[s][n] = in ? *reinterpret_cast<const bf16x8 *>(a.lo + ph[n] + k) : zero;
            }
        }
#pragma unroll
        for (int s = 0; s < U; ++s)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n] = mfma16(x[s], h[s][n], acc[n]);
                if constexpr (WIDE)
                    left[n] = mfma16(x[s], l[s][n], left[n]);
            }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if constexpr (WIDE) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[n][e] = with_left(acc[n][e], left[n][e]);
        }
        red[w][n][lane] = acc[n];
    }
    __syncthreads();
    // one thread: 8 outputs of one position, the halves of two lanes of the sums
    const int n = threadIdx.x / 32, q = threadIdx.x % 32;
    const int64_t t = 16 * n + q % 16;
    if (n >= NT || t >= a.T)
        return;
    const int from = q % 16 + 32 * (q / 16);   // lanes from and from + 16
    f32x4 lo = red[0][n][from], hi = red[0][n][from + 16];
#pragma unroll
    for (int p = 1; p < kFewDown; ++p) {
        lo += red[p][n][from];
        hi += red[p][n][from + 16];
    }
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    put_rows<false>(a, drop::key_of(a.mask), t * kD + d0 + 8 * (q / 16), v);
}

struct DwArgs {
    const uint16_t *X, *dY, *S, *lo;   // lo: as in Args
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

// One tile of one part of k: rows n of the result with m contiguous.  Both
// operands are k-major, so nothing is transposed in memory.  49,152 x 2048: 440 us in
// 7 parts and 12 us to add them (1.05 PFLOP/s of products).
//   dWg | dWu: n = f of 2 Fp (B = dG | dU), m = d (A = X)
//   dWd:       n = d (B = dY'),             m = f (A = H)
template <class S>
constexpr uint32_t kDwLds = smem_for<S, S::WM>(S::template smem<true, true, S::WM>());

template <class S, bool WIDE>
__device__ __forceinline__ void dw_tile(const DwArgs &a, uint32_t block, uint8_t *sm)
{
    const uint32_t first = a.tiles_f2 * a.tiles_d, tiles = first + a.tiles_e * a.tiles_h;
    uint32_t part, ti;
    {
        // parts outermost: the blocks that run together share their rows of k
        const uint32_t total = tiles * (uint32_t)a.parts, per = (total + kXcds - 1) / kXcds;
        const uint32_t t = (block % kXcds) * per + block / kXcds;
        if (block / kXcds >= per || t >= total)
            return;
        part = t / tiles;
        ti = t % tiles;
    }
    const bool down = ti >= first;
    int64_t n0, m0;
    if (!down) {
        n0 = (int64_t)(ti / a.tiles_d) * S::BN;
        m0 = (int64_t)(ti % a.tiles_d) * S::BM;
    } else {
        ti -= first;
        m0 = (int64_t)(ti / a.tiles_e) * S::BM;
        n0 = (int64_t)(ti % a.tiles_e) * S::BN;
    }
    const int64_t nk = (a.T + kBK - 1) / kBK, k0 = part * nk / a.parts * kBK, k1 = (part + 1) * nk / a.parts * kBK;
    const int64_t ls = 3 * a.Fp, valid = (a.T < k1 ? a.T : k1) - k0;
    Operand A = down ? rows_of(a.S + 2 * a.Fp + k0 * ls, ls, m0, a.F, valid)
                     : rows_of(a.X + k0 * kD, kD, m0, kD, valid);
    Operand B = down ? rows_of(a.dY + k0 * kD, kD, n0, kD, valid)
                     : rows_of(a.S + k0 * ls, ls, n0, 2 * a.Fp, valid);
    f32x16 acc[S::WM][S::WN];
    clear(acc);
    if constexpr (WIDE) {   // one stage of positions, and the same again with the left-overs
        A.seg = B.seg = kBK;
        (down ? A : B).src[1] = a.lo + (down ? 2 * a.Fp : 0);
        f32x16 left[S::WM][S::WN];
        clear(left);
        product_1_1<true, true, S::WM, S::WN, S::GM, S::GN>(A, B, sm, acc, left);
        add_left(acc, left);
    } else {
        S::template run<true, true, S::WM>(A, B, 0, k1 - k0, sm, acc);
    }
    const int w = threadIdx.x >> 6, wm = w / S::GN, wn = w % S::GN;
    float *lds = reinterpret_cast<float *>(sm + w * Rows<S::WM>::BYTES);
    float *pp = a.parts > 1 ? a.part + part * (3 * a.Fp * kD) : nullptr;
#pragma unroll
    for (int nb = 0; nb < S::WN; ++nb) {
        const int64_t nw = n0 + (wn * S::WN + nb) * 32, mw = m0 + wm * 32 * S::WM;
        Rows<S::WM>::write(
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

template <class S>
__global__ __launch_bounds__(S::THREADS) void dw_kernel(DwArgs a)
{
    __shared__ __align__(16) uint8_t sm[kDwLds<S>];
    dw_tile<S, false>(a, blockIdx.x, sm);
}

// dX and the weights' gradients in one launch: neither needs the other, and
// alone neither fills the chip while a backward is short (T = 257, F = 1000: 13.3
// us against 19.4, T = 4096, F = 2048: 71 against 97; from about 6,000 x 2048 on
// the larger tiles of dw_kernel win, 8,192 x 2304: 162 against 157).
template <class S, bool WIDE>
__global__ __launch_bounds__(S::THREADS) void tail_kernel(Args a, DwArgs d, uint32_t row_blocks)
{
    static_assert(S::THREADS == Small::THREADS, "one block size");
    __shared__ __align__(16) uint8_t sm[cmax(kRowsLds<S, true>, kDwLds<Small>)];
    if (blockIdx.x < row_blocks)
        rows_tile<S, true, WIDE>(a, blockIdx.x, sm);
    else
        dw_tile<Small, WIDE>(d, blockIdx.x - row_blocks, sm);
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
    add_parts(a.part, 3 * a.Fp * kD, a.parts, at, v);
    put_dw(a, which == 0 ? a.dWg : which == 1 ? a.dWu : a.dWd, i, which == 2 ? a.scale : 1.0f, v);
}

// dY' as the products take it: bf16, dropped places 0, unscaled (49,152 rows of
// bf16: 24 us, one pass over 151 MB; masking in the products' loads would need them
// to pass through registers).
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
    }
    uint64_t part = row_part_bytes(c->max_tokens);
    if (pass == FFN_PASS_BWD)
        part = std::max({part, dw_part_bytes(c->max_tokens, L.Fp), wide_bytes(c->max_tokens, c->hidden, L.Fp)});
    L.part = take(part);
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

template <class S>
void launch_up(Args a, int act, hipStream_t s)
{
    a.tiles_t = blocks(a.T, S::BN);
    a.tiles_o = blocks(a.F, S::BM / 2);
    auto k = act == FFN_ACT_SILU ? up_kernel<S, FFN_ACT_SILU>
             : act == FFN_ACT_GELU ? up_kernel<S, FFN_ACT_GELU> : up_kernel<S, FFN_ACT_RELU2>;
    k<<<grid_blocks(a.tiles_t * a.tiles_o), S::THREADS, 0, s>>>(a);
}

// T of at least G8::BN, F of at least G8::BM / 2
template <bool BWD>
void launch_hidden8(Args a, int act, hipStream_t s)
{
    a.tiles_t = blocks(a.T, G8::BN);
    a.tiles_o = blocks(a.F, G8::BM / 2);
    const uint32_t n = grid_blocks(a.tiles_t * a.tiles_o);
    auto k = act == FFN_ACT_SILU ? hidden8_kernel<FFN_ACT_SILU, BWD>
             : act == FFN_ACT_GELU ? hidden8_kernel<FFN_ACT_GELU, BWD> : hidden8_kernel<FFN_ACT_RELU2, BWD>;
    k<<<n < kCUs ? n : kCUs, G8::THREADS, 0, s>>>(a);
}

// a with the tiles and parts of a [T][768] result; its blocks
template <class S>
uint32_t set_rows(Args &a, int parts)
{
    a.tiles_t = blocks(a.T, S::BN);
    a.tiles_o = kD / S::BM;
    a.parts = parts;
    return grid_blocks(a.tiles_t * a.tiles_o * (uint32_t)parts);
}

template <bool DX>
void reduce_rows(const Args &a, hipStream_t s)
{
    if (a.parts > 1)
        rows_reduce_kernel<DX><<<blocks(a.T * kD, 8 * 256), 256, 0, s>>>(a);
}

template <class S, bool DX>
void launch_rows(Args a, int parts, hipStream_t s)
{
    const uint32_t n = set_rows<S>(a, parts);
    rows_kernel<S, DX><<<n, S::THREADS, 0, s>>>(a);
    reduce_rows<DX>(a, s);
}

template <int NT, bool WIDE>
void launch_few(const Args &a, int act, hipStream_t s)
{
    auto k = act == FFN_ACT_SILU ? up_few_kernel<FFN_ACT_SILU, NT, WIDE>
             : act == FFN_ACT_GELU ? up_few_kernel<FFN_ACT_GELU, NT, WIDE> : up_few_kernel<FFN_ACT_RELU2, NT, WIDE>;
    k<<<blocks(a.F, 16), 64 * kFewWaves, 0, s>>>(a);
    down_few_kernel<NT, WIDE><<<kD / 16, 64 * kFewDown, 0, s>>>(a);
}

template <class S>
void launch_grad(Args a, int act, hipStream_t s)
{
    a.tiles_t = blocks(a.T, S::BN);
    a.tiles_o = blocks(a.F, S::BM / 2);
    auto k = act == FFN_ACT_SILU ? grad_kernel<S, FFN_ACT_SILU>
             : act == FFN_ACT_GELU ? grad_kernel<S, FFN_ACT_GELU> : grad_kernel<S, FFN_ACT_RELU2>;
    k<<<grid_blocks(a.tiles_t * a.tiles_o), S::THREADS, 0, s>>>(a);
}

// The same for the weights' gradients.
template <class S>
uint32_t set_dw(DwArgs &d, int parts)
{
    d.tiles_f2 = blocks(2 * d.Fp, S::BN);
    d.tiles_d = kD / S::BM;
    d.tiles_e = kD / S::BN;
    d.tiles_h = blocks(d.F, S::BM);
    d.parts = parts;
    return grid_blocks((d.tiles_f2 * d.tiles_d + d.tiles_e * d.tiles_h) * (uint32_t)parts);
}

void reduce_dw(const DwArgs &d, hipStream_t s)
{
    if (d.parts > 1)
        dw_reduce_kernel<<<dim3(blocks(d.F * kD, 8 * 256), 3), 256, 0, s>>>(d);
}

template <class S>
void launch_dw(DwArgs d, int parts, hipStream_t s)
{
    const uint32_t n = set_dw<S>(d, parts);
    dw_kernel<S><<<n, S::THREADS, 0, s>>>(d);
    reduce_dw(d, s);
}

// (with parts of the weights' gradients both sums would lie in one place)
template <class S, bool WIDE>
void launch_tail(Args a, int parts, DwArgs d, hipStream_t s)
{
    const uint32_t n = set_rows<S>(a, parts), m = set_dw<Small>(d, 1);
    tail_kernel<S, WIDE><<<n + m, S::THREADS, 0, s>>>(a, d, n);
    reduce_rows<true>(a, s);
}

void up(const Args &a, const Choice &c, int act, hipStream_t s)
{
    (c.shape == 0 ? launch_up<Half> : c.shape == 1 ? launch_up<Small> : launch_hidden8<false>)(a, act, s);
}

void grad(const Args &a, const Choice &c, int act, hipStream_t s)
{
    (c.shape == 0 ? launch_grad<Half> : c.shape == 1 ? launch_grad<Small> : launch_hidden8<true>)(a, act, s);
}

template <bool DX>
void rows(const Args &a, const Choice &c, hipStream_t s)
{
    (c.shape == 0 ? launch_rows<Half, DX> : c.shape == 1 ? launch_rows<Small, DX> : launch_rows<Mid, DX>)(a, c.parts, s);
}

// dX and the weights' gradients
void tail(const Args &a, const DwArgs &d, const Bwd &p, hipStream_t s)
{
    if (p.merged) {
        // (at most a tile of positions where wide: Small tiles are then as many, and longer)
        (p.wide ? launch_tail<Half, true> : p.rows.shape == 0 ? launch_tail<Half, false> : launch_tail<Small, false>)(
            a, p.rows.parts, d, s);
        return;
    }
    rows<true>(a, p.rows, s);
    (p.dw.shape == 0 ? launch_dw<Small> : launch_dw<Square>)(d, p.dw.parts, s);
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
    const Span rng{drop ? drop->rng : nullptr, sizeof(drop_rng)};
    if (meet(rng, work))
        return FFN_EARG;
    for (int i = 0; i < n_out; ++i)
        if (meet(rng, outs[i]))
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
    a.part = (float *)((uint8_t *)ws + L.part);
    a.T = T;
    a.F = cfg->hidden;
    a.Fp = L.Fp;
    a.mask = drop ? drop::mask_of(*drop) : no_drop();
    a.res = res;
    a.out = Y;
    a.out_f32 = cfg->y_dtype == FFN_DTYPE_F32;
    hipStream_t s = (hipStream_t)stream;
    const Fwd p = plan_fwd(T, a.F);
    if (p.wide)
        a.lo = (uint16_t *)a.part;   // 2 T Fp <= 16,384 T bytes; part holds 49,152 T
    if (!p.few) {
        up(a, p.hidden, cfg->act, s);
        rows<false>(a, p.rows, s);
    } else if (a.lo) {
        (T > 32 ? launch_few<4, true> : T > 16 ? launch_few<2, true> : launch_few<1, true>)(a, cfg->act, s);
    } else {
        (T > 32 ? launch_few<4, false> : T > 16 ? launch_few<2, false> : launch_few<1, false>)(a, cfg->act, s);
    }
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
    a.part = (float *)((uint8_t *)ws + L.part);
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
    d.X = a.X;
    d.dY = a.dY;
    d.S = a.S;
    d.scale = a.mask.scale;
    d.part = (float *)((uint8_t *)ws + L.part);
    const Bwd p = plan_bwd(T, a.F);
    if (p.wide) {
        a.lo = (uint16_t *)(a.part + kMaxRowParts * T * kD);   // behind the parts of dX: wide_bytes
        d.lo = a.lo;
    }
    grad(a, p.hidden, cfg->act, s);
    tail(a, d, p, s);
    return done();
}

}   // extern "C"
