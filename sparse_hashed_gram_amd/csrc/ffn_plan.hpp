// Which kernels a call of the feed-forward block takes: rules on sizes alone,
// host code with no HIP in it, so that a test compiles it and sees which cases
// reach which kernel.  ffn.hip launches what plan_fwd and plan_bwd say.
#pragma once

#include <stdint.h>

namespace ffn_plan {

constexpr int kD = 768;
constexpr int kStep = 64;        // k values of a stage
constexpr int kMaxParts = 8;     // parts of k of the weights' gradients
constexpr uint32_t kCUs = 256, kXcds = 8;

struct Size {
    int bm, bn;   // a block tile
};
constexpr Size kHalf{128, 64}, kSmall{128, 128}, kMid{128, 192}, kSquare{256, 256};

inline int64_t rup(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline uint32_t grid_blocks(uint32_t tiles) { return kXcds * ((tiles + kXcds - 1) / kXcds); }

// ---- few positions (up_few_kernel, down_few_kernel; their times stand there)

inline bool few_rows(int64_t T, int64_t F)
{
    return T <= 64 && F <= 8192 && T * F <= (T <= 32 ? 96 : 64) * 1024;
}

constexpr int kFewT = 64;   // most positions of wide_rows: one stage of the weights' gradients

// Calls of few values keep 16 bits of H, dG and dU, as two bf16 values (the
// rounded one and what that left).  One bf16 value makes a result's error sqrt(2)
// times that of the result's own rounding, on average over calls of any size
// (an operand's rounding weighs as much as the result's, however many products
// are summed).  What T F, the number of values rounded, decides is how far the
// error of one call's results (their norm) strays from that: up to 1.8 times the
// own rounding's at T F = 128 - 424, 1.66 at 2,048, 1.56 at 4,096 - 8,192, 1.5 at
// 16,384, 1.42 at 257,000 (24 - 120 calls of each size).  So this is a bound of about
// 1.5 on a call's error, not a promise about one element.  Every F of 128 or more
// meets it by T F alone; narrower layers of more than 64 positions do not get it.
// In a captured graph: forward of 1 x 2048 7.9 -> 8.5 us, 32 x 256 7.7 -> 8.4, 64 x 128
// 9.2 -> 10.1; backward of 1 x 424 19.8 -> 20.9, 1 x 2048 22.0 -> 23.8, 32 x 256 20.4 ->
// 26.0, 64 x 128 18.8 -> 21.9.  For larger calls the products would double.
constexpr int64_t kFewValues = 8192;

inline bool wide_rows(int64_t T, int64_t F)
{
    return T <= kFewT && T * F <= kFewValues;
}

// ---- which tile, and how many parts of k
//
// Time of a launch in us, besides 2.5 that all have: turns(blocks) x (step x
// steps of 64 k + rest), and for parts their sums' way through memory and the
// launch that adds them.  turns(): a block alone on its CU is bound by latency,
// a second one fits beside it for a third more, and from about five on the
// CU's load path (see mfma_tile.hpp) makes them add up.  The constants are
// measured (T = 30 ... 49,152, F = 128 ... 8000, warm, one process; over 93 pairs
// of T and F the chosen launches take 1.00 (H and its gradients), 1.01 (Y) and 1.02
// times (dX and the weights' gradients) the best ones' time):
//   a step of rows: Half 0.45 - 0.5, Small 0.62, Mid 0.80 us; of dW: Small 0.47, Square 1.47 us;
//   up (12 steps and epilogue): Half 4.2, Small 7.75, hidden8 22 us a block;
//   grad (24 steps and epilogue): Half 7.6 (8.6 past two a CU), Small 14.5, hidden8 40 us a block.
// E.g. T = 1024, F = 2048: up 10.5 / 10.3 / 24 us (Half / Small / hidden8), T =
// 49,152: Small 371, hidden8 263 us; grad at T = 100: 11.4 / 15.3 us (Half /
// Small), T = 49,152: Small 620, hidden8 503 us; down at T = 49,152: Small 167,
// Mid 146 us; dW at T = 1024: Small 19.5, Square 28 us, at T = 49,152: Small
// 532 (7 parts), Square 451 us (7 parts) against 1,132 (1 part).
constexpr double kBytesPerUs = 4.5e6;
constexpr int kMaxRowParts = 16;   // of a [T][768] result

inline double rounds(int64_t blocks) { return (double)((blocks + kCUs - 1) / kCUs); }

inline double turns(int64_t blocks)
{
    static const double few[] = {1.0, 1.0, 1.3, 2.0, 2.9};
    const int64_t r = (blocks + kCUs - 1) / kCUs;
    return r < 5 ? few[r] : 0.93 * (double)r;
}

// the parts of a [T][768] result, written, read and added in a launch of their own
inline double reduce_us(int64_t T, int p) { return 3.0 + 0.1 * p + p * T * (2.0 * 4 * kD) / kBytesPerUs; }

struct Choice {
    int shape, parts;   // index into the candidates
    double us;
};

inline void consider(Choice &best, int shape, int parts, double us)
{
    if (best.parts == 0 || us < best.us)
        best = Choice{shape, parts, us};
}

// Tiles of positions x units; 0 Half, 1 Small, 2 hidden8_kernel's.  A second
// Half block on a CU costs less than the first, a chip full of Small ones more
// than a few (gradients, T = 1800, F = 1000: Half, 464 blocks, 19 us, Small, 240, 22; T =
// 4000, F = 264: 315 blocks 15, 160 blocks 20).
inline Choice choose_hidden(int64_t T, int64_t F, bool bwd)
{
    Choice c{};
    auto tiles = [&](Size s) { return ceil_div(T, s.bn) * ceil_div(F, s.bm / 2); };
    const int64_t half = tiles(kHalf), small = tiles(kSmall);
    const double h = (double)half / kCUs, m = (double)small / kCUs;
    consider(c, 0, 1, h <= 2.0 ? (bwd ? 7.6 : 4.2) * (h > 1.0 ? 1.2 + 0.4 * h : 1.0) : (bwd ? 8.6 : 4.2) * rounds(half));
    consider(c, 1, 1, (bwd ? 14.5 : 7.75) * (m <= 1.0 ? 1.0 + 0.3 * m : rounds(small)));
    if (T >= kSquare.bn && F >= kSquare.bm / 2)
        consider(c, 2, 1, (bwd ? 40.0 : 22.0) * rounds(tiles(kSquare)));
    return c;
}

// Tiles of the three weights' gradients.
inline int64_t dw_tiles(int64_t F, int64_t Fp, Size s)
{
    return ceil_div(2 * Fp, s.bn) * (kD / s.bm) + (kD / s.bn) * ceil_div(F, s.bm);
}

// A step of Small tiles of the weights' gradients.  Where the operands exceed
// the L2s, a block alone on its CU waits for them (T = 15,000, F = 400: 198 blocks
// 0.74 us a step, 462 blocks 0.5).
inline double dw_step(int64_t T, int64_t Fp, int64_t blocks)
{
    return T * (2 * kD + 6 * Fp) <= (32 << 20) ? 0.47 : blocks <= kCUs ? 0.74 : 0.57;
}

// A [T][768] result over `steps` stages of k; 0 Half, 1 Small, 2 Mid.  A part
// has at least two stages, and parts only where a round of blocks holds them.
// step: 1.4 where the weights' rows are not whole 128-byte lines, else 1; many
// blocks feel it (Y at T = 3001: F = 2048 23 us, F = 2056 29 us), but not two Small
// ones on a CU (T = 4000, F = 4104: 1 part 55 us, 2 parts 45).
inline Choice choose_rows(int64_t T, int64_t steps, double step)
{
    Choice c{};
    for (int p = 1; p <= kMaxRowParts && (p == 1 || 2 * p <= steps); ++p) {
        const double add = p > 1 ? reduce_us(T, p) : 0.0;
        const double n = (double)ceil_div(steps, p);
        const int64_t half = ceil_div(T, kHalf.bn) * (kD / kHalf.bm) * p, small = ceil_div(T, kSmall.bn) * (kD / kSmall.bm) * p;
        if (p == 1 || half <= 2 * kCUs)
            consider(c, 0, p, turns(half) * ((2 * half > kCUs ? 0.45 * step : 0.5) * n + 1.0) + add);
        if (p == 1 || small <= 2 * kCUs)
            consider(c, 1, p, turns(small) * (0.62 * (2 * small > kCUs && small <= kCUs ? step : 1.0) * n + 2.0) + add);
        if (p == 1)
            consider(c, 2, p, turns(ceil_div(T, kMid.bn) * (kD / kMid.bm)) * (0.80 * n + 2.0));
    }
    return c;
}

// dX and the weights' gradients in one launch, dX on Half or Small tiles: two
// blocks fit on a CU, and dX's are dispatched first.  While not all are resident
// the CUs' work adds up; what is left then is a launch of its own, in which a
// block that shares its CU takes about half as long again (T = 4096, F = 2048,
// 480 blocks: 67 us expected, 70 measured; 6,000 x 2048, 570: 137 / 131; 6,000 x
// 4104, 870: 198 / 199; 2,500 x 1000, 264: 32 / 35).
inline Choice choose_tail(int64_t T, int64_t F, int64_t Fp)
{
    Choice c{};
    const int64_t steps = 2 * Fp / kStep, dn = grid_blocks((uint32_t)dw_tiles(F, Fp, kSmall)), slots = 2 * kCUs;
    const double dt = 0.47 * ceil_div(T, kStep) + 1.3;
    auto one = [&](int shape, int p, int64_t tiles, double t) {
        const int64_t n = grid_blocks((uint32_t)(tiles * p));   // slots are an XCD's: whole eighths
        if (p > 1 && n > slots)
            return;
        const double add = p > 1 ? reduce_us(T, p) : 0.0;
        double us = 0.0;
        int64_t x = n, w = dn;   // blocks left
        while (x + w > slots) {
            const int64_t xs = x < slots ? x : slots, ws = slots - xs;
            us += (xs * t + ws * dt) / kCUs;
            x -= xs;
            w -= ws;
        }
        const double last = x && t > dt ? t : dt, sum = (x * t + w * dt) / kCUs;
        const double alone = (x + w <= kCUs ? 1.1 : 1.45) * last, longest = (n + dn <= kCUs ? 1.1 : 1.45) * t;
        us += sum > alone ? sum : alone;
        consider(c, shape, p, add + (us > longest ? us : longest));
    };
    for (int p = 1; p <= kMaxRowParts && (p == 1 || 2 * p <= steps); ++p) {
        const double n = (double)ceil_div(steps, p);
        one(0, p, ceil_div(T, kHalf.bn) * (kD / kHalf.bm), 0.5 * n + 1.0);
        one(1, p, ceil_div(T, kSmall.bn) * (kD / kSmall.bm), 0.62 * n + 2.0);
    }
    return c;
}

// The most bytes the parts' sums take for any T up to max_tokens: with parts a
// result has at most 2 kCUs blocks of 128 x 128.
inline uint64_t row_part_bytes(int64_t max_tokens)
{
    const uint64_t all = 2ull * kCUs * kSmall.bm * kSmall.bn * 4, few = 4ull * kMaxRowParts * max_tokens * kD;
    return all < few ? all : few;
}

// The same for the weights' gradients.
inline uint64_t dw_part_bytes(int64_t max_tokens, int64_t Fp)
{
    const int64_t steps = ceil_div(max_tokens, kStep), parts = steps < kMaxParts ? steps : kMaxParts;
    return parts > 1 ? 4ull * parts * 3 * Fp * kD : 0;
}

// What calls of wide_rows keep there in the backward: the parts of dX, then the left-overs.
inline uint64_t wide_bytes(int64_t max_tokens, int64_t F, int64_t Fp)
{
    int64_t most = kFewValues / F;   // positions
    most = most < kFewT ? most : kFewT;
    most = most < max_tokens ? most : max_tokens;
    return most * (4ull * kMaxRowParts * kD + 6ull * Fp);
}

// The weights' gradients; 0 Small, 1 Square.
inline Choice choose_dw(int64_t T, int64_t F, int64_t Fp)
{
    Choice c{};
    const int64_t steps = ceil_div(T, kStep);
    for (int p = 1; p <= kMaxParts && p <= steps; ++p) {
        const double add = p > 1 ? 3.0 + p * Fp * (2.0 * 4 * 3 * kD) / kBytesPerUs : 0.0, n = (double)ceil_div(steps, p);
        const int64_t small = p * dw_tiles(F, Fp, kSmall);
        consider(c, 0, p, rounds(small) * (dw_step(T, Fp, small) * n + 1.3) + add);
        consider(c, 1, p, rounds(p * dw_tiles(F, Fp, kSquare)) * (1.47 * n + 3.5) + add);
    }
    return c;
}

// ---- a call

struct Fwd {
    bool few, wide;       // few: up_few_kernel and down_few_kernel, nothing below
    Choice hidden, rows;
};

inline Fwd plan_fwd(int64_t T, int64_t F)
{
    const int64_t Fp = rup(F, kStep);
    Fwd p{few_rows(T, F), wide_rows(T, F), {}, {}};
    if (!p.few) {
        p.hidden = choose_hidden(T, F, false);
        p.rows = choose_rows(T, Fp / kStep, F % kStep ? 1.4 : 1.0);
    }
    return p;
}

struct Bwd {
    bool wide, merged;    // merged: tail_kernel, rows of which says how; else rows and dw
    Choice hidden, rows, dw;
};

inline Bwd plan_bwd(int64_t T, int64_t F)
{
    const int64_t Fp = rup(F, kStep);
    Bwd p{wide_rows(T, F), false, choose_hidden(T, F, true), choose_rows(T, 2 * Fp / kStep, 1.0), choose_dw(T, F, Fp)};
    const Choice both = choose_tail(T, F, Fp);
    if (p.wide || both.us < p.rows.us + p.dw.us + 2.5) {
        p.merged = true;
        p.rows = both;
        p.dw = Choice{0, 1, 0.0};
    }
    return p;
}

}   // namespace ffn_plan
