// Block tiles of a bf16 product on the matrix cores (gfx950):
//   C[m][n] = sum_k A(m, k) B(n, k),  fp32 sums,
// each operand stored k-contiguous (rows of m or n) or k-major (rows of k,
// read through the LDS transpose read).  The accumulators hold 4 consecutive
// m of one n per lane, so outputs are written with m contiguous.
//
// What bounds a tile (measured on MI355X): on real data the matrix cores
// sustain 1.64 - 1.72 PFLOP/s, and a CU takes about 44 bytes per clock through
// direct global -> LDS loads if they cover whole 128-byte lines (27 TB/s over
// the chip; 17 TB/s with 64-byte pieces, hence stages of 64 values of k).  A
// step of 64 k moves 32 KB for a 128 x 128 tile (745 clocks against 512 of
// products) and 64 KB for a 256 x 256 tile (1,490 against 2,048), so large
// tiles are for full chips and small ones for latency.  With one wavefront on a
// SIMD the loops below are bound by their instruction count, so their bodies
// hold little address arithmetic: loads take a scalar base and a constant lane
// offset, LDS reads constant offsets from a few lane addresses.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tile {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short v4i16 __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int kBK = 64;   // k values of a stage; every contraction's k is padded to it

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// s_waitcnt vmcnt(N), other counters left alone (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Barrier without a memory fence: a fence would wait for every LDS-bound load
// in flight.  The caller has waited for the loads it needs; this waits for the
// wavefront's LDS reads.
__device__ __forceinline__ void barrier_nofence()
{
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// threadIdx.x, worked out anew where it is used: what is derived from it is not
// kept in registers from one place to the next.
__device__ __forceinline__ int fresh_tid()
{
    int t = (int)threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// One operand of a contraction.  Rows past the last and columns past the last
// chunk read a row or chunk that exists (their results are dropped); k values
// past the last read 16 bytes of zeros in both operands, so they add 0.
//   k-contiguous: element (r, k) at src[.] + row ld + k
//   k-major:      element (c, k) at src[0] + k ld + c, from k = seg on at src[1] + (k - seg) ld + c
struct Operand {
    const uint16_t *src[2];
    int64_t ld;
    int64_t first;      // first row (k-contiguous) or column (k-major) of the block's tile, below count
    int64_t count;      // rows or columns that exist (columns: a multiple of 8)
    int32_t seg;        // k values of the first source, padded to a multiple of kBK; INT32_MAX: one source
                        // (k-contiguous: both lie in src[0], one after the other)
    int32_t k_valid;    // k values that exist in each source
    int32_t pair;       // k-contiguous: 0, or the rows of a block: blocks of `pair` tile rows (a multiple of
                        // 8) alternate between src[0] and src[1], both from row `first` on
};

// Zeros that the loads of k values past the end read.
static __device__ __attribute__((aligned(16))) const uint16_t kZeros[8] = {};

// Loads of R rows (or columns) of the tile by NW wavefronts, one stage a call,
// direct to LDS: lane l of a wavefront lands its 16 bytes at base + 16 l.
// k-contiguous rows are 128 bytes, 8 chunks of 16 bytes, chunk c of row r at
// position c ^ ((r >> 1) & 7); k-major rows are 2 R bytes, chunk c of row r at
// c ^ (4 (r & 3)) (within the row's chunks): the lanes of one read spread over
// the banks either way.  A load's lanes cover 8 rows (k-contiguous) or whole
// k rows, full lines in both.
template <bool KMAJ, int R, int NW>
struct Loader {
    static constexpr uint32_t BYTES = (uint32_t)R * kBK * 2;
    static constexpr int L = (int)(BYTES / (1024 * NW));   // loads per wavefront and stage
    static_assert(BYTES % (1024 * NW) == 0, "whole loads per wavefront");
    static_assert(!KMAJ || (R & (R - 1)) == 0, "k-major rows swizzle within a power of two");
    static constexpr int CH = KMAJ ? R / 8 : kBK / 8;

    uint32_t off[L];           // bytes from the tile's base to the lane's chunk
    const uint8_t *cur[2];     // the stage's base in each source
    const uint8_t *next_src;   // k-major: the second source's base
    int64_t step;              // bytes from a stage to the next
    int32_t k, seg, k_valid, w;
    bool second[L];            // k-contiguous pairs: load j comes from src[1] (uniform)

    // row and chunk that load j of thread tid fills
    static __device__ __forceinline__ void place(int tid, int j, int &r, int &ch)
    {
        const int q = (j * NW) * 64 + tid, pos = q % CH;
        r = q / CH;
        ch = KMAJ ? pos ^ (4 * (r & 3) & (CH - 1)) : pos ^ ((r >> 1) & 7);
    }

    // The lanes' offsets.  They hold for every tile that lies inside the operand.
    __device__ __forceinline__ void set_lanes(const Operand &o)
    {
        w = wave_id();
        const int tid = fresh_tid();
#pragma unroll
        for (int j = 0; j < L; ++j) {
            int r, ch;
            place(tid, j, r, ch);
            second[j] = false;
            if constexpr (KMAJ) {
                const int64_t c = o.first + 8 * ch < o.count ? 8 * ch : 0;
                off[j] = (uint32_t)(2 * (r * o.ld + c));
            } else {
                int64_t i = r;
                if (o.pair) {
                    const int b = r / o.pair;
                    i = (b >> 1) * o.pair + r % o.pair;
                    second[j] = (((j * NW + w) * 8) / o.pair) & 1;   // 8 rows per load
                }
                i = o.first + i < o.count ? i : o.count - 1 - o.first;
                off[j] = (uint32_t)(2 * (i * o.ld + 8 * ch));
            }
        }
    }

    // The first stage: k0, a multiple of kBK.  Scalar work only.
    __device__ __forceinline__ void set_base(const Operand &o, int32_t k0)
    {
        k = k0;
        seg = o.seg;
        k_valid = o.k_valid;
        const int64_t at = KMAJ ? o.first : o.first * o.ld;
        step = 2 * (KMAJ ? kBK * o.ld : kBK);
        next_src = (const uint8_t *)(o.src[1] + at);
        cur[0] = (const uint8_t *)(o.src[0] + at) + k0 / kBK * step;
        cur[1] = next_src + k0 / kBK * step;
        if (KMAJ && k0 >= seg)
            cur[0] = next_src + (k0 - seg) / kBK * step;
    }

    // The next stage, to lds.
    __device__ __forceinline__ void issue(lds_u8 *lds)
    {
        const int32_t left = k_valid - (k >= seg ? k - seg : k);   // at least 1
        if (left >= kBK) {
#pragma unroll
            for (int j = 0; j < L; ++j) {
                // widened here, not before the loop, so that the load takes base and
                // offset as they are instead of a 64-bit sum
                uint32_t o = off[j];
                asm volatile("" : "+v"(o));
                load((!KMAJ && second[j] ? cur[1] : cur[0]) + o, lds, j);
            }
        } else {
            const int tid = fresh_tid();   // rare
#pragma unroll
            for (int j = 0; j < L; ++j) {
                int r, ch;
                place(tid, j, r, ch);
                uint32_t o = off[j];
                asm volatile("" : "+v"(o));
                const uint8_t *p = (!KMAJ && second[j] ? cur[1] : cur[0]) + o;
                load((KMAJ ? r : 8 * ch) < left ? p : (const uint8_t *)kZeros, lds, j);
            }
        }
        k += kBK;
        cur[0] += step;
        if constexpr (KMAJ) {
            if (k == seg)
                cur[0] = next_src;
        } else {
            cur[1] += step;
        }
    }

    __device__ __forceinline__ void load(const uint8_t *g, lds_u8 *lds, int j) const
    {
        __builtin_amdgcn_global_load_lds((const void *)g, lds + (j * NW + w) * 1024, 16, 0, 0);
    }
};

// Fragments of a wavefront's N blocks of 32 rows (columns) from row0 of a stage.
template <bool KMAJ, int R, int N>
struct Reader {
    static_assert(!KMAJ || (N & (N - 1)) == 0, "k-major: a wavefront's span is a power of two");
    uint32_t ad[KMAJ ? N : kBK / 16];   // bytes in the stage; k-major: by block; k-contiguous: by sub-step of 16 k

    // at: the operand's bytes into a stage
    __device__ __forceinline__ void init(uint32_t at, int row0)
    {
        const int lane = fresh_tid() & 63;
        if constexpr (KMAJ) {
            // within each 16 lanes, lane p addresses row p / 4, columns 4 (p % 4) .. of the
            // four k rows, and receives rows 0 .. 3 of column p.  row0 is a multiple of the
            // wavefront's span, a power of two: block b's chunk bits do not meet row0's
            const int tp = lane & 15, tg = lane >> 4;
            const uint32_t row = at + (8 * (tg >> 1) + (tp >> 2)) * (2 * R) + 8 * (tp & 1);
            const int ch = row0 / 8 + 2 * (tg & 1) + ((tp >> 1) & 1), sw = 4 * (tp >> 2) & (R / 8 - 1);
#pragma unroll
            for (int b = 0; b < N; ++b)
                ad[b] = row + 16 * ((ch ^ (4 * b)) ^ sw);
        } else {
            const int r = row0 + (lane & 31);
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
                ad[kk] = at + r * (2 * kBK) + 16 * ((2 * kk + (lane >> 5)) ^ ((r >> 1) & 7));
        }
    }

    // block b, k values 16 kk .. + 15 of the stage
    __device__ __forceinline__ bf16x8 get(const lds_u8 *stage, int b, int kk) const
    {
        typedef __attribute__((address_space(3))) v4i16 lds_v4;
        typedef __attribute__((address_space(3))) const bf16x8 lds_v8;
        if constexpr (KMAJ) {
            const lds_u8 *q = stage + ad[b] + 16 * kk * (2 * R);
            const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)q);
            const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4 *)(q + 4 * (2 * R)));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return *(lds_v8 *)(stage + ad[kk] + 32 * b * (2 * kBK));
        }
    }
};

// A block tile of (32 WM GM) x (32 WN GN) on GM x GN wavefronts, two stages.
template <bool AK, bool BK, int WM, int WN, int GM, int GN>
struct Tile {
    static constexpr int NW = GM * GN, RA = 32 * WM * GM, RB = 32 * WN * GN;
    using LA = Loader<AK, RA, NW>;
    using LB = Loader<BK, RB, NW>;
    using FA = Reader<AK, RA, WM>;
    using FB = Reader<BK, RB, WN>;
    static constexpr uint32_t STAGE = LA::BYTES + LB::BYTES, SMEM = 2 * STAGE;

    LA la;
    LB lb;
    FA ra;
    FB rb;

    __device__ __forceinline__ void init(const Operand &A, const Operand &B, int32_t k0)
    {
        const int w = wave_id();
        la.set_lanes(A);
        la.set_base(A, k0);
        lb.set_lanes(B);
        lb.set_base(B, k0);
        ra.init(LB::BYTES, w / GN * 32 * WM);
        rb.init(0, w % GN * 32 * WN);
    }

    __device__ __forceinline__ void issue(lds_u8 *stage)
    {
        lb.issue(stage);
        la.issue(stage + LB::BYTES);
    }

    __device__ __forceinline__ void read(const lds_u8 *stage, int kk, bf16x8 (&a)[WM], bf16x8 (&b)[WN]) const
    {
#pragma unroll
        for (int mb = 0; mb < WM; ++mb)
            a[mb] = ra.get(stage, mb, kk);
#pragma unroll
        for (int nb = 0; nb < WN; ++nb)
            b[nb] = rb.get(stage, nb, kk);
    }
};

template <int WM, int WN>
__device__ __forceinline__ void multiply(const bf16x8 (&a)[WM], const bf16x8 (&b)[WN], f32x16 (&acc)[WM][WN])
{
#pragma unroll
    for (int mb = 0; mb < WM; ++mb)
#pragma unroll
        for (int nb = 0; nb < WN; ++nb)
            acc[mb][nb] = mfma(a[mb], b[nb], acc[mb][nb]);
}

// The bodies below take their two stages as __restrict__ pointers: a load to one
// then does not alias a read of the other, or the compiler would put a wait for
// every load in flight before each transpose read.

// Products of one sub-step with the reads of the next, one read after each product.
template <typename T, bool AK, bool BK, int WM, int WN>
__device__ __forceinline__ void sub_step(const T &t, const lds_u8 *stage, int kk, const bf16x8 (&a)[WM],
                                         const bf16x8 (&b)[WN], bf16x8 (&na)[WM], bf16x8 (&nb)[WN],
                                         f32x16 (&acc)[WM][WN])
{
    __builtin_amdgcn_sched_barrier(0);
    t.read(stage, kk, na, nb);
    multiply(a, b, acc);
    constexpr int NR = (AK ? 2 : 1) * WM + (BK ? 2 : 1) * WN, NM = WM * WN, NP = NR < NM ? NR : NM;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one matrix-core op
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
    }
    if constexpr (NM > NP)
        __builtin_amdgcn_sched_group_barrier(0x008, NM - NP, 0);
    if constexpr (NR > NP)
        __builtin_amdgcn_sched_group_barrier(0x100, NR - NP, 0);
    __builtin_amdgcn_sched_barrier(0);
}

// Two steps of the four-wavefront loop, stages kt (s0) and kt + 1 (s1) of nk.
// Sub-step 0's fragments of a stage are in fa[0], fb[0] when its step begins.  At
// each step a wavefront waits for the stage it reads next, meets the others at
// a barrier that also frees the stage read last, refills that one, and reads
// the next fragments from LDS while the current products run.  (Past the last
// stage it reads what the other one held: the loop has one body, so the
// accumulators stay in their registers.)
template <bool AK, bool BK, int WM, int WN, int GM, int GN>
__device__ __forceinline__ void steps4(Tile<AK, BK, WM, WN, GM, GN> &t, int kt, int nk, lds_u8 *__restrict__ s0,
                                       lds_u8 *__restrict__ s1, bf16x8 (&fa)[2][WM], bf16x8 (&fb)[2][WN],
                                       f32x16 (&acc)[WM][WN])
{
    using T = Tile<AK, BK, WM, WN, GM, GN>;
    constexpr int KK = kBK / 16;
    static_assert(KK == 4, "fragment buffers alternate within a stage");
    sub_step<T, AK, BK>(t, s0, 1, fa[0], fb[0], fa[1], fb[1], acc);
    sub_step<T, AK, BK>(t, s0, 2, fa[1], fb[1], fa[0], fb[0], acc);
    sub_step<T, AK, BK>(t, s0, 3, fa[0], fb[0], fa[1], fb[1], acc);
    wait_vmcnt<0>();
    barrier_nofence();
    sub_step<T, AK, BK>(t, s1, 0, fa[1], fb[1], fa[0], fb[0], acc);
    if (kt + 1 >= nk)
        return;
    if (kt + 2 < nk)
        t.issue(s0);
    sub_step<T, AK, BK>(t, s1, 1, fa[0], fb[0], fa[1], fb[1], acc);
    sub_step<T, AK, BK>(t, s1, 2, fa[1], fb[1], fa[0], fb[0], acc);
    sub_step<T, AK, BK>(t, s1, 3, fa[0], fb[0], fa[1], fb[1], acc);
    wait_vmcnt<0>();
    barrier_nofence();
    sub_step<T, AK, BK>(t, s0, 0, fa[1], fb[1], fa[0], fb[0], acc);
    if (kt + 3 < nk)
        t.issue(s1);
}

// The same on eight wavefronts in two groups of four, one wavefront of each
// group on every SIMD.  The groups run the same half steps (32 values of k) one
// phase apart: while one reads its fragments from LDS and starts loads, the
// other has the matrix cores, and at each barrier they change places.  A SIMD's
// matrix core is then fed by one wavefront while the other waits for LDS, and
// one block per CU (large tiles, little traffic per product) is enough.
//
// Stage H is half steps 2 H and 2 H + 1.  Group 0 reads half step h in phase 2 h
// and multiplies in phase 2 h + 1, group 1 one phase later; a barrier ends every
// phase.
//   - Stage H + 1 is started in the reading phase of half step 2 H (4 H or
//     4 H + 1), into the buffer of stage H - 1, which group 1 has read by the end
//     of phase 4 H - 1.
//   - Every wavefront's share of stage H + 1 has landed by the end of phase
//     4 H + 3: group 0 waits after its products, group 1 after its reads.
template <int WM, int WN>
__device__ __forceinline__ void products8(const bf16x8 (&fa)[2][WM], const bf16x8 (&fb)[2][WN], f32x16 (&acc)[WM][WN])
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    multiply(fa[0], fb[0], acc);
    multiply(fa[1], fb[1], acc);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
}

// One stage of a group; next(other) starts what follows it, if anything.
template <int GROUP, typename T, int WM, int WN, typename Next>
__device__ __forceinline__ void step8(T &t, const lds_u8 *__restrict__ stage,
                                      lds_u8 *__restrict__ other, f32x16 (&acc)[WM][WN], Next next)
{
    bf16x8 fa[2][WM], fb[2][WN];
    t.read(stage, 0, fa[0], fb[0]);
    t.read(stage, 1, fa[1], fb[1]);
    next(other);
    barrier_nofence();
    products8(fa, fb, acc);
    barrier_nofence();
    t.read(stage, 2, fa[0], fb[0]);
    t.read(stage, 3, fa[1], fb[1]);
    if (GROUP == 1)
        wait_vmcnt<0>();
    barrier_nofence();
    products8(fa, fb, acc);
    if (GROUP == 0)
        wait_vmcnt<0>();
    barrier_nofence();
}

template <int GROUP, typename T, int WM, int WN, typename Next>
__device__ __forceinline__ void loop8(T &t, int nk, lds_u8 *&s0, lds_u8 *&s1,
                                      f32x16 (&acc)[WM][WN], Next next)
{
    if (GROUP == 1)
        barrier_nofence();
    for (int H = 0; H < nk; ++H) {
        step8<GROUP>(t, s0, s1, acc, [&](lds_u8 *other) {
            if (H + 1 < nk)
                t.issue(other);
            else
                next(other);
        });
        lds_u8 *const other = s0;
        s0 = s1;
        s1 = other;
    }
    if (GROUP == 0)
        barrier_nofence();
}

// acc += the product over nk stages of t (a Tile, or its like: issue, read), whose first stage lies in s0, landed
// for every wavefront.  next(stage) starts the first stage of whatever is
// multiplied after it (or nothing): afterwards that lies in s0, landed for every
// wavefront, and s1 is free.
template <typename T, int WM, int WN, typename Next>
__device__ __forceinline__ void chain8(T &t, int nk, lds_u8 *&s0, lds_u8 *&s1, f32x16 (&acc)[WM][WN], Next next)
{
    if (wave_id() < 4)
        loop8<0>(t, nk, s0, s1, acc, next);
    else
        loop8<1>(t, nk, s0, s1, acc, next);
}

// The two stages' places.  The second as a value, not a constant: past the 64 KB
// that an LDS read's offset reaches, folded constants would cost a register per
// read.
__device__ __forceinline__ void places(uint8_t *sm, uint32_t stage, lds_u8 *&s0, lds_u8 *&s1)
{
    asm volatile("" : "+s"(stage));
    s0 = (lds_u8 *)sm;
    s1 = s0 + stage;
}

// acc += the product over K values of k from k0 on (both multiples of kBK, K at
// least kBK).  Ends with the LDS free.
template <bool AK, bool BK, int WM, int WN, int GM, int GN>
__device__ __forceinline__ void product(const Operand &A, const Operand &B, int32_t k0, int32_t K, uint8_t *sm,
                                        f32x16 (&acc)[WM][WN])
{
    using T = Tile<AK, BK, WM, WN, GM, GN>;
    static_assert(GM * GN <= 4 || GM * GN == 8, "one group, or two of four");
    T t;
    t.init(A, B, k0);
    lds_u8 *s0, *s1;
    places(sm, T::STAGE, s0, s1);
    const int nk = K / kBK;
    t.issue(s0);
    if constexpr (GM * GN == 8) {
        wait_vmcnt<0>();
        barrier_nofence();
        chain8(t, nk, s0, s1, acc, [](lds_u8 *) {});
    } else {
        if (nk > 1) {
            t.issue(s1);
            wait_vmcnt<T::LA::L + T::LB::L>();
        } else {
            wait_vmcnt<0>();
        }
        barrier_nofence();
        bf16x8 fa[2][WM], fb[2][WN];
        t.read(s0, 0, fa[0], fb[0]);
        for (int kt = 0; kt < nk; kt += 2)
            steps4(t, kt, nk, s0, s1, fa, fb, acc);
    }
    __syncthreads();
}

// Two products of one stage each, the first kBK values of k and the next, into
// sums of their own; both stages' loads are in flight at once.
template <bool AK, bool BK, int WM, int WN, int GM, int GN>
__device__ __forceinline__ void product_1_1(const Operand &A, const Operand &B, uint8_t *sm, f32x16 (&acc1)[WM][WN],
                                            f32x16 (&acc2)[WM][WN])
{
    using T = Tile<AK, BK, WM, WN, GM, GN>;
    T t;
    t.init(A, B, 0);
    lds_u8 *s0, *s1;
    places(sm, T::STAGE, s0, s1);
    t.issue(s0);
    t.issue(s1);
    wait_vmcnt<0>();
    barrier_nofence();
    bf16x8 a[WM], b[WN];
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
        t.read(s0, kk, a, b);
        multiply(a, b, acc1);
    }
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
        t.read(s1, kk, a, b);
        multiply(a, b, acc2);
    }
    __syncthreads();
}

// Two products over the same K, step by step together.  A step of a small tile is
// its own chain of LDS reads, dependent matrix instructions and a barrier (0.3
// us for two instructions a sub-step), so two of them cost little more than one.
template <typename T1, typename T2, bool AK1, bool AK2, bool BK, int M1, int M2, int WN>
__device__ __forceinline__ void pair_steps(T1 &t1, T2 &t2, int kt, int nk, lds_u8 *__restrict__ s0,
                                           lds_u8 *__restrict__ s1, lds_u8 *__restrict__ u0,
                                           lds_u8 *__restrict__ u1, bf16x8 (&a1)[2][M1], bf16x8 (&b1)[2][WN],
                                           bf16x8 (&a2)[2][M2], bf16x8 (&b2)[2][WN], f32x16 (&acc1)[M1][WN],
                                           f32x16 (&acc2)[M2][WN])
{
    auto sub = [&](const lds_u8 *s, const lds_u8 *u, int kk, int from) {
        sub_step<T1, AK1, BK>(t1, s, kk, a1[from], b1[from], a1[1 - from], b1[1 - from], acc1);
        sub_step<T2, AK2, BK>(t2, u, kk, a2[from], b2[from], a2[1 - from], b2[1 - from], acc2);
    };
    sub(s0, u0, 1, 0);
    sub(s0, u0, 2, 1);
    sub(s0, u0, 3, 0);
    wait_vmcnt<0>();
    barrier_nofence();
    sub(s1, u1, 0, 1);
    if (kt + 1 >= nk)
        return;
    if (kt + 2 < nk) {
        t1.issue(s0);
        t2.issue(u0);
    }
    sub(s1, u1, 1, 0);
    sub(s1, u1, 2, 1);
    sub(s1, u1, 3, 0);
    wait_vmcnt<0>();
    barrier_nofence();
    sub(s0, u0, 0, 1);
    if (kt + 3 < nk) {
        t1.issue(s1);
        t2.issue(u1);
    }
}

// acc1 += A1 B1, acc2 += A2 B2 over K values of k (at least two stages).
template <bool AK1, bool AK2, bool BK, int M1, int M2, int WN, int GM, int GN>
struct Pair {
    using T1 = Tile<AK1, BK, M1, WN, GM, GN>;
    using T2 = Tile<AK2, BK, M2, WN, GM, GN>;
    static constexpr uint32_t SMEM = T1::SMEM + T2::SMEM;

    static __device__ __forceinline__ void run(const Operand &A1, const Operand &B1, const Operand &A2,
                                               const Operand &B2, int32_t K, uint8_t *sm, f32x16 (&acc1)[M1][WN],
                                               f32x16 (&acc2)[M2][WN])
    {
        static_assert(GM * GN <= 4, "the four-wavefront loop");
        T1 t1;
        T2 t2;
        lds_u8 *s0, *s1, *u0, *u1;
        places(sm, T1::STAGE, s0, s1);
        places(sm + T1::SMEM, T2::STAGE, u0, u1);
        const int nk = K / kBK;
        t1.init(A1, B1, 0);
        t2.init(A2, B2, 0);
        t1.issue(s0);
        t2.issue(u0);
        t1.issue(s1);
        t2.issue(u1);
        wait_vmcnt<T1::LA::L + T1::LB::L + T2::LA::L + T2::LB::L>();
        barrier_nofence();
        bf16x8 a1[2][M1], b1[2][WN], a2[2][M2], b2[2][WN];
        t1.read(s0, 0, a1[0], b1[0]);
        t2.read(u0, 0, a2[0], b2[0]);
        for (int kt = 0; kt < nk; kt += 2)
            pair_steps<T1, T2, AK1, AK2, BK>(t1, t2, kt, nk, s0, s1, u0, u1, a1, b1, a2, b2, acc1, acc2);
        __syncthreads();
    }
};

template <int WM, int WN>
__device__ __forceinline__ void clear(f32x16 (&acc)[WM][WN])
{
#pragma unroll
    for (int mb = 0; mb < WM; ++mb)
#pragma unroll
        for (int nb = 0; nb < WN; ++nb)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[mb][nb][e] = 0.0f;
}

}  // namespace tile
