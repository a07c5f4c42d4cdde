// Block tiles of a bf16 product on the matrix cores (gfx950):
//   C[m][n] = sum_k A(m, k) B(n, k),  fp32 sums,
// each operand stored k-contiguous (rows of m or n) or k-major (rows of k,
// read through the LDS transpose read).  The accumulators hold 4 consecutive
// m of one n per lane, so outputs are written with m contiguous.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tile {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short v4i16 __attribute__((ext_vector_type(4)));

constexpr int kBK = 64;   // k values of a stage; every contraction's k is padded to it

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Lane l of a wavefront lands its 16 bytes at LDS base + 16 l; the base is
// wavefront-uniform.
__device__ __forceinline__ void lds_load16(const uint16_t *g, uint8_t *lds)
{
    __builtin_amdgcn_global_load_lds((const void *)g, (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
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

// One operand of a contraction.  Rows past the last and columns past the last
// chunk read a row or chunk that exists (their results are dropped); k values
// past the last read 16 bytes of zeros in both operands, so they add 0.
//   k-contiguous: element (r, k) at src[.] + row ld + k
//   k-major:      element (c, k) at src[0] + k ld + c, from k = seg on at src[1] + (k - seg) ld + c
struct Operand {
    const uint16_t *src[2];
    int64_t ld;
    int64_t first;       // first row (k-contiguous) or column (k-major) of the block's tile
    int64_t count;       // rows or columns that exist (columns: a multiple of 8)
    int64_t seg;         // k values of the first source, padded to a multiple of kBK; INT64_MAX: one source
                         // (k-contiguous: both lie in src[0], one after the other)
    int64_t k_valid;     // k values that exist in each source
    int32_t pair;        // k-contiguous: 0, or the rows of a block: blocks of `pair` tile rows alternate
                         // between src[0] and src[1] (both from row `first` on)
};

// Zeros that the loads of k values past the end read.
static __device__ __attribute__((aligned(16))) const uint16_t kZeros[8] = {};

// R rows (or columns) of the tile by kBK values of k, NW wavefronts.
// k-contiguous rows are 128 bytes, 8 chunks of 16 bytes, chunk c of row r at
// position c ^ ((r >> 1) & 7); k-major rows are 2 R bytes, chunk c of row r at
// c ^ (4 (r & 3)) (within the row's chunks): the lanes of one read spread over the banks either way.
template <bool KMAJ, int R, int NW>
struct Loader {
    static constexpr uint32_t BYTES = (uint32_t)R * kBK * 2;
    static constexpr int L = (int)(BYTES / (1024 * NW));   // loads per wavefront and stage
    static_assert(BYTES % (1024 * NW) == 0, "whole loads per wavefront");
    static_assert(!KMAJ || (R & (R - 1)) == 0, "k-major rows swizzle within a power of two");
    static constexpr int CH = KMAJ ? R / 8 : kBK / 8;

    const uint16_t *p[L];
    int kk[L];   // the load's k within a stage
    Operand op;

    __device__ __forceinline__ void init(const Operand &o)
    {
        op = o;
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int q = (j * NW + w) * 64 + lane, r = q / CH, pos = q % CH;
            if constexpr (KMAJ) {
                int64_t c = o.first + 8 * (pos ^ (4 * (r & 3) & (CH - 1)));
                c = c < o.count ? c : 0;
                kk[j] = r;
                p[j] = o.src[0] + (int64_t)r * o.ld + c;
            } else {
                const int ch = pos ^ ((r >> 1) & 7);
                int64_t i;
                const uint16_t *s = o.src[0];
                if (o.pair) {
                    const int b = r / o.pair;
                    i = o.first + (int64_t)(b >> 1) * o.pair + r % o.pair;
                    s = (b & 1) ? o.src[1] : o.src[0];
                } else {
                    i = o.first + r;
                }
                i = i < o.count ? i : o.count - 1;
                kk[j] = 8 * ch;
                p[j] = s + i * o.ld + 8 * ch;
            }
        }
    }

    __device__ __forceinline__ void issue(int64_t k0, uint8_t *lds) const
    {
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const bool second = k0 >= op.seg;
        const int64_t left = op.k_valid - (second ? k0 - op.seg : k0);
        int64_t off = k0;
        if constexpr (KMAJ)
            off = second ? (op.src[1] - op.src[0]) + (k0 - op.seg) * op.ld : k0 * op.ld;
        if (left >= kBK) {
#pragma unroll
            for (int j = 0; j < L; ++j)
                lds_load16(p[j] + off, lds + (j * NW + w) * 1024);
        } else {
#pragma unroll
            for (int j = 0; j < L; ++j)
                lds_load16(kk[j] < left ? p[j] + off : kZeros, lds + (j * NW + w) * 1024);
        }
    }
};

// The fragments of 32 rows (columns) from row0 of the stage, k values 16 kk .. + 15.
template <bool KMAJ, int R>
struct Reader {
    int at, sw;   // lane's offset and swizzle

    __device__ __forceinline__ void init(int row0)
    {
        const int lane = threadIdx.x & 63;
        if constexpr (KMAJ) {
            // within each 16 lanes, lane p addresses row p / 4, columns 4 (p % 4) .. of the
            // four k rows, and receives rows 0 .. 3 of column p
            const int tp = lane & 15, tg = lane >> 4;
            at = (8 * (tg >> 1) + (tp >> 2)) * (2 * R) + 8 * (tp & 1);
            sw = (row0 / 8 + 2 * (tg & 1) + ((tp >> 1) & 1)) ^ (4 * (tp >> 2) & (R / 8 - 1));
        } else {
            const int r = row0 + (lane & 31);
            at = r * (2 * kBK);
            sw = (r >> 1) & 7;
        }
    }

    // block b: rows row0 + 32 b
    __device__ __forceinline__ bf16x8 get(const uint8_t *lds, int b, int kk) const
    {
        if constexpr (KMAJ) {
            // row0 is a multiple of the wavefront's span, a power of two: block b's chunk
            // bits do not meet row0's
            const int ch = sw ^ (4 * b);
            const uint8_t *q = lds + at + 16 * kk * (2 * R) + 16 * ch;
            const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16 *)q);
            const v4i16 hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16 *)(q + 4 * (2 * R)));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int c = 2 * kk + ((threadIdx.x & 63) >> 5);
            return *(const bf16x8 *)(lds + at + 32 * b * (2 * kBK) + 16 * (c ^ sw));
        }
    }
};

// A block tile of (32 WM GM) x (32 WN GN) on GM x GN wavefronts, NS stages of
// kBK.
template <bool AK, bool BK, int WM, int WN, int GM, int GN, int NS>
struct Tile {
    static constexpr int NW = GM * GN, RA = 32 * WM * GM, RB = 32 * WN * GN;
    using LA = Loader<AK, RA, NW>;
    using LB = Loader<BK, RB, NW>;
    static constexpr uint32_t STAGE = LA::BYTES + LB::BYTES, SMEM = NS * STAGE;
    static constexpr int L = LA::L + LB::L;
    static_assert(!AK || (WM & (WM - 1)) == 0, "k-major: a wavefront's span is a power of two");
    static_assert(!BK || (WN & (WN - 1)) == 0, "k-major: a wavefront's span is a power of two");
    static_assert(NS >= 2 && (NS - 2) * L < 64, "loads in flight fit the counter");
};

// acc += the product over K (a multiple of kBK) values of k.  All NS stages
// start filling at once; at each k-step a wavefront waits for the stage it
// reads next, meets the others at a barrier that also frees the stage read
// last, refills that one, and reads the next fragments from LDS while the
// current products run.  Ends with the LDS free.
template <bool AK, bool BK, int WM, int WN, int GM, int GN, int NS>
__device__ __forceinline__ void product(const Operand &A, const Operand &B, int64_t K, uint8_t *sm,
                                        f32x16 (&acc)[WM][WN])
{
    using T = Tile<AK, BK, WM, WN, GM, GN, NS>;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / GN, wn = w % GN;
    typename T::LA la;
    typename T::LB lb;
    la.init(A);
    lb.init(B);
    Reader<AK, T::RA> ra;
    Reader<BK, T::RB> rb;
    ra.init(wm * 32 * WM);
    rb.init(wn * 32 * WN);
    auto issue = [&](int stage, int64_t kt) {
        la.issue(kt * kBK, sm + stage * T::STAGE);
        lb.issue(kt * kBK, sm + stage * T::STAGE + T::LA::BYTES);
    };
    constexpr int KK = kBK / 16;
    const int64_t nk = K / kBK;
#pragma unroll
    for (int st = 0; st < NS; ++st)
        if (st < nk)
            issue(st, st);
    bf16x8 fa[2][WM], fb[2][WN];
    auto rd = [&](int stage, int kk, bf16x8 (&a)[WM], bf16x8 (&b)[WN]) {
        const uint8_t *ab = sm + stage * T::STAGE, *bb = ab + T::LA::BYTES;
#pragma unroll
        for (int mb = 0; mb < WM; ++mb)
            a[mb] = ra.get(ab, mb, kk);
#pragma unroll
        for (int nb = 0; nb < WN; ++nb)
            b[nb] = rb.get(bb, nb, kk);
    };
    auto phase = [&](bool more, int stage, int kk, const bf16x8 (&a)[WM], const bf16x8 (&b)[WN], bf16x8 (&na)[WM],
                     bf16x8 (&nb_)[WN]) {
        __builtin_amdgcn_sched_barrier(0);
        if (more)
            rd(stage, kk, na, nb_);
#pragma unroll
        for (int mb = 0; mb < WM; ++mb)
#pragma unroll
            for (int nb = 0; nb < WN; ++nb)
                acc[mb][nb] = mfma(a[mb], b[nb], acc[mb][nb]);
        if (more) {
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
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    if (nk >= NS)
        wait_vmcnt<(NS - 1) * T::L>();
    else
        wait_vmcnt<0>();
    barrier_nofence();
    rd(0, 0, fa[0], fb[0]);
    int cur = 0;
    constexpr int last = (KK - 1) & 1;
    auto inner = [&]() {
#pragma unroll
        for (int kk = 0; kk + 1 < KK; ++kk)
            phase(true, cur, kk + 1, fa[kk & 1], fb[kk & 1], fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
    };
    for (int64_t kt = 0; kt + 1 < nk; ++kt) {
        inner();
        if (kt + NS - 1 < nk)
            wait_vmcnt<(NS - 2) * T::L>();
        else
            wait_vmcnt<0>();
        barrier_nofence();
        if (kt + NS < nk)
            issue(cur, kt + NS);
        cur = cur + 1 == NS ? 0 : cur + 1;
        phase(true, cur, 0, fa[last], fb[last], fa[0], fb[0]);
    }
    inner();
    phase(false, cur, 0, fa[last], fb[last], fa[0], fb[0]);
    __syncthreads();
}

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
