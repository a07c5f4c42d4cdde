// The n-gram forward with its output dropped in the same pass (gfx950):
//   out[i][j] = k[i][j] c (s_b W_b[r_b(i)][j] + s_t W_t[r_t(i)][j]),
// k and c the mask and scale of include/drop.h for a [T][768] tensor.
//
// The sweep is the plain forward's: a block hashes its positions into LDS, then
// its threads take the positions' 96 groups of 8 elements each, consecutive
// lanes on consecutive pieces of a row.  A thread holds whole mask groups, so it
// makes one Philox call for the 48 (bf16) or 96 (fp32) bytes a group moves:
// bound by HBM and cache bandwidth like the plain forward, with no second pass
// that reads and writes the output again.  8 positions per block, three groups
// per thread, all their loads in flight: 34.3 us for 49,152 positions of 16 GB
// of bf16 tables (6.6 TB/s of rows and output, Zipf rows partly from the
// caches) against 36.0 us with 64 positions per block, and 10.3 against 14.6 us
// for 2,048 positions, which then are 256 blocks instead of 32.
#include "ngram_dev.hpp"
#include "philox.hpp"

#include "../../include/ngram.h"

namespace ngram {

namespace {

constexpr int kTok = 8;   // positions per block
constexpr int kThreads = 256;
constexpr int kGroups = kDim / 8;   // mask groups of a row

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 8 elements of a table row as stored.
template <int ELT>
struct Piece {
    uint4 w[ELT / 2];
};

template <int ELT>
__device__ __forceinline__ Piece<ELT> load_piece(const uint8_t *table, uint32_t row, int group)
{
    const uint4 *p = reinterpret_cast<const uint4 *>(table + (size_t)row * (kDim * ELT)) + group * (ELT / 2);
    Piece<ELT> r;
#pragma unroll
    for (int k = 0; k < ELT / 2; ++k)
        r.w[k] = p[k];
    return r;
}

template <int ELT>
__device__ __forceinline__ void widen(const Piece<ELT> &a, uint32_t sign, float (&v)[8])
{
    const uint32_t *u = reinterpret_cast<const uint32_t *>(a.w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t x = ELT == 2 ? ((k & 1) ? u[k / 2] & 0xFFFF0000u : u[k / 2] << 16) : u[k];
        v[k] = __uint_as_float(x ^ sign);
    }
}

// ELT: table element bytes, OELT: output element bytes; DIRECT: one
// token-indexed table, the output is its row, dropped.
template <int ELT, int OELT, bool DIRECT>
__global__ __launch_bounds__(kThreads) void fwd_drop_kernel(const int32_t *__restrict__ tok, int64_t T, HashParams hp,
                                                            const uint8_t *__restrict__ wb,
                                                            const uint8_t *__restrict__ wt, drop::Mask mask,
                                                            uint8_t *__restrict__ out, uint32_t *__restrict__ flags)
{
    constexpr int kIter = kTok * kGroups / kThreads;   // 3, all in flight
    static_assert(kTok * kGroups % kThreads == 0 && kTok <= kThreads, "whole sweeps");
    __shared__ uint32_t s_idx[2][kTok];
    const int tid = threadIdx.x;
    const drop::Key key = drop::key_of(mask);
    for (int64_t t0 = (int64_t)blockIdx.x * kTok; t0 < T; t0 += (int64_t)gridDim.x * kTok) {
        if (tid < kTok) {
            uint32_t ib = 0, it = 0;
            const int64_t i = t0 + tid;
            if (i < T && ngram_index(tok, i, hp, ib, it) && flags)
                atomicOr(flags, NGRAM_FLAG_BAD_TOKEN);
            s_idx[0][tid] = ib;
            s_idx[1][tid] = it;
        }
        __syncthreads();
        const int ntok = (int)min<int64_t>(kTok, T - t0);
        Piece<ELT> a[kIter], b[kIter];
        uint32_t sa[kIter], sb[kIter];   // sign bits
#pragma unroll
        for (int u = 0; u < kIter; ++u) {
            const int e = tid + u * kThreads, lt = e / kGroups, c = e - lt * kGroups;
            if (lt < ntok) {
                const uint32_t ib = s_idx[0][lt], it = s_idx[1][lt];
                sa[u] = ib & 0x80000000u;
                sb[u] = it & 0x80000000u;
                a[u] = load_piece<ELT>(wb, ib & 0x7FFFFFFFu, c);
                if (!DIRECT)
                    b[u] = load_piece<ELT>(wt, it & 0x7FFFFFFFu, c);
            }
        }
#pragma unroll
        for (int u = 0; u < kIter; ++u) {
            const int e = tid + u * kThreads, lt = e / kGroups;
            if (lt >= ntok)
                continue;
            float v[8];
            widen<ELT>(a[u], sa[u], v);
            if (!DIRECT) {
                float x[8];
                widen<ELT>(b[u], sb[u], x);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] += x[k];
            }
            const uint64_t group = (uint64_t)t0 * kGroups + e;
            if (mask.thr != 0) {
                const uint4 w = drop::bits_of(key, group);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = drop::dropped(v[k], w, k, mask.thr, mask.scale);
            }
            const uint64_t o = (uint64_t)out + group * (8 * OELT);
            if constexpr (OELT == 2) {
                st_global_nt<uint4>(o, make_uint4(bf16_pack_rne(v[0], v[1]), bf16_pack_rne(v[2], v[3]),
                                                  bf16_pack_rne(v[4], v[5]), bf16_pack_rne(v[6], v[7])));
            } else {
                st_global_nt<float4>(o, make_float4(v[0], v[1], v[2], v[3]));
                st_global_nt<float4>(o + 16, make_float4(v[4], v[5], v[6], v[7]));
            }
        }
        __syncthreads();   // s_idx is the next turn's
    }
}

}  // namespace

hipError_t launch_fwd_drop(int dtype, bool out_f32, const HashParams &hp, const void *wb, const void *wt,
                           const int32_t *tok, int64_t T, const drop_spec &spec, void *out, uint32_t *flags,
                           hipStream_t s)
{
    if (T == 0)
        return hipSuccess;
    // a launch counts its threads in 32 bits: a longer micro-step takes several turns of the grid
    const unsigned g = (unsigned)min((T + kTok - 1) / kTok, int64_t(1) << 23);
    auto k = dtype == NGRAM_DTYPE_BF16 ? (out_f32 ? fwd_drop_kernel<2, 4, false> : fwd_drop_kernel<2, 2, false>)
                                       : fwd_drop_kernel<4, 4, false>;
    if (hp.direct)
        k = dtype == NGRAM_DTYPE_BF16 ? (out_f32 ? fwd_drop_kernel<2, 4, true> : fwd_drop_kernel<2, 2, true>)
                                      : fwd_drop_kernel<4, 4, true>;
    launch_prof(NGRAM_PROF_FWD, true, true, k, dim3(g), dim3(kThreads), 0, s, tok, T, hp, (const uint8_t *)wb,
                (const uint8_t *)wt, drop::mask_of(spec), (uint8_t *)out, flags);
    return hipGetLastError();
}

}  // namespace ngram
