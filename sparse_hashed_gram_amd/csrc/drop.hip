// Counter-based dropout (include/drop.h): y = (res +) k c x, and dx = k c dy,
// which is the same kernel without res.
//
// One thread, one group of 8 neighbouring elements of a row: one Philox call
// for 16 (bf16) or 32 (fp32) bytes of each operand.  HBM-bound: every operand
// moves once, the mask never does.  393,216 x 768 bf16 backward: 204 us (5.9
// TB/s of reads and writes; a copy of 2 GiB reaches 4.95); 49,152 x 768 bf16 plus
// an fp32 residual to fp32: 68 us (5.6 TB/s).  Small calls are the launch: 37 x
// 768 7.3 us with the binding, 3.2 of them the launch itself.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/drop.h"
#include "ngram_dev.hpp"
#include "philox.hpp"

namespace {

using namespace drop;

constexpr int kThreads = 256;

// 8 elements at p as floats; n < 8 reads the first n only.  Rows of an odd
// width start at any element, so the 16-byte accesses claim no more than the
// elements' own alignment (global memory takes them unaligned).
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

template <int ELT>
__device__ __forceinline__ void load8(const uint8_t *p, int n, float (&v)[8])
{
    if constexpr (ELT == 2) {
        if (n == 8) {
            const u32x4_a2 w = *reinterpret_cast<const u32x4_a2 *>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = ngram::bf16_lo(w[k]);
                v[2 * k + 1] = ngram::bf16_hi(w[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = k < n ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[k] << 16) : 0.0f;
        }
    } else {
        if (n == 8) {
            const f32x4_a4 a = reinterpret_cast<const f32x4_a4 *>(p)[0], b = reinterpret_cast<const f32x4_a4 *>(p)[1];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = a[k];
                v[4 + k] = b[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = k < n ? reinterpret_cast<const float *>(p)[k] : 0.0f;
        }
    }
}

template <int ELT>
__device__ __forceinline__ void store8(uint8_t *p, int n, const float (&v)[8])
{
    if constexpr (ELT == 2) {
        if (n == 8) {
            u32x4_a2 w;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = ngram::bf16_pack_rne(v[2 * k], v[2 * k + 1]);
            *reinterpret_cast<u32x4_a2 *>(p) = w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n)
                    reinterpret_cast<uint16_t *>(p)[k] = (uint16_t)ngram::bf16_pack_rne(v[k], 0.0f);
        }
    } else {
        if (n == 8) {
            f32x4_a4 a, b;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k] = v[k];
                b[k] = v[4 + k];
            }
            reinterpret_cast<f32x4_a4 *>(p)[0] = a;
            reinterpret_cast<f32x4_a4 *>(p)[1] = b;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n)
                    reinterpret_cast<float *>(p)[k] = v[k];
        }
    }
}

// XE, YE: element bytes of x and of res / y.  Group g is (row g / per, piece
// g % per), and the counter of its mask is g itself.
template <int XE, int YE, bool RES>
__global__ __launch_bounds__(kThreads) void drop_kernel(Mask m, const uint8_t *x, const uint8_t *res, uint8_t *y,
                                                        uint64_t groups, uint32_t per, uint32_t cols)
{
    const Key key = key_of(m);
    for (uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x; g < groups; g += (uint64_t)gridDim.x * kThreads) {
        uint64_t at = g * 8;   // the group's first element
        int n = 8;
        if (cols % 8 != 0) {
            const uint64_t row = groups >> 32 ? g / per : (uint64_t)((uint32_t)g / per);
            const uint32_t piece = (uint32_t)(g - row * per);
            at = row * cols + (uint64_t)piece * 8;
            n = (int)min(8u, cols - piece * 8);
        }
        float v[8], r[8];
        load8<XE>(x + at * XE, n, v);
        if constexpr (RES)
            load8<YE>(res + at * YE, n, r);
        if (m.thr != 0) {
            const uint4 w = bits_of(key, g);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = dropped(v[e], w, e, m.thr, m.scale);
        }
        if constexpr (RES) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] += r[e];
        }
        store8<YE>(y + at * YE, n, v);
    }
}

int elt_of(int dtype) { return dtype == DROP_DTYPE_F32 ? 4 : 2; }

// y may be a whole operand of its own dtype, else it has to lie apart from it.
bool apart(const void *a, uint64_t na, const void *b, uint64_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x + na <= y || y + nb <= x;
}

int run(const drop_spec *spec, const void *x, int x_dtype, const void *res, void *y, int y_dtype, int64_t rows,
        int64_t cols, void *stream)
{
    const int rc = check_spec(spec);
    if (rc)
        return rc;
    if ((x_dtype != DROP_DTYPE_F32 && x_dtype != DROP_DTYPE_BF16) ||
        (y_dtype != DROP_DTYPE_F32 && y_dtype != DROP_DTYPE_BF16))
        return DROP_EARG;
    if (rows < 0 || cols < 0 || cols > INT32_MAX || (cols > 0 && rows > (int64_t(1) << 40) / cols))
        return DROP_ESIZE;
    if (rows == 0 || cols == 0)
        return DROP_OK;
    if (!x || !y)
        return DROP_ENULL;
    const int xe = elt_of(x_dtype), ye = elt_of(y_dtype);
    if ((uintptr_t)x % xe || (uintptr_t)y % ye || (uintptr_t)res % ye)
        return DROP_EALIGN;
    const uint64_t n = (uint64_t)rows * (uint64_t)cols;
    if (!(x == y && xe == ye) && !apart(x, n * xe, y, n * ye))
        return DROP_EARG;
    if (res && res != y && !apart(res, n * ye, y, n * ye))
        return DROP_EARG;
    if (spec->rng && !apart(spec->rng, sizeof(drop_rng), y, n * ye))   // read by every block, after others wrote
        return DROP_EARG;
    const uint32_t per = (uint32_t)((cols + 7) / 8);
    const uint64_t groups = (uint64_t)rows * per;
    const Mask m = mask_of(*spec);
    hipStream_t s = (hipStream_t)stream;
    // a launch counts its threads in 32 bits: larger tensors take several groups a thread
    const unsigned grid = (unsigned)std::min<uint64_t>((groups + kThreads - 1) / kThreads, 1u << 23);
    auto k = res ? (xe == 2 ? (ye == 2 ? drop_kernel<2, 2, true> : drop_kernel<2, 4, true>)
                            : (ye == 2 ? drop_kernel<4, 2, true> : drop_kernel<4, 4, true>))
                 : (xe == 2 ? (ye == 2 ? drop_kernel<2, 2, false> : drop_kernel<2, 4, false>)
                            : (ye == 2 ? drop_kernel<4, 2, false> : drop_kernel<4, 4, false>));
    k<<<grid, kThreads, 0, s>>>(m, (const uint8_t *)x, (const uint8_t *)res, (uint8_t *)y, groups, per,
                                (uint32_t)cols);
    return hipGetLastError() == hipSuccess ? DROP_OK : DROP_EHIP;
}

}   // namespace

extern "C" {

int drop_abi_version(void) { return DROP_ABI_VERSION; }

const char *drop_status_string(int status)
{
    switch (status) {
    case DROP_OK: return "ok";
    case DROP_ENULL: return "a required pointer is NULL";
    case DROP_EALIGN: return "a pointer is misaligned";
    case DROP_ESIZE: return "size out of range";
    case DROP_EARG: return "argument out of range";
    case DROP_EHIP: return "HIP runtime error";
    default: return "unknown status";
    }
}

int drop_fwd(const drop_spec *spec, const void *x, int x_dtype, const void *res, void *y, int y_dtype,
             int64_t rows, int64_t cols, void *stream)
{
    return run(spec, x, x_dtype, res, y, y_dtype, rows, cols, stream);
}

int drop_bwd(const drop_spec *spec, const void *dy, int dy_dtype, void *dx, int dx_dtype, int64_t rows,
             int64_t cols, void *stream)
{
    return run(spec, dy, dy_dtype, nullptr, dx, dx_dtype, rows, cols, stream);
}

}   // extern "C"
