/*
 * drop.h -- C ABI of counter-based dropout, for AMD Instinct MI355X (gfx950).
 * Built into the same libngram.so as ngram.h.
 *
 * The mask is a function of (seed, offset, row, column) and is never stored:
 * the backward pass, a recomputation, or a kernel that drops its own output
 * (ngram_embed_fwd_drop, ffn_fwd) computes it again.
 *
 *   y[r][j]  = (res[r][j] +) k[r][j] c x[r][j]
 *   dx[r][j] = k[r][j] c dy[r][j]               (dres = dy)
 *
 * k is 1 for a kept element and 0 for a dropped one, c = 65536 / (65536 -
 * thr) rounded to fp32, thr = round(65536 p) (ties to even): p is held to
 * 2^-17, and c belongs to the share that is really kept, so E[y] = x.  A
 * dropped element is 0 whatever x holds there, NaN and infinities included.
 *
 * The bits: Philox4x32 with 10 rounds (Salmon, Moraes, Dror & Shaw, "Parallel
 * random numbers: as easy as 1, 2, 3", 2011).  Eight neighbouring elements of
 * a row share a call: element j of row r of a [rows][cols] tensor belongs to
 * group g = r ceil(cols / 8) + j / 8, the counter is (g low, g high, offset
 * low, offset high), the key (seed low, seed high), and element j takes bits
 * 16 (j % 2) .. + 15 of output word (j % 8) / 2.  It is kept iff these 16
 * bits, as a number, are at least thr.  Two tensors dropped under one seed
 * need offsets of their own (a counter of calls, say); the same (seed,
 * offset, shape) gives the same mask in every call, on every grid.
 *
 * Conventions: device pointers unless marked "host"; the caller owns every
 * buffer; calls only enqueue on `stream` (a hipStream_t, NULL = the null
 * stream) and never allocate, free or synchronise, so they may be captured in
 * a HIP graph (with drop_spec.rng, a replay takes a new mask); a negative
 * return is a host-detected error with nothing enqueued.
 */
#ifndef DROP_H
#define DROP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DROP_ABI_VERSION 1

#define DROP_OK 0
#define DROP_ENULL -1  /* a required pointer is NULL                          */
#define DROP_EALIGN -2 /* a pointer is not aligned to its elements (rng: 16)  */
#define DROP_ESIZE -4  /* rows or cols negative, cols over 2^31 - 1, or over
                          2^40 elements                                       */
#define DROP_EARG -5   /* p outside [0, 1] or NaN, reserved not 0, an unknown
                          dtype, or buffers that may not overlap as given     */
#define DROP_EHIP -6   /* the HIP runtime reported an error                   */

#define DROP_DTYPE_F32 0
#define DROP_DTYPE_BF16 1

/* The generator's state in device memory (16 bytes, 16-byte aligned): read
 * by the kernels when they run, so a captured graph draws the mask of
 * whatever the caller stored there last.  It lies outside a call's results
 * and workspace. */
typedef struct drop_rng {
    uint64_t seed;
    uint64_t offset;
} drop_rng;

/* Host. */
typedef struct drop_spec {
    float p;             /* share of elements to drop, in [0, 1]; 0 keeps all  */
    int32_t reserved;    /* must be 0                                          */
    uint64_t seed;       /* used where rng is NULL                             */
    uint64_t offset;
    const drop_rng *rng; /* device, or NULL                                    */
} drop_spec;

int drop_abi_version(void);
const char *drop_status_string(int status);

/* y = (res +) dropout(x).  x: [rows][cols] of x_dtype; res (may be NULL) and
 * y: [rows][cols] of y_dtype; all contiguous and aligned to their elements.
 * fp32 inside, one rounding to y_dtype (bf16: nearest, ties to even; a NaN
 * stays a NaN).  y may be x (same dtype) or res, whole; it must not overlap
 * them otherwise.  rows or cols 0 enqueues nothing. */
int drop_fwd(const drop_spec *spec, const void *x, int x_dtype, const void *res, void *y, int y_dtype,
             int64_t rows, int64_t cols, void *stream);

/* dx = dropout(dy) with the forward's spec and shape: the gradient of x (res
 * has dy itself).  dx may be dy (same dtype), whole. */
int drop_bwd(const drop_spec *spec, const void *dy, int dy_dtype, void *dx, int dx_dtype, int64_t rows,
             int64_t cols, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DROP_H */
