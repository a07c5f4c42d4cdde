/*
 * norm.h -- C ABI of the norms around a block, alone and joined with the
 * block's gate and the residual stream, for AMD Instinct MI355X (gfx950).
 * Built into the same libngram.so as ngram.h.
 *
 * The norm of a row x of D values (w, b may be absent: 1 and 0):
 *
 *   mu = 0 (RMS) or mean(x) (LAYER),  rho = 1 / sqrt(mean((x - mu)^2) + eps)
 *   xh = (x - mu) rho,  norm(x; w, b) = xh w + b
 *
 * norm_fwd:       X = norm(R; w, b)           in front of a block
 * norm_join_fwd:  N = norm(B; post_w, post_b) (NORM_OPT_POST, else N = B)
 *                 R1 = s R + g N              behind it; g: nothing (1), one
 *                                             number, [D], or sigmoid(G), G [T][D]
 *                 X = norm(R1; w, b)          in front of the next one (NORM_OPT_PRE)
 *
 * and backwards, with dxh = dX w and dR1 the gradient that reaches R1 along
 * the residual stream:
 *
 *   E = dR1 + rho (dxh - [LAYER] mean(dxh) - xh mean(dxh xh))   (of R1, or of R)
 *   dw (+)= sum_t dX xh,  db (+)= sum_t dX
 *   dR = s E,  ds (+)= sum_t E R  (one number: over D too)
 *   dg (+)= sum_t E N  (one number: over D too), or dG = E N sigmoid'(G)
 *   dN = g E,  and dB, dpost_w, dpost_b from dN as E, dw, db from dX
 *
 * R, R1, dR1, dR: [T][D] of r_dtype; B, X, G, dX, dB, dG: [T][D] of x_dtype;
 * the parameters (w, b, post_w, post_b [D]; g, s: [D] or one number) of p_dtype
 * and their gradients of dp_dtype.  All contiguous, aligned to their elements.
 *
 * Precision: fp32 inside, the rows' sums and the sums over t too; each result is
 * rounded once (bf16: nearest, ties to even).  X is the norm of R1 as it is
 * before it is rounded to r_dtype; the backward takes R1 as it was stored.  A row
 * whose squares pass fp32's range is normalised all the same, with LAYER to 0 where
 * all its values are equal.  (Otherwise the mean is rounded to fp32: deviations below
 * some 2^-22 of it are noise.)  The norm of a row with a NaN or an infinity is NaN, all of
 * it, and with it the row's gradient and the sums over t that its xh is in; no other row.
 *
 * Conventions: device pointers unless marked "host"; the caller owns every
 * buffer; calls only enqueue on `stream` (a hipStream_t, NULL = the null
 * stream), never allocate, free or synchronise, and may be captured in a HIP
 * graph; a negative return is a host-detected error with nothing enqueued.
 * The workspace (of the backward only) holds nothing between calls: calls that
 * share one must be ordered (one stream), and graphs that were captured with
 * the same one must not run at the same time.  Results are the same, bit for
 * bit, in every run of the same call.
 */
#ifndef NORM_H
#define NORM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define NORM_ABI_VERSION 1

#define NORM_OK 0
#define NORM_ENULL -1   /* a required pointer is NULL                          */
#define NORM_EALIGN -2  /* a pointer is not aligned to its elements (workspace: 256) */
#define NORM_ECONFIG -3 /* the config is invalid                               */
#define NORM_ESIZE -4   /* T negative or over 2^31 - 1, or a workspace too small */
#define NORM_EARG -5    /* an output that overlaps an operand or another output
                           otherwise than it may                               */
#define NORM_EHIP -6    /* the HIP runtime reported an error                   */

#define NORM_KIND_RMS 0
#define NORM_KIND_LAYER 1

#define NORM_DTYPE_F32 0
#define NORM_DTYPE_BF16 1

/* of the gate g and (the first three) the residual scale s */
#define NORM_BY_NONE 0   /* 1                                                  */
#define NORM_BY_SCALAR 1 /* one number in device memory                        */
#define NORM_BY_VECTOR 2 /* [D]                                                */
#define NORM_BY_TOKEN 3  /* sigmoid(G), G [T][D] of x_dtype                    */

#define NORM_OPT_PRE 0x1   /* the join gives X = norm(R1)                      */
#define NORM_OPT_POST 0x2  /* the join takes the norm of B                     */
#define NORM_OPT_ACCUM 0x4 /* the backward adds to the parameters' gradients
                              what it finds there                              */

typedef struct norm_config {
    int32_t dim;      /* D, in [1, 4096]                                       */
    int32_t kind;     /* NORM_KIND_*                                           */
    int32_t x_dtype;  /* NORM_DTYPE_*; where it is F32, r_dtype is too         */
    int32_t r_dtype;
    int32_t p_dtype;
    int32_t dp_dtype;
    int32_t gate;     /* NORM_BY_*                                             */
    int32_t scale;    /* NORM_BY_*, not TOKEN                                  */
    int32_t options;  /* NORM_OPT_* bits                                       */
    float eps;        /* in [1e-12, 1]                                         */
} norm_config;

/* Host structs of device pointers.  NULL: absent (w, post_w: 1; b, post_b: 0).
 * gate and scale are given where the config names them. */
typedef struct norm_params {
    const void *post_w;
    const void *post_b;
    const void *gate;
    const void *scale;
    const void *w;
    const void *b;
} norm_params;

/* The gradients of norm_params; NULL: not wanted. */
typedef struct norm_grads {
    void *dpost_w;
    void *dpost_b;
    void *dgate;
    void *dscale;
    void *dw;
    void *db;
} norm_grads;

int norm_abi_version(void);
const char *norm_status_string(int status);

/* Validates a config on the host.  Returns NORM_OK or NORM_ECONFIG. */
int norm_config_check(const norm_config *cfg);

/* Bytes of workspace that the backward of cfg needs (host output `bytes`), whatever T
 * is: 10,248 (parts of the sums over t) times D rounded up to 4, rounded up to 256. */
int norm_workspace_bytes(const norm_config *cfg, uint64_t *bytes);

/* X = norm(R; w, b); the config's gate, scale and options are not looked at.
 * T = 0 enqueues nothing. */
int norm_fwd(const norm_config *cfg, const void *R, const void *w, const void *b, int64_t T, void *X, void *stream);

/* dR = dR1 + the gradient through the norm (dR1 may be NULL: 0; dR may be dR1,
 * whole); dw and db may be NULL.  T = 0 gives zero dw and db (with
 * NORM_OPT_ACCUM: leaves them alone). */
int norm_bwd(const norm_config *cfg, void *ws, uint64_t ws_bytes, const void *R, const void *dX, const void *dR1,
             const void *w, int64_t T, void *dR, void *dw, void *db, void *stream);

/* R1 may be R, whole.  X is left alone (and may be NULL) without NORM_OPT_PRE,
 * as post_w, post_b, w and b are where the config has no norm for them. */
int norm_join_fwd(const norm_config *cfg, const void *R, const void *B, const norm_params *p, int64_t T, void *R1,
                  void *X, void *stream);

/* R is read only for dscale (else it may be NULL); R1 and dX only with
 * NORM_OPT_PRE; dR1 may be NULL with it.  dR may be dR1, whole.  dgate of
 * NORM_BY_TOKEN is [T][D] and overwritten; the other gradients of g as above. */
int norm_join_bwd(const norm_config *cfg, void *ws, uint64_t ws_bytes, const void *R, const void *B, const void *R1,
                  const void *dX, const void *dR1, const norm_params *p, int64_t T, void *dR, void *dB,
                  const norm_grads *g, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NORM_H */
