/*
 * ffn.h -- C ABI of the gated feed-forward block, forward and backward, for
 * AMD Instinct MI355X (gfx950).  Built into the same libngram.so as ngram.h.
 *
 *   G = X Wg^T,  U = X Wu^T,  H = a(G) * U            ([T][F])
 *   Y = (res +) dropout(H Wd^T)                        ([T][768])
 *
 *   dY' = dropout(dY)  (the same mask),  dH = dY' Wd
 *   dU = dH * a(G),  dG = dH * U * a'(G)
 *   dX = dG Wg + dU Wu,  dWg (+)= dG^T X,  dWu (+)= dU^T X,  dWd (+)= dY'^T H
 *   (the gradient of res is dY)
 *
 * X: bf16 [T][768]; Wg, Wu: bf16 [F][768]; Wd: bf16 [768][F]; res, Y, dY, dX
 * of y_dtype, [T][768]; dWg, dWu, dWd shaped as their weights, of dw_dtype.
 * All row-major and contiguous.
 *
 * Precision: products of bf16 values on the matrix cores, summed in fp32;
 * the activation and its derivative in fp32 from the fp32 sums.  Rounded to
 * bf16 (nearest, ties to even) on the way, each once and only because it is an
 * operand of a further product: H, dG and dU, and dY where it is fp32.  Each
 * makes a result's error about sqrt(2) times that of its own rounding; calls of
 * at most 64 positions and T F <= 8192, where a call's error strays far from that
 * average, keep 16 bits of H, dG and dU (not of an fp32 dY), as two bf16 values.
 * So a position's result may differ in its last bits with the number of
 * positions in its call.  The
 * scale of the dropout is applied to fp32 sums.  Y, dX and the weights'
 * gradients are rounded once, at the end.  The backward computes G and U
 * again from X: the forward keeps nothing, which saves 4 T F bytes of
 * activations and the two roundings that keeping them in bf16 would put on
 * every gradient, for a third more matrix work.
 *
 * Conventions: device pointers unless marked "host"; the caller owns every
 * buffer; ffn_fwd and ffn_bwd only enqueue on `stream` (a hipStream_t, NULL =
 * the null stream), never allocate, free or synchronise, and may be captured
 * in a HIP graph; a negative return is a host-detected error with nothing
 * enqueued.  16-byte aligned buffers.  The workspace holds nothing between
 * calls: calls that share one must be ordered (one stream), and graphs that
 * were captured with the same one must not run at the same time.  Results are
 * the same, bit for bit, in every run of the same call.
 */
#ifndef FFN_H
#define FFN_H

#include <stdint.h>

#include "drop.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FFN_ABI_VERSION 1

#define FFN_OK 0
#define FFN_ENULL -1   /* a required pointer is NULL                           */
#define FFN_EALIGN -2  /* a pointer is not 16-byte (workspace: 256-byte) aligned */
#define FFN_ECONFIG -3 /* the config is invalid                                */
#define FFN_ESIZE -4   /* T outside [0, max_tokens] or a workspace too small   */
#define FFN_EARG -5    /* a bad drop_spec, an output that overlaps an operand
                          (res may be Y, whole), or an unknown pass            */
#define FFN_EHIP -6    /* the HIP runtime reported an error                    */

#define FFN_ACT_SILU 0  /* a(g) = g / (1 + exp(-g))                            */
#define FFN_ACT_GELU 1  /* a(g) = g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) */
#define FFN_ACT_RELU2 2 /* a(g) = max(g, 0)^2                                  */

#define FFN_DTYPE_F32 0
#define FFN_DTYPE_BF16 1

#define FFN_OPT_ACCUM 0x1 /* the backward adds to dWg, dWu, dWd what it finds
                             there (micro-steps of an accumulation window)    */

#define FFN_PASS_FWD 0
#define FFN_PASS_BWD 1

typedef struct ffn_config {
    int32_t dim;        /* D: must be 768                                      */
    int32_t hidden;     /* F: a multiple of 8 in [8, 65536]                    */
    int32_t act;        /* FFN_ACT_*                                           */
    int32_t y_dtype;    /* FFN_DTYPE_* of res, Y, dY and dX                    */
    int32_t dw_dtype;   /* FFN_DTYPE_* of the weights' gradients               */
    int32_t options;    /* FFN_OPT_* bits                                      */
    int64_t max_tokens; /* largest T of any call, in [1, 2^24]                 */
} ffn_config;

int ffn_abi_version(void);
const char *ffn_status_string(int status);

/* Validates a config on the host.  Returns FFN_OK or FFN_ECONFIG. */
int ffn_config_check(const ffn_config *cfg);

/* Bytes of workspace that a pass of cfg needs (host output `bytes`); one of
 * the backward's size serves both.  About 2 T F bytes for the forward and
 * 6 T F + 1536 T for the backward, T the config's max_tokens, and room for parts
 * of k: 49,152 T, at most 33.6 MB; in the backward, where it is more and T is
 * over 64, 9,216 F for each 64 of T, at most 73,728 F. */
int ffn_workspace_bytes(const ffn_config *cfg, int pass, uint64_t *bytes);

/* Forward.  ws: ws_bytes bytes, at least what FFN_PASS_FWD needs, 256-byte
 * aligned; res (may be NULL) may be Y; drop (host, may be NULL: keep all): the
 * mask of a [T][768] tensor.  T = 0 enqueues nothing. */
int ffn_fwd(const ffn_config *cfg, void *ws, uint64_t ws_bytes, const void *X, const void *Wg, const void *Wu,
            const void *Wd, const void *res, const drop_spec *drop, int64_t T, void *Y, void *stream);

/* Backward under the forward's inputs and drop_spec; dX is overwritten, the
 * weights' gradients too unless FFN_OPT_ACCUM.  T = 0 leaves dX alone and
 * gives zero weight gradients (with FFN_OPT_ACCUM: leaves them alone). */
int ffn_bwd(const ffn_config *cfg, void *ws, uint64_t ws_bytes, const void *X, const void *Wg, const void *Wu,
            const void *Wd, const void *dY, const drop_spec *drop, int64_t T, void *dX, void *dWg, void *dWu,
            void *dWd, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FFN_H */
