/*
 * recur.h -- C ABI of a gated linear recurrence over packed sequences, forward,
 * backward, and its step for single tokens, for AMD Instinct MI355X (gfx950).
 * Built into the same libngram.so as ngram.h.
 *
 * Every channel j by itself, s(v) = 1 / (1 + exp(-v)), sp(v) = log(1 + exp(v)):
 *
 *   a_t = exp(-c sp(lam_j) s(r_t)),  u_t = sqrt(1 - a_t^2) s(i_t) x_t
 *   h_t = a_t h_{t-1} + u_t,  y_t = h_t
 *
 * h before the first position of a sequence is its row of h0, or 0.  Backwards,
 * with m_t = sqrt(1 - a_t^2), g_t = s(i_t), rho_t = s(r_t):
 *
 *   G_t = dy_t + a_{t+1} G_{t+1}  (behind the last position: its row of dhT, or 0)
 *   dx_t = G_t m_t g_t,  di_t = G_t m_t x_t g_t (1 - g_t)
 *   dz_t = a_t G_t h_{t-1} - G_t g_t x_t a_t^2 / m_t  (the second term 0 where m_t is)
 *   dr_t = -c sp(lam) dz_t rho_t (1 - rho_t),  dh0 = a_1 G_1
 *   dlam (+)= s(lam) sum_t -c rho_t dz_t
 *
 * x, r, i (and dx, dr, di): T rows of D values of the config's dtype, each with a
 * distance between rows of its own, so they may be columns of one projection's
 * result; y, dy: [T][D] of that dtype; lam, dlam: fp32 [D]; h0, hT, dhT, dh0: fp32
 * [n][D], a row a sequence; saved: what the backward needs of the forward beside
 * its inputs, a state for every RECUR_CHUNK positions.  All aligned to their
 * elements.
 *
 * Sequences: offsets (device, int32 [n + 1], ascending from >= 0 to <= T):
 * sequence k is rows offsets[k] .. offsets[k + 1] - 1; one without rows has hT =
 * h0 (or 0), dh0 = dhT (or 0).  Rows in front of the first and behind the last
 * sequence count for nothing, whatever they hold, and are left as they were in every
 * output.  offsets NULL: n has to be 1, and the sequence is all T rows.  Offsets that do not ascend give unspecified results,
 * but nothing outside the buffers is touched.  Nothing of one sequence reaches
 * another, NaN and infinities included; within a sequence a NaN stays.
 *
 * Precision: fp32 inside, states and sums over t too; a and 1 - a^2 keep their
 * relative precision for fast decays and for slow ones (an a or a gate below 2^-126
 * counts as 0); y, dx, dr and di are rounded once (bf16: nearest, ties to even).
 * The backward computes the gates and states again.
 *
 * Conventions: device pointers unless marked "host"; the caller owns every
 * buffer; calls only enqueue on `stream` (a hipStream_t, NULL = the null
 * stream), never allocate, free or synchronise, and may be captured in a HIP
 * graph; a negative return is a host-detected error with nothing enqueued.
 * The workspace holds nothing between calls: calls that share one must be
 * ordered (one stream), and graphs that were captured with the same one must
 * not run at the same time.  Results are the same, bit for bit, in every run of
 * the same call.  Blocks of a call wait for states of others that have begun before
 * them; a wait ends after 2^20 looks, over half a second, which takes a workspace that
 * something else writes meanwhile, and the values behind it are NaN then.
 */
#ifndef RECUR_H
#define RECUR_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RECUR_ABI_VERSION 1

#define RECUR_OK 0
#define RECUR_ENULL -1   /* a required pointer is NULL                         */
#define RECUR_EALIGN -2  /* a pointer is not aligned to its elements (workspace: 256) */
#define RECUR_ECONFIG -3 /* the config is invalid                              */
#define RECUR_ESIZE -4   /* T outside [0, max_tokens], n outside [0, 2^24] (1
                            without offsets), a distance between rows under D or
                            over 2^31 - 1, a workspace too small, or 2^23 and
                            more blocks: pieces of 32 (forward: 64) positions by
                            128 (D up to 64, backward of fp32: 64) channels    */
#define RECUR_EARG -5    /* an output that overlaps an operand or another output,
                            or an unknown pass                                 */
#define RECUR_EHIP -6    /* the HIP runtime reported an error                  */

#define RECUR_DTYPE_F32 0
#define RECUR_DTYPE_BF16 1

#define RECUR_OPT_ACCUM 0x1 /* the backward adds to dlam what it finds there   */

#define RECUR_PASS_FWD 0
#define RECUR_PASS_BWD 1

#define RECUR_CHUNK 32 /* positions to a saved state                           */

typedef struct recur_config {
    int32_t dim;        /* D, in [1, 16384]                                    */
    int32_t dtype;      /* RECUR_DTYPE_*                                       */
    float c;            /* in (0, 64]                                          */
    int32_t options;    /* RECUR_OPT_* bits                                    */
    int64_t max_tokens; /* largest T of any call, in [1, 2^24]                 */
} recur_config;

/* Host structs of device pointers; ld: elements from one row to the next. */
typedef struct recur_inputs {
    const void *x;
    const void *r;
    const void *i;
    int64_t ldx;
    int64_t ldr;
    int64_t ldi;
} recur_inputs;

typedef struct recur_grads {
    void *dx;
    void *dr;
    void *di;
    int64_t lddx;
    int64_t lddr;
    int64_t lddi;
} recur_grads;

int recur_abi_version(void);
const char *recur_status_string(int status);

/* Validates a config on the host.  Returns RECUR_OK or RECUR_ECONFIG. */
int recur_config_check(const recur_config *cfg);

/* Bytes of workspace that a pass of cfg needs (host output `bytes`); one of the
 * backward's size serves both.  With n pieces of 32 positions in max_tokens (forward:
 * of 64; a single one up to 128, forward 256) and E = D rounded up to 128:
 * 256 ceil(D / 64) + 8 E (n + floor(n / 16) + 1), and for the backward 4 D n, rounded
 * up to 256.  Of wide rows that is 2 / 5 D max_tokens bytes (forward: 1 / 7). */
int recur_workspace_bytes(const recur_config *cfg, int pass, uint64_t *bytes);

/* Bytes of `saved` for T positions: 4 D ceil(T / RECUR_CHUNK). */
int recur_saved_bytes(const recur_config *cfg, int64_t T, uint64_t *bytes);

/* Forward.  hT and saved may be NULL: not wanted. */
int recur_fwd(const recur_config *cfg, void *ws, uint64_t ws_bytes, const recur_inputs *in, const float *lam,
              const int32_t *offsets, int64_t n, const float *h0, int64_t T, void *y, float *hT, float *saved,
              void *stream);

/* Backward under the forward's inputs and its `saved`.  dhT and dh0 may be NULL;
 * dlam is overwritten unless RECUR_OPT_ACCUM.  T = 0 gives a zero dlam (with
 * RECUR_OPT_ACCUM: leaves it alone). */
int recur_bwd(const recur_config *cfg, void *ws, uint64_t ws_bytes, const recur_inputs *in, const float *lam,
              const int32_t *offsets, int64_t n, const float *h0, const float *saved, const void *dy,
              const float *dhT, int64_t T, const recur_grads *out, float *dlam, float *dh0, void *stream);

/* One position of each of n rows (single tokens of a serving loop): row k takes
 * state row slots[k] (slots NULL: row k, and `states` >= n), fp32 [states][D], one
 * position on, in place, and y gets its new values.  A row whose slot is negative
 * or not below `states` is unused: its y is 0.  Rows of the same slot are that
 * state's next positions, in the rows' order.  n in [0, 2^16]; T and max_tokens
 * do not count here.  With slots every row looks for its own among all n: from some
 * 2,000 rows on that costs the most and grows as n^2, and several calls of 1,000 to
 * 2,000 rows are faster than one (their order is that of the rows). */
int recur_step(const recur_config *cfg, const recur_inputs *in, const float *lam, float *state, int64_t states,
               const int32_t *slots, int64_t n, void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* RECUR_H */
