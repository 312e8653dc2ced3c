/*
 * ssd_mixer.h - C ABI of the operators that stand around the SSD scan in a mixer
 * (same library, conventions and status codes as ssd.h):
 *
 *   ssd_linattn_*   linear attention with a fixed decay per head: prompts (forward
 *                   and backward) and single tokens.  The scan of ssd.h takes its
 *                   decays from dt and B, C shared by a group; this one takes q, k, v
 *                   and one decay per head, and sequences of any length.
 *   ssd_token_step  the single-token form of the whole conv1d + SSD path of ssd.h:
 *                   it continues from the forward's final state, token by token.
 *   ssd_norm_*      the group norm with an activation over a mixer's output,
 *                   channels last, forward and backward.
 *
 * Conventions beyond ssd.h's
 *  - Token arrays may be views whose tokens are further apart than packed rows
 *    (a slice of a projection's output): strides are in elements between tokens,
 *    0 means packed; the channels of a token are contiguous, and rows of a batch
 *    follow each other at seqlen times the token stride.
 *  - Nothing is written behind the last sequence, nor for a skipped row.
 *  - Outputs do not overlap inputs or each other, except where an entry point says so.
 *  - Results do not depend on the order in which workgroups run: every sum has a
 *    fixed order, no floating-point atomics.
 *  - No call keeps anything for the next one; a workspace is only used between the
 *    launches of one call, so calls that may overlap need a workspace each.
 */
#ifndef MI355X_SSD_MIXER_H
#define MI355X_SSD_MIXER_H

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- linear attention with a decay per head -------------------------------------
 *
 * Per sequence and head h, with l = exp(log_decay[h]) and head h reading key/value
 * head h / (nheads / nkvheads):
 *   S_t = l S_(t-1) + v_t k_t^T          [valdim][keydim], S before the first token:
 *                                        init, or zero
 *   o_t = scale S_t q_t
 * log_decay <= 0 is meant (minus infinity: every token sees itself alone); larger
 * values are not refused, the state then grows without bound (a power of a decay beyond
 * float32's range counts as its largest value).  The decays are constants of the model:
 * the backward gives no gradient for them.
 *
 * Sums, states and decays are float32, and bf16 outputs are rounded once: where a float32
 * value meets a bf16 one in a product it is taken in parts, good to 2^-16 (scores, states
 * that enter an output), 2^-24 (values on their way into a state) or, where no state is
 * asked for, 2^-17.  A value of q, k, v or do that is not finite reaches no other sequence
 * and no output before it (backwards: behind it); its channel's states and later outputs
 * are then not finite. */
typedef struct {
    int64_t batch;      /* rows; 1 with cu_seqlens                               */
    int64_t seqlen;     /* tokens per row (with cu_seqlens: all tokens)          */
    int32_t nheads;     /* H, query heads                                        */
    int32_t nkvheads;   /* key/value heads, H % nkvheads == 0                    */
    int32_t keydim;     /* 64 or 128                                             */
    int32_t valdim;     /* 64 or 128                                             */
    int32_t act_dtype;  /* ssd_dtype of q, k, v, o and their gradients           */
    float scale;        /* factor of the outputs                                 */
    /* elements between tokens, 0 = packed; multiples of 16 bytes.  o_stride is
     * that of o and of do. */
    int64_t q_stride, k_stride, v_stride, o_stride;
    int64_t dq_stride, dk_stride, dv_stride;
} ssd_linattn;
/* Size limits (SSD_ERR_SHAPE beyond them): batch * seqlen <= 2^31 - 128 tokens,
 * nheads <= 65535, sequences <= 2^24, token strides below 2^23 elements, and every
 * launch grid within the hardware's limits. */

/* Bytes of workspace for the forward (SSD_WS_FORWARD) or backward (SSD_WS_BACKWARD)
 * of `nseq` sequences (rows, or packed in one row); 0 for an invalid problem, number or
 * kind.  It is bounded by the tokens, however many sequences they are packed into: a
 * float32 state per head for 256 tokens or more (three in the backward), and in the
 * backward dv and dk per head in float32 where heads share keys and values. */
size_t ssd_linattn_workspace_bytes(const ssd_linattn* problem, int32_t nseq, int32_t kind);

/* Prompts.
 *   q          [batch][seqlen][H][keydim]                                     (in)
 *   k, v       [batch][seqlen][nkvheads][keydim or valdim]                    (in)
 *   log_decay  [H] float32                                                    (in)
 *   cu_seqlens [nseq + 1] int32, non-decreasing from >= 0 to <= seqlen: sequence s is
 *              the tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (none if equal);
 *              needs batch 1.  NULL: every row is a sequence, nseq == batch   (in)
 *   init       [nseq][H][valdim][keydim] float32 or NULL (zero)               (in)
 *   o          [batch][seqlen][H][valdim]; tokens outside every sequence are
 *              left as they were                                              (out)
 *   final_state [nseq][H][valdim][keydim] float32 or NULL: the state after each
 *              sequence's last token (its init where it is empty)             (out) */
int ssd_linattn_fwd(const ssd_linattn* problem, int32_t nseq, const void* q, const void* k,
                    const void* v, const float* log_decay, const int32_t* cu_seqlens,
                    const float* init, void* o, float* final_state, void* ws, size_t ws_bytes,
                    void* stream);

/* Gradients.  With G_t = scale do_t q_t^T + l G_(t+1), G behind the last token being
 * dfinal without a decay (zero if NULL):
 *   dq_t = scale S_t^T do_t,  dv_t = G_t k_t,  dk_t = G_t^T v_t  (summed over the
 *   heads that share k and v),  dinit = l G_first (dfinal where a sequence is empty).
 * The states are recomputed from k, v and init.
 *   do         [batch][seqlen][H][valdim]                                      (in)
 *   dfinal     [nseq][H][valdim][keydim] float32 or NULL                       (in)
 *   dq, dk, dv as q, k, v; tokens outside every sequence are left as they were (out)
 *   dinit      [nseq][H][valdim][keydim] float32 or NULL                       (out) */
int ssd_linattn_bwd(const ssd_linattn* problem, int32_t nseq, const void* q, const void* k,
                    const void* v, const float* log_decay, const int32_t* cu_seqlens,
                    const void* dout, const float* init, const float* dfinal, void* dq, void* dk,
                    void* dv, float* dinit, void* ws, size_t ws_bytes, void* stream);

/* Single tokens: `seqlen` new tokens (1, or a few) of `batch` rows, each row continuing
 * the state in its slot, which is updated in place.
 *   q, k, v, log_decay   as for ssd_linattn_fwd                                 (in)
 *   slots      [batch] int32 or NULL (row r uses slot r; nslots >= batch).  A row
 *              whose slot is outside [0, nslots) is padding: it is skipped and its
 *              outputs are left as they were.  Of several rows with one slot the first
 *              is computed and the others are skipped                          (in)
 *   positions  [batch] int32 or NULL: the place of the row's first new token in its
 *              sequence.  At 0 the state starts from zero, whatever the slot holds; a
 *              negative place skips the row                                    (in)
 *   state      [nslots][H][valdim][keydim] float32                         (in/out)
 *   o          [batch][seqlen][H][valdim]                                      (out) */
int ssd_linattn_step(const ssd_linattn* problem, const void* q, const void* k, const void* v,
                     const float* log_decay, const int32_t* slots, int64_t nslots,
                     const int32_t* positions, float* state, void* o, void* stream);

/* ---- the conv1d + SSD path, token by token ---------------------------------------
 *
 * `problem` as in ssd.h (batch = rows, seqlen = new tokens per row, chunk not used): one
 * call does for every row what ssd_conv1d_fwd, the scan and D x do for its tokens, the
 * convolved channels kept in float32.  The last inputs stand in a ring: the xBC row of a
 * sequence's token t is entry t mod ring_len, so nothing moves.
 *   xBC       [batch][seqlen][C] act_dtype, the new tokens                      (in)
 *   conv_w, dt_raw [batch][seqlen][H], dt_bias, A_log, D   as in ssd.h          (in)
 *   slots, nslots   as for ssd_linattn_step                                     (in)
 *   positions [batch] int32: the place of the row's first new token in its sequence;
 *             taps before place 0 are zero, and at 0 the state starts from zero; a
 *             negative place skips the row                                      (in)
 *   conv_ring [nslots][ring_len][C] act_dtype, ring_len >= conv_width - 1 + seqlen:
 *             entries of the conv_width - 1 tokens before `positions` are read, those
 *             of the new tokens written                                     (in/out)
 *   state     [nslots][H][P][N] float32                                     (in/out)
 *   y         [batch][seqlen][H][P] act_dtype                                   (out)
 * The state is aligned to 16 bytes, the other tensors need be to their elements only. */
int ssd_token_step(const ssd_problem* problem, const void* xBC, const float* conv_w,
                   const void* dt_raw, const float* dt_bias, const float* A_log, const float* D,
                   const int32_t* slots, int64_t nslots, const int32_t* positions, void* conv_ring,
                   int32_t ring_len, float* state, void* y, void* stream);

/* ---- group norm with an activation, channels last ---------------------------------
 *
 * Per row (token) and group of channels / ngroups neighbouring channels:
 *   norm(u) = (u - m) / sqrt(mean((u - m)^2) + eps), m = mean(u) if `center`, else 0
 *   SSD_NORM_NONE    y = norm(x) w + b
 *   SSD_NORM_SILU    y = silu(norm(x) w + b)
 *   SSD_NORM_BEFORE  y = norm(x silu(z)) w + b       (gated before the norm)
 *   SSD_NORM_AFTER   y = (norm(x) w + b) silu(z)     (gated after it)
 * The statistics never cross tokens: they would let a causal model read its future. */
typedef enum {
    SSD_NORM_NONE = 0,
    SSD_NORM_SILU = 1,
    SSD_NORM_BEFORE = 2,
    SSD_NORM_AFTER = 3
} ssd_norm_mode;
typedef struct {
    int64_t rows;
    int32_t channels;   /* channels % ngroups == 0                               */
    int32_t ngroups;
    int32_t act_dtype;  /* ssd_dtype of x, z, y and their gradients              */
    int32_t mode;       /* ssd_norm_mode                                         */
    int32_t center;     /* 0 or 1                                                */
    float eps;          /* > 0                                                   */
    /* elements between rows, 0 = packed; any value >= channels, and tensors need be
     * aligned to their elements only.  y_stride is that of y and of dy. */
    int64_t x_stride, z_stride, y_stride, dx_stride, dz_stride;
} ssd_norm;
/* Size limits (SSD_ERR_SHAPE beyond them): rows <= 2^31 - 1, channels <= 2^20, rows *
 * ngroups <= 2^31 - 1. */

/* x [rows][channels], z (gated modes only) likewise, weight [channels] float32, bias
 * [channels] float32 or NULL -> y [rows][channels].  y may be x or z itself. */
int ssd_norm_fwd(const ssd_norm* problem, const void* x, const void* z, const float* weight,
                 const float* bias, void* y, void* stream);

/* Bytes of workspace of ssd_norm_bwd; 0 for an invalid problem. */
size_t ssd_norm_workspace_bytes(const ssd_norm* problem);

/* dx, dz (gated modes only) [rows][channels]; dweight, dbias [channels] float32, summed
 * over the rows; dbias may be NULL.  dx and dz may be x, z or dy themselves. */
int ssd_norm_bwd(const ssd_norm* problem, const void* x, const void* z, const float* weight,
                 const float* bias, const void* dy, void* dx, void* dz, float* dweight,
                 float* dbias, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MI355X_SSD_MIXER_H */
