/*
 * ssd_layer.h - C ABI of more operators of a layer around a recurrent mixer (same library
 * and status codes as ssd.h, same conventions as ssd_mixer.h):
 *
 *   ssd_gdelta_*    the gated delta rule: a state with a decay and an update rate per token and
 *                   head; prompts (forward and backward) and single tokens.
 *   ssd_block_norm_* the norms before and after a block, with its gate and residual scale.
 *   ssd_rope        rotary positions of queries and keys, and their gradient.
 */
#ifndef MI355X_SSD_LAYER_H
#define MI355X_SSD_LAYER_H

#include "ssd_mixer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the gated delta rule --------------------------------------------------------
 *
 * Per sequence and head h, which reads query/key head h / (nheads / nkheads), with a_t =
 * exp(g_t):
 *   u_t = beta_t (v_t - a_t S_(t-1) k_t)
 *   S_t = a_t S_(t-1) + u_t k_t^T        [valdim][keydim], S before the first token: init, or zero
 *   o_t = scale S_t q_t
 * The state forgets by a_t and then replaces, by the rate beta_t, what it answers to k_t.  Keys
 * are taken as they are; a model makes them unit length before (ssd_norm_fwd with a group per
 * head and weights of keydim^-1/2 does).  g_t <= 0 is meant (minus infinity: nothing before t
 * is kept); larger values are not refused as long as the exponentials of their sums over 64 tokens
 * (of single tokens that of g_t / 2) stay within float32's range.  beta_t may be any value with which
 * u_t does.
 *
 * Sums, states and decays are float32 (sums of log decays float64) and bf16 outputs are rounded
 * once: a float32 value that meets another operand on its way to a float32 output (states, gate
 * gradients) is taken whole, to a bf16 output alone to 2^-18 of it.  (The states are on their way to a float32
 * output if a last state is asked for, so that the last bits of bf16 outputs may depend on that.)  A value of q, k, v,
 * g or beta that is not finite reaches no other sequence and no output before it; the outputs that
 * it reaches (of v: its channel's) and the last state are then not finite.  In the backward
 * it, or one of dout, may reach every gradient of its sequence. */
typedef struct {
    int64_t batch;      /* rows; 1 with cu_seqlens                               */
    int64_t seqlen;     /* tokens per row (with cu_seqlens: all tokens)          */
    int32_t nheads;     /* H, heads of v, g, beta, o and the states              */
    int32_t nkheads;    /* Hk, heads of q and k, H % Hk == 0                     */
    int32_t keydim;     /* 64 or 128                                             */
    int32_t valdim;     /* 64 or 128                                             */
    int32_t act_dtype;  /* ssd_dtype of q, k, v, o and their gradients           */
    float scale;        /* factor of the outputs                                 */
    /* elements between tokens, 0 = packed; multiples of 16 bytes but for g and beta, whose
     * rows are float32.  o_stride is that of o and of dout. */
    int64_t q_stride, k_stride, v_stride, o_stride, g_stride, beta_stride;
    int64_t dq_stride, dk_stride, dv_stride;
} ssd_gdelta;
/* Size limits (SSD_ERR_SHAPE beyond them): batch * seqlen <= 2^31 - 128 tokens,
 * nheads <= 65535, sequences <= 2^24, token strides below 2^22 elements, and every
 * launch grid within the hardware's limits. */

/* Bytes of workspace for the forward (SSD_WS_FORWARD) or backward (SSD_WS_BACKWARD)
 * of `nseq` sequences (rows, or packed in one row); 0 for an invalid problem, number or
 * kind.  It grows with the tokens, not with the sequences they are packed into.  `final_state`
 * of the forward makes no difference. */
size_t ssd_gdelta_workspace_bytes(const ssd_gdelta* problem, int32_t nseq, int32_t kind);

/* Prompts.
 *   q, k       [batch][seqlen][Hk][keydim]                                    (in)
 *   v          [batch][seqlen][H][valdim]                                     (in)
 *   g, beta    [batch][seqlen][H] float32                                     (in)
 *   cu_seqlens as for ssd_linattn_fwd                                         (in)
 *   init       [nseq][H][valdim][keydim] float32 or NULL (zero)               (in)
 *   o          [batch][seqlen][H][valdim]; tokens outside every sequence are
 *              left as they were                                              (out)
 *   final_state [nseq][H][valdim][keydim] float32 or NULL: the state after each
 *              sequence's last token (its init where it is empty); may be init itself (out)
 * No other output may share memory with an input. */
int ssd_gdelta_fwd(const ssd_gdelta* problem, int32_t nseq, const void* q, const void* k,
                   const void* v, const float* g, const float* beta, const int32_t* cu_seqlens,
                   const float* init, void* o, float* final_state, void* ws, size_t ws_bytes,
                   void* stream);

/* Gradients.  With G_t of the state behind token t (dfinal behind the last one, zero if NULL):
 *   D = G_t + scale dout_t q_t^T,  du = D k_t,  B = D - beta_t du k_t^T
 *   dq_t = scale S_t^T dout_t,  dv_t = beta_t du
 *   dk_t = D^T u_t - a_t S_(t-1)^T (beta_t du)       (dq, dk: summed over the heads that share them)
 *   dbeta_t = du . (v_t - a_t S_(t-1) k_t),  dg_t = <B, a_t S_(t-1)>
 *   G_(t-1) = a_t B,  dinit = G before the first token (dfinal where a sequence is empty)
 * The states are recomputed.  No output may share memory with an input.
 * dg_t is formed as a sum, over the tokens i from t to the end of a run of 64, of q_i . dq_i - v_i . dv_i, and of
 * <G, S> behind the run: it is good to some 2^-20 of these terms, which a strong decay at t does not make
 * smaller as it does dg_t (of e^g below 1e-6 little of dg_t is left).  Where e^(g_t) is zero in float32 dg_t is zero.
 *   dout       [batch][seqlen][H][valdim]                                      (in)
 *   dfinal     [nseq][H][valdim][keydim] float32 or NULL                       (in)
 *   dq, dk, dv as q, k, v; dg, dbeta [batch][seqlen][H] float32; tokens outside
 *              every sequence are left as they were                            (out)
 *   dinit      [nseq][H][valdim][keydim] float32 or NULL                       (out) */
int ssd_gdelta_bwd(const ssd_gdelta* problem, int32_t nseq, const void* q, const void* k,
                   const void* v, const float* g, const float* beta, const int32_t* cu_seqlens,
                   const void* dout, const float* init, const float* dfinal, void* dq, void* dk,
                   void* dv, float* dg, float* dbeta, float* dinit, void* ws, size_t ws_bytes,
                   void* stream);

/* Single tokens: `seqlen` new tokens (1, or a few) of `batch` rows, each row continuing the
 * state in its slot, which is updated in place; slots, nslots and positions as for
 * ssd_linattn_step.
 *   state      [nslots][H][valdim][keydim] float32                         (in/out)
 *   o          [batch][seqlen][H][valdim]                                      (out) */
int ssd_gdelta_step(const ssd_gdelta* problem, const void* q, const void* k, const void* v,
                    const float* g, const float* beta, const int32_t* slots, int64_t nslots,
                    const int32_t* positions, float* state, void* o, void* stream);

/* ---- norms around a block ---------------------------------------------------------
 *
 * Per row (token) of `channels`, with norm(u) = (u - m) / sqrt(mean((u - m)^2) + eps), m = mean(u)
 * if `center`, else 0; x the residual stream and y what the block gives:
 *   u = norm(y) post_weight + post_bias      (post; else y)
 *   m = u act(z)                             (a gate; else u)
 *   r = alpha x + scale m                    the residual stream behind the block
 *   h = norm(r) pre_weight + pre_bias        (pre) what the next block reads
 * All in float32; r and h are rounded once, and h is made of r before its rounding. */
typedef enum {
    SSD_GATE_NONE = 0,
    SSD_GATE_LINEAR = 1,   /* act(z) = z          */
    SSD_GATE_SIGMOID = 2,
    SSD_GATE_SILU = 3
} ssd_gate;
typedef struct {
    int64_t rows;
    int32_t channels;   /* up to 16384 (SSD_ERR_UNSUPPORTED beyond)               */
    int32_t act_dtype;  /* ssd_dtype of y, z, h and their gradients              */
    int32_t res_dtype;  /* ssd_dtype of x, r and their gradients: act_dtype's, or SSD_F32 */
    int32_t post, pre;  /* 0 or 1: the two norms                                 */
    int32_t gate;       /* ssd_gate                                              */
    int32_t center;     /* 0 or 1, of both norms                                 */
    float alpha, eps;   /* eps > 0                                               */
    /* elements between rows, 0 = packed; any value >= channels below 2^28, and tensors need be
     * aligned to their elements only.  r_stride is that of r and of dr, h_stride of h and dh. */
    int64_t x_stride, y_stride, z_stride, r_stride, h_stride, dx_stride, dy_stride, dz_stride;
} ssd_block;
/* Size limit (SSD_ERR_SHAPE beyond it): rows <= 2^31 - 1. */

/* x [rows][channels] res_dtype, y and z (a gate only) act_dtype, scale [channels] float32 or NULL (one),
 * post_weight and pre_weight [channels] float32 (their norms only), post_bias and pre_bias likewise or
 * NULL -> r, and h with `pre`.  r may be x itself, h may be y or z itself. */
int ssd_block_norm_fwd(const ssd_block* problem, const void* x, const void* y, const void* z,
                       const float* scale, const float* post_weight, const float* post_bias,
                       const float* pre_weight, const float* pre_bias, void* r, void* h, void* stream);

/* Bytes of workspace of ssd_block_norm_bwd; 0 for an invalid problem. */
size_t ssd_block_norm_workspace_bytes(const ssd_block* problem);

/* Gradients, with dr of r (NULL: zero; only with `pre`) and dh of h (with `pre`).  dx, dy and dz (a gate
 * only) [rows][channels]; dscale, dpost_*, dpre_* [channels] float32, summed over the rows; each of
 * these may be NULL.  dx may be x or dr itself, dy may be y or dh, dz may be z. */
int ssd_block_norm_bwd(const ssd_block* problem, const void* x, const void* y, const void* z,
                       const float* scale, const float* post_weight, const float* post_bias,
                       const float* pre_weight, const void* dr, const void* dh, void* dx, void* dy,
                       void* dz, float* dscale, float* dpost_weight, float* dpost_bias,
                       float* dpre_weight, float* dpre_bias, void* ws, size_t ws_bytes, void* stream);

/* ---- rotary positions --------------------------------------------------------------
 *
 * The first `rotdim` channels of every head are taken as rotdim / 2 pairs, pair i is turned by the
 * angle p frequencies[i] at position p and multiplied by `factor`; the others are copied:
 *   y1 = factor (x1 cos - x2 sin),  y2 = factor (x2 cos + x1 sin)
 * Pairs are channels (i, i + rotdim / 2) (SSD_ROPE_HALF) or (2 i, 2 i + 1) (SSD_ROPE_INTERLEAVED).
 * Frequencies that stretch a model to longer contexts are the caller's to choose; angles are formed
 * in float64, so that far positions lose nothing. */
typedef enum { SSD_ROPE_HALF = 0, SSD_ROPE_INTERLEAVED = 1 } ssd_rope_style;
typedef struct {
    int64_t batch, seqlen;
    int32_t nheads, nkheads;  /* heads of q and of k; 0 of k: none                */
    int32_t headdim;          /* up to 1024 (SSD_ERR_UNSUPPORTED beyond)          */
    int32_t rotdim;           /* even, 2 .. headdim                               */
    int32_t act_dtype;        /* ssd_dtype of all                                 */
    int32_t style;            /* ssd_rope_style                                   */
    float factor;
    /* elements between tokens, 0 = packed, below 2^28; the tensors need be aligned to their
     * elements only */
    int64_t q_stride, k_stride, qo_stride, ko_stride;
} ssd_rope_problem;
/* Size limits (SSD_ERR_SHAPE beyond them): batch * seqlen <= 2^31 - 128 tokens, heads <= 65535. */

/*   q [batch][seqlen][nheads][headdim], k [batch][seqlen][nkheads][headdim] (in)
 *   frequencies [rotdim / 2] float64, radians per position                  (in)
 *   positions  [batch][seqlen] int32, of any sign, or NULL: a token's place in its row, or in its
 *              sequence where cu_seqlens is given                           (in)
 *   cu_seqlens [nseq + 1] int32 or NULL, as for ssd_linattn_fwd: tokens outside every
 *              sequence are left as they were                               (in)
 *   inverse    0, or 1: turned back by the same angles (and multiplied by `factor`), which takes
 *              gradients of the outputs to those of the inputs
 *   q_out, k_out as q, k; they may be q and k themselves                    (out) */
int ssd_rope(const ssd_rope_problem* problem, const void* q, const void* k, const double* frequencies,
             const int32_t* positions, const int32_t* cu_seqlens, int32_t nseq, int32_t inverse,
             void* q_out, void* k_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MI355X_SSD_LAYER_H */
