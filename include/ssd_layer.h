/*
 * ssd_layer.h - C ABI of more operators of a layer around a recurrent mixer (same library
 * and status codes as ssd.h, same conventions as ssd_mixer.h):
 *
 *   ssd_gdelta_*    the gated delta rule: a state with a decay and an update rate per token and
 *                   head; prompts (forward and backward) and single tokens.
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
 * stay within float32's range.  beta_t may be any value.
 *
 * Sums, states and decays are float32 (sums of log decays float64) and bf16 outputs are rounded
 * once: a float32 value that meets another operand on its way to a float32 output (states, gate
 * gradients) is taken in parts good to 2^-24, to a bf16 output alone to 2^-16.  A value of q, k, v,
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
 *              sequence's last token (its init where it is empty)             (out) */
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
 * The states are recomputed.
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

#ifdef __cplusplus
}
#endif

#endif /* MI355X_SSD_LAYER_H */
