// Internal types of the operators of a layer (include/ssd_layer.h).
#pragma once

#include "../../include/ssd_layer.h"
#include "mixer_internal.h"

namespace ssd {

// ---- gated delta rule --------------------------------------------------------------

constexpr int GD_CHUNK = 64;  // tokens per chunk

// A call of the gated delta rule.  Workspace arrays hold a row per (head, token), so that their size
// follows from the tokens, however these are packed; chunk states are kept by the tokens' place.
struct GdArgs {
    const void *q, *k, *v, *dout;             // token rows, act_dtype
    int64_t q_ts, k_ts, v_ts, o_ts;           // elements between tokens (o_ts: o and dout)
    const float *g, *beta;                    // [tokens] rows of H
    int64_t g_ts, b_ts;
    const int32_t* cu;                        // [nseq + 1] or null (rows of `seqlen` tokens)
    int nseq;
    int64_t seqlen, tokens;                   // tokens of a row, of all rows
    const float *init, *dfin;                 // [nseq][H][DV][DK] or null
    float *fin, *dinit;
    void *o, *dq, *dk, *dv;
    int64_t dq_ts, dk_ts, dv_ts;
    float *dg, *dbeta;                        // [tokens][H]
    int H, share, keydim, valdim;             // value heads, of which `share` read one key head
    float scale;
    // workspace
    void *T, *P;                              // [H][tokens][64 columns in parts], see GdMat
    float *in, *out, *beta_of;                // [H][tokens]: e^c, e^(C - c) (-1: see GdScalars), beta
    double* c2;                               // [H][tokens]: c in units of log 2 (backward)
    float *S, *G;                             // [place][H][DK][DV] states entering, gradients leaving
    float *U, *Z;                             // [H][tokens][DV]
    float* sums;                              // [H][tokens][2][DK], dq and dk of every head, or null
};
size_t gd_fwd_ws(const GdArgs& a, int act);
size_t gd_bwd_ws(const GdArgs& a, int act);
hipError_t launch_gd_fwd(GdArgs a, int act, void* ws, hipStream_t s);
hipError_t launch_gd_bwd(GdArgs a, int act, void* ws, hipStream_t s);

struct GdStep {
    const void *q, *k, *v;
    int64_t q_ts, k_ts, v_ts, o_ts, g_ts, b_ts;
    const float *g, *beta;
    const int32_t *slots, *positions;
    int64_t nslots;
    float* state;
    void* o;
    int rows, tokens, H, share, keydim, valdim;
    float scale;
};
hipError_t launch_gd_step(const GdStep& a, int act, hipStream_t s);

// ---- norms around a block ------------------------------------------------------------
struct BlockArgs {
    const void *x, *y, *z, *dr, *dh;
    const float *scale, *w1, *b1, *w2, *b2;  // 1: of the norm behind the block, 2: before the next
    void *r, *h, *dx, *dy, *dz;
    float *dscale, *dw1, *db1, *dw2, *db2;
    int64_t rows, xs, ys, zs, rs, hs, dxs, dys, dzs;
    int C, post, pre, gate, center;
    float alpha, eps;
};
constexpr int BLOCK_MAX_CHANNELS = 16384;
size_t block_bwd_ws(const BlockArgs& a);
hipError_t launch_block_fwd(const BlockArgs& a, int act, int res, hipStream_t s);
hipError_t launch_block_bwd(const BlockArgs& a, int act, int res, float* part, hipStream_t s);

// ---- rotary positions ------------------------------------------------------------------
struct RopeArgs {
    const void *q, *k;
    void *qo, *ko;
    int64_t qs, ks, qos, kos;
    const double* freq;
    const int32_t *positions, *cu;
    int nseq;
    int64_t seqlen, tokens;
    int H, K, D, R, style;
    float factor, turn;  // turn: 1 or -1
};
constexpr int ROPE_MAX_DIM = 1024;
hipError_t launch_rope(const RopeArgs& a, int act, hipStream_t s);

}  // namespace ssd
