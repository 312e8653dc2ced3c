// Host side of the C ABI declared in include/ssd_layer.h: argument validation and kernel
// dispatch.  As in ssd_api.cpp, every check runs before anything is enqueued.
#include <algorithm>
#include <climits>
#include <hip/hip_runtime.h>

#include "layer_internal.h"

using namespace ssd;

namespace {

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

// Workgroups of a one-dimensional launch of up to 512 threads: at most 2^32 - 1 work-items.
constexpr int64_t MAX_BLOCKS = 0xffffffffll / 512;

// ---- gated delta rule ----------------------------------------------------------------

// Sizes and strides of a call, in `a`.
int check_gdelta(const ssd_gdelta* p, GdArgs* a) {
    if (!p) return SSD_ERR_NULL;
    if (p->batch < 1 || p->seqlen < 1 || p->nheads < 1 || p->nkheads < 1 || p->keydim < 1 ||
        p->valdim < 1)
        return SSD_ERR_SHAPE;
    if (p->nheads % p->nkheads != 0 || p->nheads > 65535) return SSD_ERR_SHAPE;
    if (p->act_dtype != SSD_F32 && p->act_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    for (int d : {p->keydim, p->valdim})
        if (d != 64 && d != 128) return SSD_ERR_UNSUPPORTED;
    if (p->batch > INT32_MAX || p->seqlen > INT32_MAX || p->batch * p->seqlen > INT32_MAX - 127)
        return SSD_ERR_SHAPE;
    const int64_t esz = p->act_dtype == SSD_BF16 ? 2 : 4;
    auto stride = [](int64_t given, int64_t packed, int64_t bytes, int64_t unit, int64_t* out) {
        *out = given == 0 ? packed : given;
        if (*out < packed || *out >= (1ll << 22)) return (int)SSD_ERR_SHAPE;
        return *out * bytes % unit == 0 ? (int)SSD_OK : (int)SSD_ERR_ALIGN;
    };
    const int64_t H = p->nheads, K = p->nkheads, Dk = p->keydim, Dv = p->valdim;
    int rc;
    if ((rc = stride(p->q_stride, K * Dk, esz, 16, &a->q_ts))) return rc;
    if ((rc = stride(p->k_stride, K * Dk, esz, 16, &a->k_ts))) return rc;
    if ((rc = stride(p->v_stride, H * Dv, esz, 16, &a->v_ts))) return rc;
    if ((rc = stride(p->o_stride, H * Dv, esz, 16, &a->o_ts))) return rc;
    if ((rc = stride(p->g_stride, H, 4, 4, &a->g_ts))) return rc;
    if ((rc = stride(p->beta_stride, H, 4, 4, &a->b_ts))) return rc;
    if ((rc = stride(p->dq_stride, K * Dk, esz, 16, &a->dq_ts))) return rc;
    if ((rc = stride(p->dk_stride, K * Dk, esz, 16, &a->dk_ts))) return rc;
    if ((rc = stride(p->dv_stride, H * Dv, esz, 16, &a->dv_ts))) return rc;
    a->seqlen = p->seqlen;
    a->tokens = p->batch * p->seqlen;
    a->H = p->nheads;
    a->share = p->nheads / p->nkheads;
    a->keydim = p->keydim, a->valdim = p->valdim;
    a->scale = p->scale;
    return SSD_OK;
}

// nseq sequences, and launches that a grid holds: a workgroup per (chunk, head), and two per
// (sequence, head), rounded up to one of 8 XCDs.
int check_gdelta_sequences(const ssd_gdelta* p, int32_t nseq, const int32_t* cu, GdArgs* a) {
    if (nseq < 1 || nseq > (1 << 24)) return SSD_ERR_SEGMENTS;
    if (cu ? p->batch != 1 : nseq != p->batch) return SSD_ERR_SEGMENTS;
    typedef unsigned __int128 u128;
    const u128 chunks = (u128)(p->batch * p->seqlen) / GD_CHUNK + nseq;
    const u128 blocks = (chunks > 2 * (u128)nseq + 16 ? chunks : 2 * (u128)nseq + 16) * p->nheads;
    if (blocks > (u128)MAX_BLOCKS) return SSD_ERR_SHAPE;
    a->cu = cu;
    a->nseq = nseq;
    return SSD_OK;
}

// ---- norms around a block --------------------------------------------------------------

int check_block(const ssd_block* p, BlockArgs* a) {
    if (!p) return SSD_ERR_NULL;
    if (p->rows < 1 || p->rows > INT32_MAX || p->channels < 1) return SSD_ERR_SHAPE;
    if (p->channels > BLOCK_MAX_CHANNELS) return SSD_ERR_UNSUPPORTED;
    if (p->act_dtype != SSD_F32 && p->act_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (p->res_dtype != SSD_F32 && p->res_dtype != p->act_dtype) return SSD_ERR_UNSUPPORTED;
    if (p->gate < SSD_GATE_NONE || p->gate > SSD_GATE_SILU) return SSD_ERR_UNSUPPORTED;
    for (int f : {p->post, p->pre, p->center})
        if (f != 0 && f != 1) return SSD_ERR_SHAPE;
    if (!(p->eps > 0.f) || !(p->eps < 1e30f)) return SSD_ERR_SHAPE;
    const int64_t given[] = {p->x_stride, p->y_stride, p->z_stride, p->r_stride,
                             p->h_stride, p->dx_stride, p->dy_stride, p->dz_stride};
    int64_t* out[] = {&a->xs, &a->ys, &a->zs, &a->rs, &a->hs, &a->dxs, &a->dys, &a->dzs};
    for (int i = 0; i < 8; ++i) {
        *out[i] = given[i] == 0 ? p->channels : given[i];
        if (*out[i] < p->channels || *out[i] >= (1ll << 28)) return SSD_ERR_SHAPE;
    }
    a->rows = p->rows;
    a->C = p->channels;
    a->post = p->post, a->pre = p->pre, a->gate = p->gate, a->center = p->center;
    a->alpha = p->alpha, a->eps = p->eps;
    return SSD_OK;
}
unsigned bytes_of(int32_t dtype) { return dtype == SSD_BF16 ? 2 : 4; }

// ---- rotary positions --------------------------------------------------------------------

int check_rope(const ssd_rope_problem* p, RopeArgs* a) {
    if (!p) return SSD_ERR_NULL;
    if (p->batch < 1 || p->seqlen < 1 || p->nheads < 1 || p->nkheads < 0 || p->headdim < 1)
        return SSD_ERR_SHAPE;
    if (p->nheads > 65535 || p->nkheads > 65535) return SSD_ERR_SHAPE;
    if (p->headdim > ROPE_MAX_DIM) return SSD_ERR_UNSUPPORTED;
    if (p->rotdim < 2 || p->rotdim > p->headdim || p->rotdim % 2 != 0) return SSD_ERR_SHAPE;
    if (p->act_dtype != SSD_F32 && p->act_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (p->style != SSD_ROPE_HALF && p->style != SSD_ROPE_INTERLEAVED) return SSD_ERR_UNSUPPORTED;
    if (p->batch > INT32_MAX || p->seqlen > INT32_MAX || p->batch * p->seqlen > INT32_MAX - 127)
        return SSD_ERR_SHAPE;
    const int64_t H = p->nheads, K = p->nkheads, D = p->headdim;
    const int64_t given[] = {p->q_stride, p->k_stride, p->qo_stride, p->ko_stride};
    const int64_t packed[] = {H * D, K * D, H * D, K * D};
    int64_t* out[] = {&a->qs, &a->ks, &a->qos, &a->kos};
    for (int i = 0; i < 4; ++i) {
        *out[i] = given[i] == 0 ? packed[i] : given[i];
        if (*out[i] < packed[i] || *out[i] >= (1ll << 28)) return SSD_ERR_SHAPE;
    }
    a->seqlen = p->seqlen;
    a->tokens = p->batch * p->seqlen;
    a->H = p->nheads, a->K = p->nkheads, a->D = p->headdim, a->R = p->rotdim, a->style = p->style;
    a->factor = p->factor;
    return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_gdelta_workspace_bytes(const ssd_gdelta* problem, int32_t nseq, int32_t kind) {
    GdArgs a = {};
    if (check_gdelta(problem, &a) != SSD_OK) return 0;
    if (kind != SSD_WS_FORWARD && kind != SSD_WS_BACKWARD) return 0;
    // rows or packed sequences, whichever needs more (one row may be either)
    const int32_t packed = 0;
    size_t n = 0;
    for (const int32_t* cu : {(const int32_t*)nullptr, &packed})
        if (check_gdelta_sequences(problem, nseq, cu, &a) == SSD_OK)
            n = std::max(n, kind == SSD_WS_FORWARD ? gd_fwd_ws(a, problem->act_dtype)
                                                   : gd_bwd_ws(a, problem->act_dtype));
    return n;
}

int ssd_gdelta_fwd(const ssd_gdelta* problem, int32_t nseq, const void* q, const void* k,
                   const void* v, const float* g, const float* beta, const int32_t* cu_seqlens,
                   const float* init, void* o, float* final_state, void* ws, size_t ws_bytes,
                   void* stream) {
    GdArgs a = {};
    int rc = check_gdelta(problem, &a);
    if (rc) return rc;
    if ((rc = check_gdelta_sequences(problem, nseq, cu_seqlens, &a))) return rc;
    if (!q || !k || !v || !g || !beta || !o) return SSD_ERR_NULL;
    if (!ws || ws_bytes < gd_fwd_ws(a, problem->act_dtype)) return SSD_ERR_WORKSPACE;
    for (const void* x : {q, k, v, (const void*)init, (const void*)o, (const void*)final_state,
                          (const void*)ws})
        if (!aligned(x, 16)) return SSD_ERR_ALIGN;
    for (const void* x : {(const void*)g, (const void*)beta, (const void*)cu_seqlens})
        if (!aligned(x, 4)) return SSD_ERR_ALIGN;
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta;
    a.init = init, a.fin = final_state, a.o = o;
    return hip_status(launch_gd_fwd(a, problem->act_dtype, ws, (hipStream_t)stream));
}

int ssd_gdelta_bwd(const ssd_gdelta* problem, int32_t nseq, const void* q, const void* k,
                   const void* v, const float* g, const float* beta, const int32_t* cu_seqlens,
                   const void* dout, const float* init, const float* dfinal, void* dq, void* dk,
                   void* dv, float* dg, float* dbeta, float* dinit, void* ws, size_t ws_bytes,
                   void* stream) {
    GdArgs a = {};
    int rc = check_gdelta(problem, &a);
    if (rc) return rc;
    if ((rc = check_gdelta_sequences(problem, nseq, cu_seqlens, &a))) return rc;
    if (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta) return SSD_ERR_NULL;
    if (!ws || ws_bytes < gd_bwd_ws(a, problem->act_dtype)) return SSD_ERR_WORKSPACE;
    for (const void* x : {q, k, v, dout, (const void*)init, (const void*)dfinal, (const void*)dq,
                          (const void*)dk, (const void*)dv, (const void*)dinit, (const void*)ws})
        if (!aligned(x, 16)) return SSD_ERR_ALIGN;
    for (const void* x : {(const void*)g, (const void*)beta, (const void*)cu_seqlens, (const void*)dg,
                          (const void*)dbeta})
        if (!aligned(x, 4)) return SSD_ERR_ALIGN;
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.dout = dout;
    a.init = init, a.dfin = dfinal, a.dinit = dinit;
    a.dq = dq, a.dk = dk, a.dv = dv, a.dg = dg, a.dbeta = dbeta;
    return hip_status(launch_gd_bwd(a, problem->act_dtype, ws, (hipStream_t)stream));
}

int ssd_gdelta_step(const ssd_gdelta* problem, const void* q, const void* k, const void* v,
                    const float* g, const float* beta, const int32_t* slots, int64_t nslots,
                    const int32_t* positions, float* state, void* o, void* stream) {
    GdArgs c = {};
    const int rc = check_gdelta(problem, &c);
    if (rc) return rc;
    if (nslots < 1 || (!slots && nslots < problem->batch)) return SSD_ERR_SHAPE;
    if (problem->batch * problem->nheads > MAX_BLOCKS / 2) return SSD_ERR_SHAPE;
    if (!q || !k || !v || !g || !beta || !state || !o) return SSD_ERR_NULL;
    for (const void* x : {q, k, v, (const void*)state, (const void*)o})
        if (!aligned(x, 16)) return SSD_ERR_ALIGN;
    for (const void* x : {(const void*)g, (const void*)beta, (const void*)slots, (const void*)positions})
        if (!aligned(x, 4)) return SSD_ERR_ALIGN;
    GdStep a = {};
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.o = o;
    a.q_ts = c.q_ts, a.k_ts = c.k_ts, a.v_ts = c.v_ts, a.o_ts = c.o_ts;
    a.g_ts = c.g_ts, a.b_ts = c.b_ts;
    a.slots = slots, a.positions = positions, a.nslots = nslots;
    a.state = state;
    a.rows = (int)problem->batch, a.tokens = (int)problem->seqlen;
    a.H = c.H, a.share = c.share, a.keydim = c.keydim, a.valdim = c.valdim;
    a.scale = c.scale;
    return hip_status(launch_gd_step(a, problem->act_dtype, (hipStream_t)stream));
}

int ssd_block_norm_fwd(const ssd_block* problem, const void* x, const void* y, const void* z,
                       const float* scale, const float* post_weight, const float* post_bias,
                       const float* pre_weight, const float* pre_bias, void* r, void* h, void* stream) {
    BlockArgs a = {};
    const int rc = check_block(problem, &a);
    if (rc) return rc;
    if (!x || !y || !r || (a.gate && !z) || (a.post && !post_weight) || (a.pre && (!pre_weight || !h)))
        return SSD_ERR_NULL;
    for (const void* p : {x, (const void*)r})
        if (!aligned(p, bytes_of(problem->res_dtype))) return SSD_ERR_ALIGN;
    for (const void* p : {y, z, (const void*)h})
        if (!aligned(p, bytes_of(problem->act_dtype))) return SSD_ERR_ALIGN;
    for (const void* p : {scale, post_weight, post_bias, pre_weight, pre_bias})
        if (!aligned(p, 4)) return SSD_ERR_ALIGN;
    a.x = x, a.y = y, a.z = a.gate ? z : nullptr, a.scale = scale;
    a.w1 = a.post ? post_weight : nullptr, a.b1 = a.post ? post_bias : nullptr;
    a.w2 = a.pre ? pre_weight : nullptr, a.b2 = a.pre ? pre_bias : nullptr;
    a.r = r, a.h = a.pre ? h : nullptr;
    return hip_status(launch_block_fwd(a, problem->act_dtype, problem->res_dtype, (hipStream_t)stream));
}

size_t ssd_block_norm_workspace_bytes(const ssd_block* problem) {
    BlockArgs a = {};
    if (check_block(problem, &a) != SSD_OK) return 0;
    return block_bwd_ws(a);
}

int ssd_block_norm_bwd(const ssd_block* problem, const void* x, const void* y, const void* z,
                       const float* scale, const float* post_weight, const float* post_bias,
                       const float* pre_weight, const void* dr, const void* dh, void* dx, void* dy,
                       void* dz, float* dscale, float* dpost_weight, float* dpost_bias,
                       float* dpre_weight, float* dpre_bias, void* ws, size_t ws_bytes, void* stream) {
    BlockArgs a = {};
    const int rc = check_block(problem, &a);
    if (rc) return rc;
    if (!x || !y || !dx || !dy || (a.gate && (!z || !dz)) || (a.post && !post_weight) ||
        (a.pre ? !pre_weight || !dh : !dr))
        return SSD_ERR_NULL;
    if (!ws || ws_bytes < block_bwd_ws(a)) return SSD_ERR_WORKSPACE;
    for (const void* p : {x, dr, (const void*)dx})
        if (!aligned(p, bytes_of(problem->res_dtype))) return SSD_ERR_ALIGN;
    for (const void* p : {y, z, dh, (const void*)dy, (const void*)dz})
        if (!aligned(p, bytes_of(problem->act_dtype))) return SSD_ERR_ALIGN;
    for (const void* p : {(const void*)scale, (const void*)post_weight, (const void*)post_bias,
                          (const void*)pre_weight, (const void*)dscale, (const void*)dpost_weight,
                          (const void*)dpost_bias, (const void*)dpre_weight, (const void*)dpre_bias,
                          (const void*)ws})
        if (!aligned(p, 4)) return SSD_ERR_ALIGN;
    a.x = x, a.y = y, a.z = a.gate ? z : nullptr, a.scale = scale;
    a.w1 = a.post ? post_weight : nullptr, a.b1 = a.post ? post_bias : nullptr;
    a.w2 = a.pre ? pre_weight : nullptr;
    a.dr = dr, a.dh = a.pre ? dh : nullptr;
    a.dx = dx, a.dy = dy, a.dz = a.gate ? dz : nullptr;
    a.dscale = dscale;
    a.dw1 = a.post ? dpost_weight : nullptr, a.db1 = a.post ? dpost_bias : nullptr;
    a.dw2 = a.pre ? dpre_weight : nullptr, a.db2 = a.pre ? dpre_bias : nullptr;
    return hip_status(
        launch_block_bwd(a, problem->act_dtype, problem->res_dtype, (float*)ws, (hipStream_t)stream));
}

int ssd_rope(const ssd_rope_problem* problem, const void* q, const void* k, const double* frequencies,
             const int32_t* positions, const int32_t* cu_seqlens, int32_t nseq, int32_t inverse,
             void* q_out, void* k_out, void* stream) {
    RopeArgs a = {};
    const int rc = check_rope(problem, &a);
    if (rc) return rc;
    if (inverse != 0 && inverse != 1) return SSD_ERR_SHAPE;
    if (cu_seqlens && (problem->batch != 1 || nseq < 1 || nseq > (1 << 24))) return SSD_ERR_SEGMENTS;
    if (!q || !q_out || !frequencies || (a.K > 0 && (!k || !k_out))) return SSD_ERR_NULL;
    const unsigned e = bytes_of(problem->act_dtype);
    for (const void* p : {q, k, (const void*)q_out, (const void*)k_out})
        if (!aligned(p, e)) return SSD_ERR_ALIGN;
    if (!aligned(frequencies, 8) || !aligned(positions, 4) || !aligned(cu_seqlens, 4)) return SSD_ERR_ALIGN;
    a.q = q, a.k = k, a.qo = q_out, a.ko = k_out;
    a.freq = frequencies, a.positions = positions, a.cu = cu_seqlens, a.nseq = nseq;
    a.turn = inverse ? -1.f : 1.f;
    return hip_status(launch_rope(a, problem->act_dtype, (hipStream_t)stream));
}

}  // extern "C"
