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

}  // extern "C"
