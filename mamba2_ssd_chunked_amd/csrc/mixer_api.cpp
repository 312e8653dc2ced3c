// Host side of the C ABI declared in include/ssd_mixer.h: argument validation and kernel
// dispatch.  As in ssd_api.cpp, every check runs before anything is enqueued.
#include <algorithm>
#include <climits>
#include <hip/hip_runtime.h>

#include "mixer_internal.h"

using namespace ssd;

namespace {

bool aligned(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

// Workgroups of a one-dimensional launch of up to 256 threads: at most 2^32 - 1 work-items.
constexpr int64_t MAX_BLOCKS = 0xffffffffll / 256;

// ---- linear attention --------------------------------------------------------------

struct LaStrides {
    int64_t q, k, v, o, dq, dk, dv;
};

int check_linattn(const ssd_linattn* p, LaStrides* st) {
    if (!p) return SSD_ERR_NULL;
    if (p->batch < 1 || p->seqlen < 1 || p->nheads < 1 || p->nkvheads < 1 || p->keydim < 1 ||
        p->valdim < 1)
        return SSD_ERR_SHAPE;
    if (p->nheads % p->nkvheads != 0 || p->nheads > 65535) return SSD_ERR_SHAPE;
    if (p->act_dtype != SSD_F32 && p->act_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!la_supported(p->keydim, p->valdim, p->act_dtype)) return SSD_ERR_UNSUPPORTED;
    if (p->batch > INT32_MAX || p->seqlen > INT32_MAX || p->batch * p->seqlen > INT32_MAX - 127)
        return SSD_ERR_SHAPE;
    const int64_t esz = p->act_dtype == SSD_BF16 ? 2 : 4;
    auto stride = [&](int64_t given, int64_t packed, int64_t* out) {
        *out = given == 0 ? packed : given;
        if (*out < packed || *out >= (1ll << 23)) return (int)SSD_ERR_SHAPE;
        return *out * esz % 16 == 0 ? (int)SSD_OK : (int)SSD_ERR_ALIGN;
    };
    const int64_t H = p->nheads, K = p->nkvheads, Dk = p->keydim, Dv = p->valdim;
    int rc;
    if ((rc = stride(p->q_stride, H * Dk, &st->q))) return rc;
    if ((rc = stride(p->k_stride, K * Dk, &st->k))) return rc;
    if ((rc = stride(p->v_stride, K * Dv, &st->v))) return rc;
    if ((rc = stride(p->o_stride, H * Dv, &st->o))) return rc;
    if ((rc = stride(p->dq_stride, H * Dk, &st->dq))) return rc;
    if ((rc = stride(p->dk_stride, K * Dk, &st->dk))) return rc;
    return stride(p->dv_stride, K * Dv, &st->dv);
}

int check_sequences(const ssd_linattn* p, int32_t nseq, const int32_t* cu) {
    if (nseq < 1 || nseq > (1 << 24)) return SSD_ERR_SEGMENTS;
    if (cu ? p->batch != 1 : nseq != p->batch) return SSD_ERR_SEGMENTS;
    return SSD_OK;
}

// What every walk of a call has in common.
LaWalk base_walk(const ssd_linattn* p, int32_t nseq, const float* log_decay, const int32_t* cu) {
    LaWalk w = {};
    w.log_decay = log_decay;
    w.cu = cu;
    w.nseq = nseq;
    w.seqlen = p->seqlen;
    w.tokens = p->batch * p->seqlen;
    w.H = p->nheads;
    w.share = p->nheads / p->nkvheads;
    w.a_div = w.b_div = w.c_div = 1;
    return w;
}

LaWalk fwd_walk(const ssd_linattn* p, const LaStrides& st, int32_t nseq, const void* q,
                const void* k, const void* v, const float* log_decay, const int32_t* cu,
                const float* init, void* o, float* final_state) {
    LaWalk w = base_walk(p, nseq, log_decay, cu);
    const int div = p->nheads / p->nkvheads;
    w.a = q, w.a_ts = st.q;
    w.b = k, w.b_ts = st.k, w.b_div = div;
    w.c = v, w.c_ts = st.v, w.c_div = div;
    w.bd = p->keydim, w.cd = p->valdim;
    w.out = o, w.out_ts = st.o;
    w.init = init, w.fin = final_state;
    w.intra = w.inter = p->scale, w.state_scale = 1.f;
    return w;
}

// The three walks of the backward.
struct BwdWalks {
    LaWalk dq, dv, dk;
};
BwdWalks bwd_walks(const ssd_linattn* p, const LaStrides& st, int32_t nseq, const void* q,
                   const void* k, const void* v, const float* log_decay, const int32_t* cu,
                   const void* dout, const float* init, const float* dfinal, void* dq, void* dk,
                   void* dv, float* dinit) {
    const int div = p->nheads / p->nkvheads;
    BwdWalks b;
    LaWalk w = base_walk(p, nseq, log_decay, cu);
    w.a = dout, w.a_ts = st.o;
    w.b = v, w.b_ts = st.v, w.b_div = div;
    w.c = k, w.c_ts = st.k, w.c_div = div;
    w.bd = p->valdim, w.cd = p->keydim;
    w.out = dq, w.out_ts = st.dq;
    w.init = init, w.trans = true;
    w.intra = w.inter = p->scale, w.state_scale = 1.f;
    b.dq = w;
    w = base_walk(p, nseq, log_decay, cu);
    w.a = k, w.a_ts = st.k, w.a_div = div;
    w.b = q, w.b_ts = st.q;
    w.c = dout, w.c_ts = st.o;
    w.bd = p->keydim, w.cd = p->valdim;
    w.out = dv, w.out_ts = st.dv;
    w.init = dfinal, w.fin = dinit;
    w.reverse = true;
    w.intra = w.state_scale = p->scale, w.inter = 1.f;
    b.dv = w;
    w.a = v, w.a_ts = st.v;
    w.b = dout, w.b_ts = st.o;
    w.c = q, w.c_ts = st.q;
    w.bd = p->valdim, w.cd = p->keydim;
    w.out = dk, w.out_ts = st.dk;
    w.fin = nullptr, w.trans = true;
    b.dk = w;
    return b;
}

size_t linattn_ws(const ssd_linattn* p, const LaStrides& st, int32_t nseq, const int32_t* cu,
                  int32_t kind) {
    // the layout depends on no other pointer
    if (kind == SSD_WS_FORWARD)
        return la_fwd_ws(fwd_walk(p, st, nseq, nullptr, nullptr, nullptr, nullptr, cu, nullptr,
                                  nullptr, nullptr));
    return la_bwd_ws(bwd_walks(p, st, nseq, nullptr, nullptr, nullptr, nullptr, cu, nullptr,
                               nullptr, nullptr, nullptr, nullptr, nullptr, nullptr).dv);
}

// Every launch of the walks fits: up to three workgroups per (span, head), spans of at least
// 256 tokens, their number rounded up to one of 8 XCDs, and up to 16 per (sequence, head)
// to compose span states.
int check_walk_grid(const ssd_linattn* p, int32_t nseq) {
    typedef unsigned __int128 u128;
    const u128 spans = (u128)(p->batch * p->seqlen) / 256 + nseq;
    const u128 blocks = (3 * (spans + 8) > (u128)nseq * 16 ? 3 * (spans + 8) : (u128)nseq * 16) *
                        p->nheads;
    return blocks <= (u128)MAX_BLOCKS ? SSD_OK : SSD_ERR_SHAPE;
}

int check_row_blocks(int64_t rows, int64_t per_row) {
    return rows <= INT32_MAX && rows * per_row <= MAX_BLOCKS ? SSD_OK : SSD_ERR_SHAPE;
}

// ---- norm ---------------------------------------------------------------------------

int check_norm(const ssd_norm* p, NormArgs* a) {
    if (!p) return SSD_ERR_NULL;
    if (p->rows < 1 || p->channels < 1 || p->ngroups < 1) return SSD_ERR_SHAPE;
    if (p->channels % p->ngroups != 0 || p->channels > (1 << 20) || p->ngroups > 65535)
        return SSD_ERR_SHAPE;
    if (p->rows > INT32_MAX || p->rows * p->ngroups > INT32_MAX) return SSD_ERR_SHAPE;
    if (p->act_dtype != SSD_F32 && p->act_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (p->mode < SSD_NORM_NONE || p->mode > SSD_NORM_AFTER) return SSD_ERR_UNSUPPORTED;
    if (p->center != 0 && p->center != 1) return SSD_ERR_SHAPE;
    if (!(p->eps > 0.f) || !(p->eps < 1e30f)) return SSD_ERR_SHAPE;
    const int64_t given[] = {p->x_stride, p->z_stride, p->y_stride, p->dx_stride, p->dz_stride};
    int64_t* out[] = {&a->xs, &a->zs, &a->ys, &a->dxs, &a->dzs};
    for (int i = 0; i < 5; ++i) {
        *out[i] = given[i] == 0 ? p->channels : given[i];
        if (*out[i] < p->channels || *out[i] >= (1ll << 28)) return SSD_ERR_SHAPE;
    }
    a->rows = p->rows;
    a->C = p->channels;
    a->G = p->ngroups;
    a->gs = p->channels / p->ngroups;
    a->mode = p->mode;
    a->center = p->center;
    a->eps = p->eps;
    return SSD_OK;
}

bool norm_gated(const ssd_norm* p) {
    return p->mode == SSD_NORM_BEFORE || p->mode == SSD_NORM_AFTER;
}

}  // namespace

extern "C" {

size_t ssd_linattn_workspace_bytes(const ssd_linattn* problem, int32_t nseq, int32_t kind) {
    LaStrides st;
    if (check_linattn(problem, &st) != SSD_OK) return 0;
    if (nseq < 1 || nseq > (1 << 24) || check_walk_grid(problem, nseq) != SSD_OK) return 0;
    if (kind != SSD_WS_FORWARD && kind != SSD_WS_BACKWARD) return 0;
    // rows or packed sequences, whichever needs more (one row may be either)
    const int32_t packed = 0;
    if (problem->batch != 1 && nseq != problem->batch) return 0;
    size_t n = 256;  // 0 would say that the problem is invalid
    if (nseq == problem->batch) n = std::max(n, linattn_ws(problem, st, nseq, nullptr, kind));
    if (problem->batch == 1) n = std::max(n, linattn_ws(problem, st, nseq, &packed, kind));
    return n;
}

int ssd_linattn_fwd(const ssd_linattn* problem, int32_t nseq, const void* q, const void* k,
                    const void* v, const float* log_decay, const int32_t* cu_seqlens,
                    const float* init, void* o, float* final_state, void* ws, size_t ws_bytes,
                    void* stream) {
    LaStrides st;
    int rc = check_linattn(problem, &st);
    if (rc) return rc;
    if ((rc = check_sequences(problem, nseq, cu_seqlens))) return rc;
    if ((rc = check_walk_grid(problem, nseq))) return rc;
    if (!q || !k || !v || !log_decay || !o) return SSD_ERR_NULL;
    if (!ws || ws_bytes < linattn_ws(problem, st, nseq, cu_seqlens, SSD_WS_FORWARD)) return SSD_ERR_WORKSPACE;
    for (const void* x : {q, k, v, (const void*)init, (const void*)o, (const void*)final_state,
                          (const void*)ws})
        if (!aligned(x, 16)) return SSD_ERR_ALIGN;
    if (!aligned(log_decay, 4) || !aligned(cu_seqlens, 4)) return SSD_ERR_ALIGN;
    const LaWalk w = fwd_walk(problem, st, nseq, q, k, v, log_decay, cu_seqlens, init, o,
                              final_state);
    return hip_status(launch_la_fwd(w, problem->act_dtype, ws, (hipStream_t)stream));
}

int ssd_linattn_bwd(const ssd_linattn* problem, int32_t nseq, const void* q, const void* k,
                    const void* v, const float* log_decay, const int32_t* cu_seqlens,
                    const void* dout, const float* init, const float* dfinal, void* dq, void* dk,
                    void* dv, float* dinit, void* ws, size_t ws_bytes, void* stream) {
    LaStrides st;
    int rc = check_linattn(problem, &st);
    if (rc) return rc;
    if ((rc = check_sequences(problem, nseq, cu_seqlens))) return rc;
    if ((rc = check_walk_grid(problem, nseq))) return rc;
    if (!q || !k || !v || !log_decay || !dout || !dq || !dk || !dv) return SSD_ERR_NULL;
    if (!ws || ws_bytes < linattn_ws(problem, st, nseq, cu_seqlens, SSD_WS_BACKWARD)) return SSD_ERR_WORKSPACE;
    for (const void* x : {q, k, v, dout, (const void*)init, (const void*)dfinal, (const void*)dq,
                          (const void*)dk, (const void*)dv, (const void*)dinit, (const void*)ws})
        if (!aligned(x, 16)) return SSD_ERR_ALIGN;
    if (!aligned(log_decay, 4) || !aligned(cu_seqlens, 4)) return SSD_ERR_ALIGN;
    const BwdWalks b = bwd_walks(problem, st, nseq, q, k, v, log_decay, cu_seqlens, dout, init,
                                 dfinal, dq, dk, dv, dinit);
    return hip_status(launch_la_bwd(b.dq, b.dv, b.dk, problem->act_dtype, ws, (hipStream_t)stream));
}

int ssd_linattn_step(const ssd_linattn* problem, const void* q, const void* k, const void* v,
                     const float* log_decay, const int32_t* slots, int64_t nslots,
                     const int32_t* positions, float* state, void* o, void* stream) {
    LaStrides st;
    int rc = check_linattn(problem, &st);
    if (rc) return rc;
    if (nslots < 1 || (!slots && nslots < problem->batch)) return SSD_ERR_SHAPE;
    if ((rc = check_row_blocks(problem->batch, (int64_t)problem->nheads * problem->valdim / 16)))
        return rc;
    if (!q || !k || !v || !log_decay || !state || !o) return SSD_ERR_NULL;
    for (const void* x : {q, k, v, (const void*)state, (const void*)o})
        if (!aligned(x, 16)) return SSD_ERR_ALIGN;
    if (!aligned(log_decay, 4) || !aligned(slots, 4) || !aligned(positions, 4))
        return SSD_ERR_ALIGN;
    LaStep a = {};
    a.q = q, a.k = k, a.v = v, a.o = o;
    a.q_ts = st.q, a.k_ts = st.k, a.v_ts = st.v, a.o_ts = st.o;
    a.log_decay = log_decay;
    a.slots = slots, a.positions = positions, a.nslots = nslots;
    a.state = state;
    a.rows = (int)problem->batch, a.tokens = (int)problem->seqlen;
    a.H = problem->nheads, a.div = problem->nheads / problem->nkvheads;
    a.keydim = problem->keydim, a.valdim = problem->valdim;
    a.scale = problem->scale;
    return hip_status(launch_la_step(a, problem->act_dtype, (hipStream_t)stream));
}

int ssd_token_step(const ssd_problem* p, const void* xBC, const float* conv_w, const void* dt_raw,
                   const float* dt_bias, const float* A_log, const float* D, const int32_t* slots,
                   int64_t nslots, const int32_t* positions, void* conv_ring, int32_t ring_len,
                   float* state, void* y, void* stream) {
    if (!p) return SSD_ERR_NULL;
    if (p->batch < 1 || p->seqlen < 1 || p->nheads < 1 || p->headdim < 1 || p->dstate < 1 ||
        p->ngroups < 1 || p->conv_width < 1)
        return SSD_ERR_SHAPE;
    if (p->nheads % p->ngroups != 0 || p->nheads > 65535) return SSD_ERR_SHAPE;
    if (p->act_dtype != SSD_F32 && p->act_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!(p->dt_min >= 0.f) || !(p->dt_max >= p->dt_min)) return SSD_ERR_SHAPE;
    if (p->conv_width > 8) return SSD_ERR_UNSUPPORTED;
    bool known = false;
#define SSD_KNOWN(PP, NN) known = known || (p->headdim == PP && p->dstate == NN);
    if (p->act_dtype == SSD_F32) {
        SSD_F32_SHAPES(SSD_KNOWN)
    } else {
        SSD_BF16_SHAPES(SSD_KNOWN)
    }
#undef SSD_KNOWN
    if (!known) return SSD_ERR_UNSUPPORTED;
    if (p->seqlen > INT32_MAX || nslots < 1 || (!slots && nslots < p->batch)) return SSD_ERR_SHAPE;
    const int rc = check_row_blocks(p->batch, p->nheads);
    if (rc) return rc;
    if (p->batch * p->seqlen > INT32_MAX) return SSD_ERR_SHAPE;
    if (ring_len < p->conv_width - 1 + p->seqlen) return SSD_ERR_SHAPE;
    if (!xBC || !conv_w || !dt_raw || !dt_bias || !A_log || !D || !positions || !conv_ring ||
        !state || !y)
        return SSD_ERR_NULL;
    // all but the state is read and written element by element
    const unsigned e = p->act_dtype == SSD_BF16 ? 2 : 4;
    for (const void* x : {xBC, dt_raw, (const void*)conv_ring, (const void*)y})
        if (!aligned(x, e)) return SSD_ERR_ALIGN;
    for (const void* x : {(const void*)conv_w, (const void*)dt_bias, (const void*)A_log,
                          (const void*)D, (const void*)slots, (const void*)positions})
        if (!aligned(x, 4)) return SSD_ERR_ALIGN;
    if (!aligned(state, 16)) return SSD_ERR_ALIGN;
    TokenStep a = {};
    a.xBC = xBC, a.conv_w = conv_w, a.dt_raw = dt_raw, a.dt_bias = dt_bias;
    a.A_log = A_log, a.D = D;
    a.slots = slots, a.positions = positions, a.nslots = nslots;
    a.ring = conv_ring, a.state = state, a.y = y;
    a.rows = (int)p->batch, a.tokens = (int)p->seqlen;
    a.H = p->nheads, a.P = p->headdim, a.N = p->dstate, a.G = p->ngroups;
    a.W = p->conv_width, a.R = ring_len;
    a.C = (int64_t)p->nheads * p->headdim + 2ll * p->ngroups * p->dstate;
    a.dt_min = p->dt_min, a.dt_max = p->dt_max;
    return hip_status(launch_token_step(a, p->act_dtype, (hipStream_t)stream));
}

int ssd_norm_fwd(const ssd_norm* problem, const void* x, const void* z, const float* weight,
                 const float* bias, void* y, void* stream) {
    NormArgs a = {};
    const int rc = check_norm(problem, &a);
    if (rc) return rc;
    if (!x || !weight || !y || (norm_gated(problem) && !z)) return SSD_ERR_NULL;
    const unsigned e = problem->act_dtype == SSD_BF16 ? 2 : 4;
    if (!aligned(x, e) || !aligned(z, e) || !aligned(y, e) || !aligned(weight, 4) ||
        !aligned(bias, 4))
        return SSD_ERR_ALIGN;
    a.x = x, a.z = z, a.w = weight, a.b = bias, a.y = y;
    return hip_status(launch_norm_fwd(a, problem->act_dtype, (hipStream_t)stream));
}

size_t ssd_norm_workspace_bytes(const ssd_norm* problem) {
    NormArgs a = {};
    if (check_norm(problem, &a) != SSD_OK) return 0;
    return norm_bwd_ws(a, problem->act_dtype);
}

int ssd_norm_bwd(const ssd_norm* problem, const void* x, const void* z, const float* weight,
                 const float* bias, const void* dy, void* dx, void* dz, float* dweight,
                 float* dbias, void* ws, size_t ws_bytes, void* stream) {
    NormArgs a = {};
    const int rc = check_norm(problem, &a);
    if (rc) return rc;
    if (!x || !weight || !dy || !dx || !dweight) return SSD_ERR_NULL;
    if (norm_gated(problem) && (!z || !dz)) return SSD_ERR_NULL;
    if (!ws || ws_bytes < ssd_norm_workspace_bytes(problem)) return SSD_ERR_WORKSPACE;
    const unsigned e = problem->act_dtype == SSD_BF16 ? 2 : 4;
    for (const void* q : {x, z, dy, (const void*)dx, (const void*)dz})
        if (!aligned(q, e)) return SSD_ERR_ALIGN;
    for (const void* q : {(const void*)weight, (const void*)bias, (const void*)dweight,
                          (const void*)dbias, (const void*)ws})
        if (!aligned(q, 4)) return SSD_ERR_ALIGN;
    a.x = x, a.z = z, a.w = weight, a.b = bias, a.dy = dy;
    a.dx = dx, a.dz = dz, a.dw = dweight, a.db = dbias;
    return hip_status(launch_norm_bwd(a, problem->act_dtype, (float*)ws, (hipStream_t)stream));
}

}  // extern "C"
