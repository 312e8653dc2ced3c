// Internal types of the operators around the scan (include/ssd_mixer.h).
#pragma once

#include "../../include/ssd_mixer.h"
#include "ssd_internal.h"

namespace ssd {

// Launch with `lds` bytes of dynamic LDS (see launch).
template <typename... KArgs, typename... Args>
inline hipError_t launch_lds(void (*kernel)(KArgs...), dim3 grid, dim3 block, int lds, hipStream_t s,
                             Args&&... args) {
    std::tuple<KArgs...> a(std::forward<Args>(args)...);
    return std::apply(
        [&](auto&... v) {
            std::array<void*, sizeof...(KArgs) + 1> p = {(void*)&v..., nullptr};
            return hipLaunchKernel((const void*)kernel, grid, block, p.data(), lds, s);
        },
        a);
}

// ---- linear attention ------------------------------------------------------------
//
// Forward and backward are the same walk over a sequence with its operands in other
// roles: M <- l M + state_scale c_t b_t^T, out_t = l^(..) M a_t, M of [CD][BD].
//   o : a = q,  b = k,  c = v,  from the first token
//   dq: a = do, b = v,  c = k,  from the first token (M is the transposed state)
//   dv: a = k,  b = q,  c = do, from the last token
//   dk: a = v,  b = do, c = q,  from the last token (M is the transposed gradient)
struct LaWalk {
    const void *a, *b, *c;           // token rows, act_dtype
    int64_t a_ts, b_ts, c_ts;        // elements between tokens
    int a_div, b_div, c_div;         // head h reads head h / div of the operand
    int bd, cd;                      // channels per head of b (and a), of c (and out)
    void* out;                       // [tokens][H][cd]
    int64_t out_ts;
    const float* log_decay;          // [H]
    const int32_t* cu;               // [nseq + 1] or null (rows of `seqlen` tokens)
    int nseq;
    int64_t seqlen, tokens;          // tokens of a row, of all rows
    const float* init;               // [nseq][H] states or null
    float* fin;                      // [nseq][H] states or null
    bool trans;                      // states in memory are [BD][CD], not [CD][BD]
    bool reverse;                    // from the last token; the given state then meets the
                                     // first visited token undecayed, and `fin` is decayed
    float intra, inter, state_scale; // factors of c_j (b_j . a_i), of M a_i, of c b^T into M
    int H, share;                    // heads; neighbouring heads that share keys and values
};

// Sequence s as token range [lo, hi) over all rows; offsets outside the tokens are cut
// off, so that no table makes a kernel leave its tensors.
struct SeqRange {
    int64_t lo, hi;
};
__device__ __forceinline__ SeqRange seq_range(const LaWalk& w, int s) {
    SeqRange r;
    if (w.cu) {
        const int64_t a = w.cu[s], b = w.cu[s + 1];
        r.lo = a < 0 ? 0 : (a > w.tokens ? w.tokens : a);
        r.hi = b < r.lo ? r.lo : (b > w.tokens ? w.tokens : b);
    } else {
        r.lo = (int64_t)s * w.seqlen;
        r.hi = r.lo + w.seqlen;
    }
    return r;
}

size_t la_fwd_ws(const LaWalk& w);
size_t la_bwd_ws(const LaWalk& dv);  // the dv walk
hipError_t launch_la_fwd(const LaWalk& w, int act, void* ws, hipStream_t s);
// dv and dk hold the gradients' own tensors, also where heads share keys and values
hipError_t launch_la_bwd(const LaWalk& dq, const LaWalk& dv, const LaWalk& dk, int act, void* ws,
                         hipStream_t s);
bool la_supported(int keydim, int valdim, int act);

struct LaStep {
    const void *q, *k, *v;
    int64_t q_ts, k_ts, v_ts, o_ts;
    const float* log_decay;
    const int32_t *slots, *positions;
    int64_t nslots;
    float* state;
    void* o;
    int rows, tokens, H, div, keydim, valdim;
    float scale;
};
hipError_t launch_la_step(const LaStep& a, int act, hipStream_t s);

// ---- SSD token step ----------------------------------------------------------------
struct TokenStep {
    const void* xBC;
    const float* conv_w;
    const void* dt_raw;
    const float *dt_bias, *A_log, *D;
    const int32_t *slots, *positions;
    int64_t nslots;
    void* ring;
    float* state;
    void* y;
    int rows, tokens, H, P, N, G, W, R;
    int64_t C;
    float dt_min, dt_max;
};
hipError_t launch_token_step(const TokenStep& a, int act, hipStream_t s);

// ---- group norm --------------------------------------------------------------------
struct NormArgs {
    const void *x, *z, *dy;
    const float *w, *b;
    void *y, *dx, *dz;
    float *dw, *db;
    int64_t rows, xs, zs, ys, dxs, dzs;
    int C, G, gs;  // channels, groups, channels per group
    int mode, center;
    float eps;
};
// bytes of the backward's partial sums of dweight and dbias
size_t norm_bwd_ws(const NormArgs& a, int act);
hipError_t launch_norm_fwd(const NormArgs& a, int act, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, int act, float* part, hipStream_t s);

// ---- serving helpers ---------------------------------------------------------------
// Slot of row r, or -1 where the row is skipped: a slot outside the pool or a negative
// position.
__device__ __forceinline__ int64_t row_slot(const int32_t* slots, const int32_t* positions,
                                            int64_t nslots, int r) {
    if (positions && positions[r] < 0) return -1;
    if (!slots) return r;
    const int slot = __builtin_amdgcn_readfirstlane(slots[r]);
    return slot < 0 || slot >= nslots ? -1 : slot;
}
// Whether an earlier row that is not skipped has row r's slot: then row r is.  All lanes of
// the wave call it and agree.  Called with the state's loads on their way, which up to some
// hundred rows take as long; then it grows with the rows' square.  1024 slots are read at once
// (16384 rows of 4 heads of 64 x 64: 775 us, 1420 with 64 at once, 400 without slots).
__device__ __forceinline__ bool row_taken(const int32_t* slots, const int32_t* positions,
                                          int64_t slot, int r, int lane) {
    if (!slots) return false;
    bool same = false;
    for (int i = lane; i < r; i += 1024) {
        int32_t v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = slots[i + 64 * u < r ? i + 64 * u : i];
#pragma unroll
        for (int u = 0; u < 16; ++u) same = same | (v[u] == slot);
    }
    if (__ballot(same) == 0) return false;
    bool seen = false;  // rare: is one of them not skipped?
    for (int i = lane; i < r; i += 64)
        seen = seen || (slots[i] == slot && (!positions || positions[i] >= 0));
    return __ballot(seen) != 0;
}

}  // namespace ssd
