// The gated delta rule over prompts, forward: launches of gdelta_prep.h and gdelta_walk.h.
#include "gdelta_prep.h"
#include "gdelta_team.h"
#include "gdelta_walk.h"

namespace ssd {

// T in three parts (two without a last state), P in two, per-token factors.
struct GdFwdWs {
    size_t T, P, sc, total;
};
static GdFwdWs fwd_layout(const GdArgs& a, int act) {
    const size_t rows = (size_t)a.H * a.tokens, e = act == SSD_BF16 ? 2 : 4;
    GdFwdWs w;
    w.T = 0;
    w.P = align256(w.T + rows * GD_Q * (act == SSD_BF16 ? 3 : 1) * e);
    w.sc = align256(w.P + rows * GD_Q * (act == SSD_BF16 ? 2 : 1) * e);
    w.total = align256(w.sc + rows * 3 * sizeof(float));
    return w;
}
size_t gd_fwd_ws(const GdArgs& a, int act) { return fwd_layout(a, act).total; }

template <typename T, int DK, int PT>
static hipError_t fwd_parts(const GdArgs& a, hipStream_t s) {
    constexpr int PO = sizeof(T) == 2 ? 2 : 1;
    const LaPlan p = gd_plan(a);
    const GdShape w = gd_shape(a, sizeof(T) == 4);
    SSD_TRY(launch(k_gd_prep<T, DK, PT, PO, true>, dim3((unsigned)(p.slots * a.H)), dim3(256), s, a, p));
    const dim3 grid = gd_grid(a, a.valdim / (16 * w.waves * w.tiles));
    if (w.waves == 1) return launch(k_gd_team<T, DK, PT, false>, grid, dim3(256), s, a, p);
    if constexpr (sizeof(T) == 2)
        if (w.waves == 2) return launch(k_gd_walk<T, DK, 1, 2, PT, false>, grid, dim3(128), s, a, p);
    if (w.tiles == 1) return launch(k_gd_walk<T, DK, 1, 4, PT, false>, grid, dim3(256), s, a, p);
    return launch(k_gd_walk<T, DK, 2, 4, PT, false>, grid, dim3(256), s, a, p);
}

template <typename T, int DK>
static hipError_t fwd_dk(const GdArgs& a, hipStream_t s) {
    if constexpr (sizeof(T) == 4) return fwd_parts<T, DK, 1>(a, s);
    else return a.fin ? fwd_parts<T, DK, 3>(a, s) : fwd_parts<T, DK, 2>(a, s);
}

template <typename T>
static hipError_t fwd_t(const GdArgs& a, hipStream_t s) {
    return a.keydim == 64 ? fwd_dk<T, 64>(a, s) : fwd_dk<T, 128>(a, s);
}

hipError_t launch_gd_fwd(GdArgs a, int act, void* ws, hipStream_t s) {
    const GdFwdWs w = fwd_layout(a, act);
    a.T = (char*)ws + w.T;
    a.P = (char*)ws + w.P;
    a.in = (float*)((char*)ws + w.sc);
    a.out = a.in + (size_t)a.H * a.tokens;
    a.beta_of = a.out + (size_t)a.H * a.tokens;
    return act == SSD_BF16 ? fwd_t<bf16>(a, s) : fwd_t<float>(a, s);
}

}  // namespace ssd
