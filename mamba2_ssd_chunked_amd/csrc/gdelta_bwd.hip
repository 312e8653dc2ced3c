// Backward of the gated delta rule over prompts: launches of gdelta_prep.h, gdelta_walk.h and
// gdelta_back.h.
#include "gdelta_back.h"
#include "gdelta_prep.h"
#include "gdelta_team.h"
#include "gdelta_walk.h"

namespace ssd {

// T and P in three parts, per-token factors, U and Z, entering states and leaving gradients, perhaps dq and dk
// of every head.
struct GdBwdWs {
    size_t T, P, sc, c2, U, Z, S, G, sums, total;
};
// Where the chunks of all key heads are too few for the CUs, the heads that share one get a workgroup each, and
// a launch of its own adds up their dq and dk (16 chunks of 2 key heads of 4 heads, 64 x 64: 41 us in turn, 16 and 4
// for the sums so).
static bool heads_apart(const GdArgs& a) {
    return a.share > 1 && a.tokens / GD_Q * (a.H / a.share) < 256;
}
static GdBwdWs bwd_layout(const GdArgs& a, int act) {
    const size_t rows = (size_t)a.H * a.tokens, mat = rows * GD_Q * (act == SSD_BF16 ? 6 : 4);
    const size_t states = (size_t)la_places(a, gd_plan(a)) * a.H * a.keydim * a.valdim * 4;
    GdBwdWs w;
    w.T = 0;
    w.P = align256(w.T + mat);
    w.sc = align256(w.P + mat);
    w.c2 = align256(w.sc + rows * 3 * sizeof(float));
    w.U = align256(w.c2 + rows * sizeof(double));
    w.Z = align256(w.U + rows * a.valdim * 4);
    w.S = align256(w.Z + rows * a.valdim * 4);
    w.G = align256(w.S + states);
    w.sums = align256(w.G + states);
    w.total = heads_apart(a) ? align256(w.sums + rows * a.keydim * 8) : w.sums;
    return w;
}
size_t gd_bwd_ws(const GdArgs& a, int act) { return bwd_layout(a, act).total; }

template <typename T, int DK>
static hipError_t walk(const GdArgs& a, const LaPlan& p, hipStream_t s) {
    constexpr int PT = sizeof(T) == 2 ? 3 : 1;
    const GdShape w = gd_shape(a, sizeof(T) == 4);
    const dim3 grid = gd_grid(a, a.valdim / (16 * w.tiles * w.waves));
    if (w.waves == 1) return launch(k_gd_team<T, DK, PT, true>, grid, dim3(256), s, a, p);
    if constexpr (sizeof(T) == 2)
        if (w.waves == 2) return launch(k_gd_walk<T, DK, 1, 2, PT, true>, grid, dim3(128), s, a, p);
    if (w.tiles == 1) return launch(k_gd_walk<T, DK, 1, 4, PT, true>, grid, dim3(256), s, a, p);
    return launch(k_gd_walk<T, DK, 2, 4, PT, true>, grid, dim3(256), s, a, p);
}

template <typename T, int DK>
static hipError_t walk_back(const GdArgs& a, const LaPlan& p, hipStream_t s) {
    constexpr int PT = sizeof(T) == 2 ? 3 : 1;
    const int waves = gd_back_waves(a);
    const dim3 grid = gd_grid(a, a.valdim / (16 * waves));
    if (waves == 2) return launch(k_gd_back<T, DK, 2, PT>, grid, dim3(128), s, a, p);
    return launch(k_gd_back<T, DK, 4, PT>, grid, dim3(256), s, a, p);
}

template <typename T, int DK, int DV>
static hipError_t bwd_dims(const GdArgs& a, hipStream_t s) {
    constexpr int PT = sizeof(T) == 2 ? 3 : 1;
    const LaPlan p = gd_plan(a);
    SSD_TRY(launch(k_gd_prep<T, DK, PT, PT, false>, dim3((unsigned)(p.slots * a.H)), dim3(256), s, a, p));
    SSD_TRY((walk<T, DK>(a, p, s)));
    SSD_TRY((walk_back<T, DK>(a, p, s)));
    const int64_t items = a.sums ? a.H : a.H / a.share;
    SSD_TRY(launch(k_gd_chunk<T, DK, DV>, dim3((unsigned)(p.slots * items)), dim3(DK * 4), s, a, p));
    if (!a.sums) return hipSuccess;
    const int64_t n = (a.tokens * (a.H / a.share) * (DK / 2) + 255) / 256;
    return launch(k_gd_sum<T>, dim3((unsigned)(n < 1024 ? n : 1024)), dim3(256), s, a);
}

template <typename T>
static hipError_t bwd_t(const GdArgs& a, hipStream_t s) {
    if (a.keydim == 64) return a.valdim == 64 ? bwd_dims<T, 64, 64>(a, s) : bwd_dims<T, 64, 128>(a, s);
    return a.valdim == 64 ? bwd_dims<T, 128, 64>(a, s) : bwd_dims<T, 128, 128>(a, s);
}

hipError_t launch_gd_bwd(GdArgs a, int act, void* ws, hipStream_t s) {
    const GdBwdWs w = bwd_layout(a, act);
    char* p = (char*)ws;
    a.T = p + w.T, a.P = p + w.P;
    a.in = (float*)(p + w.sc), a.c2 = (double*)(p + w.c2);
    a.out = a.in + (size_t)a.H * a.tokens;
    a.beta_of = a.out + (size_t)a.H * a.tokens;
    a.U = (float*)(p + w.U), a.Z = (float*)(p + w.Z);
    a.S = (float*)(p + w.S), a.G = (float*)(p + w.G);
    a.sums = heads_apart(a) ? (float*)(p + w.sums) : nullptr;
    return act == SSD_BF16 ? bwd_t<bf16>(a, s) : bwd_t<float>(a, s);
}

}  // namespace ssd
