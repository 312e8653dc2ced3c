// Linear attention with a decay per head over prompts: launches of the walk (la_walk.h),
// the composition of span states and the sum over heads that share keys and values.
//
// Whole calls: 134 us forward and 351 us backward for 2 x 8192 tokens, 32 heads of 128 x 64 in
// bf16 (every tensor once at a copy's rate: 78 and 143 us).
#include "la_walk.h"

namespace ssd {

// States entering the spans of a sequence from the states its spans add, in place.  One lane per
// four state elements of a (sequence, head).
__device__ __forceinline__ void la_compose(const LaWalk& w, const LaPlan& plan,
                                           f32x4* __restrict__ ws, int64_t block) {
    const int quads = w.bd * w.cd / 4, per = quads / 256;
    const int h = (int)(block / per % w.H), s = (int)(block / per / w.H);
    const int q = (int)(block % per) * 256 + threadIdx.x;
    const SeqRange r = seq_range(w, s);
    const int64_t n = (r.hi - r.lo + plan.span - 1) / plan.span;
    if (n < 3) return;  // what the first span adds is what enters the second
    const float keep = la_held((float)exp((double)plan.span * (double)w.log_decay[h]));
    const int64_t step = (int64_t)w.H * quads;
    f32x4* p = ws + la_place(w, plan, s, r.lo, 1) * step + (int64_t)h * quads + q;
    f32x4 m = *p;
    for (int64_t j = 2; j < n; ++j) {
        p += step;
        m = m * keep + *p;
        *p = m;
    }
}
__global__ void __launch_bounds__(256) k_la_spans(LaWalk w, LaPlan plan, f32x4* __restrict__ ws) {
    la_compose(w, plan, ws, blockIdx.x);
}
__global__ void __launch_bounds__(256) k_la_spans_bwd(LaBwd b, LaPlan plan) {
    la_compose(b.w[blockIdx.y], plan, b.ws[blockIdx.y], blockIdx.x);
}

// out[t][hk][d] = sum over the group's heads of part[t][h][d], tokens of sequences only; four
// channels to a lane.
struct LaSum {
    const float* part[2];
    void* out[2];
    int64_t out_ts[2];
    int cd[2];
};
template <typename T>
__global__ void __launch_bounds__(256) k_la_group_sum(LaWalk w, LaSum s) {
    const int k = blockIdx.y, cd = s.cd[k], r = w.share, n = w.H / r * (cd / 4);
    const int64_t lo = seq_range(w, 0).lo, hi = seq_range(w, w.nseq - 1).hi;
    typedef typename Vec4<T>::type vt;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < (hi - lo) * n; i += gridDim.x * 256ll) {
        const int64_t t = lo + i / n;
        const int c = (int)(i % n), hk = c / (cd / 4), d = c % (cd / 4) * 4;
        const float* p = s.part[k] + (t * w.H + (int64_t)hk * r) * cd + d;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < r; ++j) v += *(const f32x4*)(p + (int64_t)j * cd);
        *(vt*)((T*)s.out[k] + t * s.out_ts[k] + hk * cd + d) = vt{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    }
}

bool la_supported(int keydim, int valdim, int act) {
    return (keydim == 64 || keydim == 128) && (valdim == 64 || valdim == 128) &&
           (act == SSD_F32 || act == SSD_BF16);
}

// Spans.  A sequence walked whole takes about a microsecond per 64 tokens; one walked in
// spans takes two launches more, a second pass over b and c and a state's round trip per
// span.  So: none up to LA_WHOLE tokens.  Longer rows are cut into the n spans that should
// take the least time, counted in tokens that a workgroup walks one after the other: the
// launch needs ceil(workgroups / LA_ROOM) turns of the CUs' room (two workgroups each), the
// pass before it, over all spans but the last, 0.55 of that per token (43 against 80 us for
// 2 x 8192 tokens, 32 heads of 128 x 64 with scores and states of one bf16, 43 against 87 with two), and the rest about 256 tokens and a 64th of a span
// for each.  (Three walks of those rows in 3 spans of 2731 tokens, 576 workgroups in two
// turns: 414 us; in 8 of 1024, 1536 in three: 394 us.)  Packed sequences have their
// lengths on the device: their tokens are cut as if into one row, but at least into two
// turns' worth, since they fill the turns unevenly, less half a span for each sequence, whose
// last span is as good as half empty (32768 tokens of 32 heads of 128 x 128: 415 us, without
// that allowance 428; these and the 414 and 394 with one bf16).
constexpr int LA_ROOM = 512, LA_MIN_SPAN = 256, LA_WHOLE = 1024;

static LaPlan la_plan(const LaWalk& w, int walks) {
    const int64_t longest = w.cu ? w.tokens : w.seqlen;
    const int64_t rows = w.cu ? 1 : w.nseq, per = rows * w.H * walks;  // workgroups per span
    auto turns = [](int64_t blocks) { return (double)((blocks + LA_ROOM - 1) / LA_ROOM); };
    int64_t best = 1;
    if (longest > LA_WHOLE) {
        double least = turns(per) * (double)longest;
        const int64_t most = (longest + LA_MIN_SPAN - 1) / LA_MIN_SPAN;
        for (int64_t n = 2; n <= (most < 256 ? most : 256); ++n) {
            const double span = (double)((longest + n - 1) / n);
            const double t = turns(per * n) * span + 0.55 * turns(per * (n - 1)) * span + 256.0 +
                             (double)n * 16.0;
            if (t < least) least = t, best = n;
        }
        if (w.cu) {
            const int64_t n = 2 * LA_ROOM / per - w.nseq / 2;
            if (n > best) best = n < most ? n : most;
        }
    }
    LaPlan p;
    p.split = best > 1;
    p.span = (int)(((longest + best - 1) / best + 63) / 64 * 64);
    p.per_row = (int)((w.seqlen + p.span - 1) / p.span);
    p.slots = w.cu ? w.tokens / p.span + w.nseq : (int64_t)w.nseq * p.per_row;
    return p;
}

static size_t state_ws(const LaWalk& w, const LaPlan& p) {
    return p.split ? align256((size_t)la_places(w, p) * w.H * w.bd * w.cd * 4) : 0;
}

size_t la_fwd_ws(const LaWalk& w) { return state_ws(w, la_plan(w, 1)); }

// Span states of the three walks, then, where heads share keys and values, dv and dk per
// head in float32.
size_t la_bwd_ws(const LaWalk& dv) {
    size_t n = 3 * state_ws(dv, la_plan(dv, 3));
    if (dv.share > 1) n += align256((size_t)dv.tokens * dv.H * (dv.bd + dv.cd) * 4);
    return n;
}

template <typename T, int BD, int CD, int SPLITS>
static hipError_t fwd_splits(const LaWalk& w, f32x4* ws, hipStream_t s) {
    const LaPlan p = la_plan(w, 1);
    const dim3 grid = la_grid(w, p, w.share), block(256);
    if (p.split) {
        SSD_TRY(launch(k_la_fwd<T, BD, CD, LA_STATE, SPLITS>, grid, block, s, w, p, ws));
        SSD_TRY(launch(k_la_spans, dim3((unsigned)((int64_t)w.nseq * w.H * (BD * CD / 1024))),
                       block, s, w, p, ws));
    }
    return launch(k_la_fwd<T, BD, CD, LA_ACT, SPLITS>, grid, block, s, w, p, ws);
}

template <typename T, int BD, int CD>
static hipError_t fwd_dims(const LaWalk& w, f32x4* ws, hipStream_t s) {
    if constexpr (sizeof(T) == 4) return fwd_splits<T, BD, CD, 1>(w, ws, s);
    else return w.fin ? fwd_splits<T, BD, CD, 3>(w, ws, s) : fwd_splits<T, BD, CD, 2>(w, ws, s);
}

template <typename T>
static hipError_t fwd_t(const LaWalk& w, f32x4* ws, hipStream_t s) {
    if (w.bd == 64) return w.cd == 64 ? fwd_dims<T, 64, 64>(w, ws, s) : fwd_dims<T, 64, 128>(w, ws, s);
    return w.cd == 64 ? fwd_dims<T, 128, 64>(w, ws, s) : fwd_dims<T, 128, 128>(w, ws, s);
}

hipError_t launch_la_fwd(const LaWalk& w, int act, void* ws, hipStream_t s) {
    return act == SSD_BF16 ? fwd_t<bf16>(w, (f32x4*)ws, s) : fwd_t<float>(w, (f32x4*)ws, s);
}

template <typename T, int DK, int DV, int OUT, int SPLITS, int SPLITS_DV>
static hipError_t bwd_splits(const LaBwd& b, hipStream_t s) {
    const LaWalk& w = b.w[0];
    const LaPlan p = la_plan(w, 3);
    const dim3 grid = la_grid(w, p, 3 * w.share), block(256);
    if (p.split) {
        SSD_TRY(launch(k_la_bwd<T, DK, DV, LA_STATE, SPLITS, SPLITS_DV>, grid, block, s, b, p));
        SSD_TRY(launch(k_la_spans_bwd,
                       dim3((unsigned)((int64_t)w.nseq * w.H * (DK * DV / 1024)), 3), block, s, b, p));
    }
    return launch(k_la_bwd<T, DK, DV, OUT, SPLITS, SPLITS_DV>, grid, block, s, b, p);
}

template <typename T, int DK, int DV, int OUT>
static hipError_t bwd_out(const LaBwd& b, hipStream_t s) {
    if constexpr (sizeof(T) == 4) return bwd_splits<T, DK, DV, OUT, 1, 1>(b, s);
    else if (b.w[LA_DV].fin) return bwd_splits<T, DK, DV, OUT, 2, 3>(b, s);
    else return bwd_splits<T, DK, DV, OUT, 2, 2>(b, s);
}

template <typename T, int DK, int DV>
static hipError_t bwd_dims(const LaBwd& b, hipStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (b.w[0].share > 1) return bwd_out<T, DK, DV, LA_F32>(b, s);
    return bwd_out<T, DK, DV, LA_ACT>(b, s);  // float32 parts are its own type
}

template <typename T>
static hipError_t bwd_t(LaBwd b, void* ws, hipStream_t s) {
    const LaWalk& dv = b.w[LA_DV];
    const size_t st = state_ws(dv, la_plan(dv, 3));
    for (int i = 0; i < 3; ++i) b.ws[i] = (f32x4*)((char*)ws + i * st);
    const bool shared = dv.share > 1;
    LaSum sum = {};
    if (shared) {
        float* part = (float*)((char*)ws + 3 * st);
        for (int i = 0; i < 2; ++i) {
            LaWalk& w = b.w[LA_DV + i];
            sum.part[i] = part;
            sum.out[i] = w.out;
            sum.out_ts[i] = w.out_ts;
            sum.cd[i] = w.cd;
            w.out = part;
            w.out_ts = (int64_t)w.H * w.cd;
            part += w.tokens * w.out_ts;
        }
    }
    const int dk = dv.bd, dvd = dv.cd;
    if (dk == 64) SSD_TRY(dvd == 64 ? bwd_dims<T, 64, 64>(b, s) : bwd_dims<T, 64, 128>(b, s));
    else SSD_TRY(dvd == 64 ? bwd_dims<T, 128, 64>(b, s) : bwd_dims<T, 128, 128>(b, s));
    if (!shared) return hipSuccess;
    const int64_t n = (dv.tokens * (dv.H / dv.share) * ((dk > dvd ? dk : dvd) / 4) + 255) / 256;
    return launch(k_la_group_sum<T>, dim3((unsigned)(n < 4096 ? n : 4096), 2), dim3(256), s, dv, sum);
}

hipError_t launch_la_bwd(const LaWalk& dq, const LaWalk& dv, const LaWalk& dk, int act, void* ws,
                         hipStream_t s) {
    LaBwd b = {};
    b.w[LA_DQ] = dq;
    b.w[LA_DV] = dv;
    b.w[LA_DK] = dk;
    return act == SSD_BF16 ? bwd_t<bf16>(b, ws, s) : bwd_t<float>(b, ws, s);
}

}  // namespace ssd
