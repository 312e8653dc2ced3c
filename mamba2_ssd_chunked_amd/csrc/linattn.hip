// Linear attention with a decay per head over prompts: launches of the walk (la_walk.h),
// the composition of span states and the sum over heads that share keys and values.
#include "la_walk.h"

namespace ssd {

// States entering the spans of a sequence from the states its spans add: in place, slot
// j >= 1 receives the state after span j - 1.  One lane per four state elements of a
// (sequence, head).
__global__ void __launch_bounds__(256) k_la_spans(LaWalk w, LaPlan plan, int quads,
                                                 f32x4* __restrict__ ws) {
    const int per = quads / 256, h = (int)(blockIdx.x / per % w.H);
    const int s = (int)(blockIdx.x / per / w.H), q = (int)(blockIdx.x % per) * 256 + threadIdx.x;
    const SeqRange r = seq_range(w, s);
    const int64_t n = (r.hi - r.lo + plan.span - 1) / plan.span;
    if (n < 2) return;
    const float keep = (float)exp((double)plan.span * (double)w.log_decay[h]);
    const int64_t step = (int64_t)w.H * quads;
    f32x4* p = ws + la_first_slot(w, plan, s) * step + (int64_t)h * quads + q;
    f32x4 m = *p;
    for (int64_t j = 1; j < n; ++j) {
        p += step;
        f32x4 add = {0.f, 0.f, 0.f, 0.f};
        if (j + 1 < n) add = *p;
        *p = m;
        m = m * keep + add;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_la_group_sum(LaWalk w, const float* __restrict__ part,
                                                     int nkv, T* __restrict__ out, int64_t out_ts) {
    const int64_t lo = seq_range(w, 0).lo, hi = seq_range(w, w.nseq - 1).hi;
    const int r = w.H / nkv, n = nkv * w.cd;
    const int64_t total = w.tokens * n;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int64_t t = i / n;
        const int hk = (int)(i % n) / w.cd, d = (int)(i % n) % w.cd;
        if (t < lo || t >= hi) continue;
        const float* p = part + (t * w.H + (int64_t)hk * r) * w.cd + d;
        float s = 0.f;
        for (int j = 0; j < r; ++j) s += p[(int64_t)j * w.cd];
        out[t * out_ts + hk * w.cd + d] = (T)s;
    }
}

// Spans: two workgroups for each of the 256 CUs where the tokens allow it, but none
// shorter than 256 tokens (a span costs a state's round trip and a pass over b and c).
constexpr int LA_BLOCKS = 512, LA_MIN_SPAN = 256;

static LaPlan la_plan(const LaWalk& w) {
    const int64_t per = (w.tokens * w.H + LA_BLOCKS - 1) / LA_BLOCKS;
    LaPlan p;
    p.span = (int)((per > LA_MIN_SPAN ? per + 63 : LA_MIN_SPAN) / 64 * 64);
    p.per_row = (int)((w.seqlen + p.span - 1) / p.span);
    p.slots = w.cu ? w.tokens / p.span + w.nseq : (int64_t)w.nseq * p.per_row;
    p.split = (w.cu ? w.tokens : w.seqlen) > p.span;
    return p;
}

size_t la_walk_ws(const LaWalk& w, int) {
    const LaPlan p = la_plan(w);
    return p.split ? (size_t)p.slots * w.H * w.bd * w.cd * 4 : 0;
}

template <typename T, int BD, int CD, bool REV>
static hipError_t walk_shape(const LaWalk& w, f32x4* ws, hipStream_t s) {
    constexpr int FINE = sizeof(T) == 2 ? 3 : 1, FAST = sizeof(T) == 2 ? 2 : 1;
    const LaPlan p = la_plan(w);
    const int64_t units = p.slots * (w.H / w.share);
    const dim3 grid((unsigned)((units + 7) / 8 * 8 * w.share)), block(256);
    if (p.split) {
        SSD_TRY(launch(k_la_walk<T, BD, CD, REV, LA_STATE, FINE>, grid, block, s, w, p, ws));
        constexpr int quads = BD * CD / 4;
        SSD_TRY(launch(k_la_spans, dim3((unsigned)((int64_t)w.nseq * w.H * (quads / 256))),
                       dim3(256), s, w, p, quads, ws));
    }
    if constexpr (REV)
        if (w.out_f32) {
            if (w.fin)
                return launch(k_la_walk<T, BD, CD, REV, LA_F32, FINE>, grid, block, s, w, p, ws);
            return launch(k_la_walk<T, BD, CD, REV, LA_F32, FAST>, grid, block, s, w, p, ws);
        }
    if (w.fin) return launch(k_la_walk<T, BD, CD, REV, LA_ACT, FINE>, grid, block, s, w, p, ws);
    return launch(k_la_walk<T, BD, CD, REV, LA_ACT, FAST>, grid, block, s, w, p, ws);
}

template <typename T, bool REV>
static hipError_t walk_dims(const LaWalk& w, f32x4* ws, hipStream_t s) {
    if (w.bd == 64) return w.cd == 64 ? walk_shape<T, 64, 64, REV>(w, ws, s)
                                      : walk_shape<T, 64, 128, REV>(w, ws, s);
    return w.cd == 64 ? walk_shape<T, 128, 64, REV>(w, ws, s)
                      : walk_shape<T, 128, 128, REV>(w, ws, s);
}

template <typename T>
static hipError_t walk_t(const LaWalk& w, void* ws, hipStream_t s) {
    return w.reverse ? walk_dims<T, true>(w, (f32x4*)ws, s)
                     : walk_dims<T, false>(w, (f32x4*)ws, s);
}

bool la_supported(int keydim, int valdim, int act) {
    return (keydim == 64 || keydim == 128) && (valdim == 64 || valdim == 128) &&
           (act == SSD_F32 || act == SSD_BF16);
}

hipError_t launch_la_walk(const LaWalk& w, int act, void* ws, hipStream_t s) {
    return act == SSD_BF16 ? walk_t<bf16>(w, ws, s) : walk_t<float>(w, ws, s);
}

hipError_t launch_la_group_sum(const LaWalk& w, int act, const float* part, int nkv, void* out,
                               int64_t out_ts, hipStream_t s) {
    const int64_t n = (w.tokens * nkv * w.cd + 255) / 256;
    const dim3 grid((unsigned)(n < 16384 ? n : 16384)), block(256);
    if (act == SSD_BF16)
        return launch(k_la_group_sum<bf16>, grid, block, s, w, part, nkv, (bf16*)out, out_ts);
    return launch(k_la_group_sum<float>, grid, block, s, w, part, nkv, (float*)out, out_ts);
}

}  // namespace ssd
