// Linear attention with a decay per head: the walk over prompts (forward and, with the
// operands in other roles, backward).
//
//   M_t = l M_(t-1) + s c_t b_t^T,   out_t = f M_t a_t
//
// One workgroup per (sequence, head): thread d keeps row d of M in registers and goes
// through the tokens one by one, their a and b rows passing through LDS.
#include "mixer_internal.h"

namespace ssd {

template <typename T, int BD>
__global__ void __launch_bounds__(128) k_la_tokens(LaWalk w) {
    __shared__ float sa[BD], sb[BD];
    const int s = blockIdx.x / w.H, h = blockIdx.x % w.H, d = threadIdx.x;
    const SeqRange r = seq_range(w, s);
    const int len = (int)(r.hi - r.lo);
    const float l = expf(w.log_decay[h]);
    const int64_t st = ((int64_t)s * w.H + h) * BD * w.cd;
    const int64_t rs = w.trans ? 1 : BD, ks = w.trans ? w.cd : 1;
    float M[BD];
#pragma unroll
    for (int e = 0; e < BD; ++e) M[e] = w.init ? w.init[st + d * rs + e * ks] : 0.f;
    for (int i = 0; i < len; ++i) {
        const int64_t t = w.reverse ? r.hi - 1 - i : r.lo + i;
        const T* a = (const T*)w.a + t * w.a_ts + (h / w.a_div) * BD;
        const T* b = (const T*)w.b + t * w.b_ts + (h / w.b_div) * BD;
        for (int e = d; e < BD; e += blockDim.x) {
            sa[e] = (float)a[e];
            sb[e] = (float)b[e];
        }
        __syncthreads();
        const float c = w.state_scale * (float)((const T*)w.c)[t * w.c_ts + (h / w.c_div) * w.cd + d];
        const float keep = w.reverse && i == 0 ? 1.f : l;
        float o = 0.f;
#pragma unroll
        for (int e = 0; e < BD; ++e) {
            M[e] = M[e] * keep + c * sb[e];
            o += M[e] * sa[e];
        }
        o *= w.inter;
        const int64_t at = t * w.out_ts + (int64_t)h * w.cd + d;
        if (w.out_f32) ((float*)w.out)[at] = o;
        else ((T*)w.out)[at] = (T)o;
        __syncthreads();
    }
    if (w.fin) {
        const float keep = w.reverse && len > 0 ? l : 1.f;
#pragma unroll
        for (int e = 0; e < BD; ++e) w.fin[st + d * rs + e * ks] = M[e] * keep;
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

bool la_supported(int keydim, int valdim, int act) {
    return (keydim == 64 || keydim == 128) && (valdim == 64 || valdim == 128) &&
           (act == SSD_F32 || act == SSD_BF16);
}

size_t la_walk_ws(const LaWalk&, int) { return 0; }

template <typename T>
static hipError_t walk_t(const LaWalk& w, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)w.nseq * w.H)), block(w.cd);
    if (w.bd == 64) return launch(k_la_tokens<T, 64>, grid, block, s, w);
    return launch(k_la_tokens<T, 128>, grid, block, s, w);
}

hipError_t launch_la_walk(const LaWalk& w, int act, void*, hipStream_t s) {
    return act == SSD_BF16 ? walk_t<bf16>(w, s) : walk_t<float>(w, s);
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
