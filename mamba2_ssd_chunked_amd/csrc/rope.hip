// Rotary positions of queries and keys (include/ssd_layer.h).
//
// Bound by HBM: q and k read and written once (16384 tokens of 40 heads of 128: 61 us, 5.5 TB/s, a part
// of it from the last-level cache).  A workgroup takes a token at a time: its threads form
// the token's cosines and sines once for all heads, then turn the heads' pairs.  An angle is p f in
// float64, less its whole turns; what is left of a turn keeps float32's relative precision.
#include "layer_internal.h"

namespace ssd {

// V: neighbouring channels that a thread moves at once, 8, or 1 where sizes or alignment ask for it (16384 tokens of 40
// heads of 96 in bf16, 24 channels turned: 39 us in neighbouring pairs, 112 in halves, which go one by one).
template <typename T, int V>
__global__ void __launch_bounds__(256) k_rope(RopeArgs a) {
    // rows are known to be aligned to 16 bytes, or to their elements, and no further
    typedef T vt __attribute__((ext_vector_type(V), aligned(V == 1 ? sizeof(T) : 16)));
    __shared__ float cs[ROPE_MAX_DIM / 2], sn[ROPE_MAX_DIM / 2];
    const int half = a.R / 2;
    const bool pairs = a.style == SSD_ROPE_HALF;
    // a thread's unit: V pairs (half) or V / 2 (interleaved; V = 1: one), or V channels that are copied
    const int turned = pairs || V == 1 ? half / V : a.R / V, units = turned + (a.D - a.R) / V;
    for (int64_t tok = blockIdx.x; tok < a.tokens; tok += gridDim.x) {
        int64_t place = tok % a.seqlen;
        if (a.cu) {
            int lo = 0, hi = a.nseq - 1;  // the last sequence that begins at or before the token
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (a.cu[mid] <= tok) lo = mid;
                else hi = mid - 1;
            }
            if (a.cu[lo] > tok || a.cu[lo + 1] <= tok) continue;  // in none
            place = tok - a.cu[lo];
        }
        const double p = (double)(a.positions ? (int64_t)a.positions[tok] : place);
        __syncthreads();  // the last token's are read
        for (int i = threadIdx.x; i < half; i += 256) {
            const double turns = p * a.freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
            const float left = (float)(turns - rint(turns));
            float s, c;
            sincospif(2.f * left, &s, &c);
            cs[i] = c * a.factor;
            sn[i] = s * a.factor * a.turn;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < (a.H + a.K) * units; x += 256) {
            const int head = x / units, u = x % units;
            const bool q = head < a.H;
            const T* in = q ? (const T*)a.q + tok * a.qs + (int64_t)head * a.D
                            : (const T*)a.k + tok * a.ks + (int64_t)(head - a.H) * a.D;
            T* out = q ? (T*)a.qo + tok * a.qos + (int64_t)head * a.D
                       : (T*)a.ko + tok * a.kos + (int64_t)(head - a.H) * a.D;
            if (u >= turned) {
                const int c = a.R + (u - turned) * V;
                *(vt*)(out + c) = *(const vt*)(in + c);
            } else if (pairs) {
                const vt v = *(const vt*)(in + u * V), w = *(const vt*)(in + half + u * V);
                vt y, z;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float c = cs[u * V + e], s = sn[u * V + e];
                    y[e] = (T)((float)v[e] * c - (float)w[e] * s);
                    z[e] = (T)((float)w[e] * c + (float)v[e] * s);
                }
                *(vt*)(out + u * V) = y;
                *(vt*)(out + half + u * V) = z;
            } else if constexpr (V == 1) {
                const float v = (float)in[2 * u], w = (float)in[2 * u + 1], c = cs[u], s = sn[u];
                out[2 * u] = (T)(v * c - w * s);
                out[2 * u + 1] = (T)(w * c + v * s);
            } else {
                const vt v = *(const vt*)(in + u * V);
                vt y;
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float c = cs[(u * V + e) / 2], s = sn[(u * V + e) / 2];
                    y[e] = (T)((float)v[e] * c - (float)v[e + 1] * s);
                    y[e + 1] = (T)((float)v[e + 1] * c + (float)v[e] * s);
                }
                *(vt*)(out + u * V) = y;
            }
        }
    }
}

template <typename T>
static hipError_t rope_t(const RopeArgs& a, hipStream_t s) {
    const int64_t e = sizeof(T);
    auto ok = [&](const void* p, int64_t stride) { return (((uintptr_t)p | (uintptr_t)(stride * e)) & 15) == 0; };
    const bool wide = a.D % 8 == 0 && a.R % (a.style == SSD_ROPE_HALF ? 16 : 8) == 0 && ok(a.q, a.qs) && ok(a.qo, a.qos) &&
                      (a.K == 0 || (ok(a.k, a.ks) && ok(a.ko, a.kos)));
    const dim3 grid((unsigned)(a.tokens < (1 << 22) ? a.tokens : (1 << 22)));
    if (wide) return launch(k_rope<T, 8>, grid, dim3(256), s, a);
    return launch(k_rope<T, 1>, grid, dim3(256), s, a);
}
hipError_t launch_rope(const RopeArgs& a, int act, hipStream_t s) {
    return act == SSD_BF16 ? rope_t<bf16>(a, s) : rope_t<float>(a, s);
}

}  // namespace ssd
