// The gated delta rule token by token:
//   S <- a S,  u = beta (v - S k),  S <- S + u k^T,  o = scale S q     (S of [valdim][keydim])
// A lane owns four neighbouring key channels of some rows of S, a group of keydim / 4 lanes a whole row;
// the state passes through registers once per call, however many tokens it has.  Bound by HBM, 8
// bytes per state element: 256 rows of 32 heads of 128 x 128 take 211 us, 5.1 TB/s; one row 6.2 us, a launch and the
// trip to memory and back.
#include <cfloat>

#include "layer_internal.h"

namespace ssd {

template <int LPR>
__device__ __forceinline__ float gd_lanes_sum(float v) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}
template <typename T>
__device__ __forceinline__ f32x4 gd_load4(const T* p) {
    const typename Vec4<T>::type v = *(const typename Vec4<T>::type*)p;
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}
__device__ __forceinline__ float gd_sum4(f32x4 v) { return (v[0] + v[1]) + (v[2] + v[3]); }

// One workgroup of four waves per (row, head, 64 value channels).
template <typename T, int BD>
__global__ void __launch_bounds__(256) k_gd_step(GdStep a) {
    constexpr int LPR = BD / 4, RPW = 64 / LPR, NR = 16 / RPW;
    const int lane = threadIdx.x % 64, col = 4 * (lane % LPR);
    const int nvb = a.valdim / 64;
    int item = blockIdx.x;
    const int vb = item % nvb;
    item /= nvb;
    const int h = item % a.H, row = item / a.H;
    const int64_t slot = row_slot(a.slots, a.positions, a.nslots, row);
    if (slot < 0) return;
    const int d0 = vb * 64 + wave_id() * 16 + lane / LPR;  // row of pass i: d0 + i RPW
    float* S = a.state + ((slot * a.H + h) * a.valdim + d0) * BD + col;
    f32x4 m[NR];
    const bool fresh = a.positions && a.positions[row] == 0;
#pragma unroll
    for (int i = 0; i < NR; ++i)
        m[i] = fresh ? f32x4{0.f, 0.f, 0.f, 0.f} : *(const f32x4*)(S + i * RPW * BD);
    if (row_taken(a.slots, a.positions, slot, row, lane)) return;
    for (int t = 0; t < a.tokens; ++t) {
        const int64_t tok = (int64_t)row * a.tokens + t;
        const f32x4 q = gd_load4((const T*)a.q + tok * a.q_ts + h / a.share * BD + col);
        const f32x4 k = gd_load4((const T*)a.k + tok * a.k_ts + h / a.share * BD + col);
        const T* v = (const T*)a.v + tok * a.v_ts + (int64_t)h * a.valdim + d0;
        const float g = a.g[tok * a.g_ts + h];
        float keep = expf(g);
        if (keep == INFINITY) {
            // Beyond float32: by the root, here and below, so that a state of zeros stays one and a product that
            // float32 holds is right.  A g of infinity is not finite and leaves nothing that is, as in a prompt.
            keep = g < INFINITY ? fminf(expf(0.5f * g), FLT_MAX) : NAN;
#pragma unroll
            for (int i = 0; i < NR; ++i) m[i] *= keep;
        }
        const float beta = a.beta[tok * a.b_ts + h];
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            m[i] *= keep;
            const float u = beta * ((float)v[i * RPW] - gd_lanes_sum<LPR>(gd_sum4(m[i] * k)));
            m[i] += k * u;
            const float o = gd_lanes_sum<LPR>(gd_sum4(m[i] * q));
            if (lane % LPR == i) mine = o;
        }
        if (lane % LPR < NR)
            ((T*)a.o)[tok * a.o_ts + (int64_t)h * a.valdim + d0 + (lane % LPR) * RPW] = (T)(mine * a.scale);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) *(f32x4*)(S + i * RPW * BD) = m[i];
}

template <typename T>
static hipError_t gd_step_t(const GdStep& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.rows * a.H * (a.valdim / 64)));
    if (a.keydim == 64) return launch(k_gd_step<T, 64>, grid, dim3(256), s, a);
    return launch(k_gd_step<T, 128>, grid, dim3(256), s, a);
}

hipError_t launch_gd_step(const GdStep& a, int act, hipStream_t s) {
    return act == SSD_BF16 ? gd_step_t<bf16>(a, s) : gd_step_t<float>(a, s);
}

}  // namespace ssd
