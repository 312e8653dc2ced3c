// Single-token forms: linear attention and the conv1d + SSD path.
//
// Both update a float32 state per (slot, head) and contract it once:
//   S <- a S + u w^T,   o = S r      (S of [rows][cols])
// A lane owns four neighbouring columns of some rows, a group of cols / 4 lanes a whole
// row; the state passes through registers once per call, however many tokens it has.
// Bound by HBM: 8 bytes per state element (linear attention, 256 rows of 32 heads of 128 x 128:
// 210 us, 5.1 TB/s; SSD path, 256 rows of 64 heads of 64 x 128: 214 us, 5.0 TB/s), and with one
// row by the loads' latency (4.8 and 6.2 us).
#include <cfloat>

#include "dt_prep.h"
#include "mixer_internal.h"

namespace ssd {

// Sum over the LPR neighbouring lanes that share a row (LPR a power of two <= 64).
template <int LPR>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

template <typename T>
__device__ __forceinline__ f32x4 load4f(const T* p) {
    const typename Vec4<T>::type v = *(const typename Vec4<T>::type*)p;
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

// One workgroup of four waves per (row, head, 64 value channels).
template <typename T, int BD>
__global__ void __launch_bounds__(256) k_la_step(LaStep a) {
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
    float l = expf(a.log_decay[h]);
    if (l == INFINITY) l = FLT_MAX;  // a state of zeros stays one
    for (int t = 0; t < a.tokens; ++t) {
        const int64_t tok = (int64_t)row * a.tokens + t;
        const f32x4 q = load4f((const T*)a.q + tok * a.q_ts + h * BD + col);
        const f32x4 k = load4f((const T*)a.k + tok * a.k_ts + (h / a.div) * BD + col);
        const T* v = (const T*)a.v + tok * a.v_ts + (h / a.div) * a.valdim + d0;
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            m[i] = m[i] * l + k * (float)v[i * RPW];
            const f32x4 p = m[i] * q;
            const float o = lanes_sum<LPR>((p[0] + p[1]) + (p[2] + p[3]));
            if (lane % LPR == i) mine = o;
        }
        if (lane % LPR < NR)
            ((T*)a.o)[tok * a.o_ts + (int64_t)h * a.valdim + d0 + (lane % LPR) * RPW] =
                (T)(mine * a.scale);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) *(f32x4*)(S + i * RPW * BD) = m[i];
}

template <typename T>
static hipError_t la_step_t(const LaStep& a, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.rows * a.H * (a.valdim / 64)));
    if (a.keydim == 64) return launch(k_la_step<T, 64>, grid, dim3(256), s, a);
    return launch(k_la_step<T, 128>, grid, dim3(256), s, a);
}

hipError_t launch_la_step(const LaStep& a, int act, hipStream_t s) {
    return act == SSD_BF16 ? la_step_t<bf16>(a, s) : la_step_t<float>(a, s);
}

// One workgroup per (row, HB heads of a group).  Per token the workgroup convolves the heads'
// x channels and their group's B and C channels into LDS.  The ring entry of a new token is
// not read by any other workgroup of the call (they take new tokens from xBC), so one of the
// workgroups that convolve a channel writes it: the head's own for x, the one of the group's
// first head for B and C.
template <typename T, int P, int N, int HB>
__global__ void __launch_bounds__(256 * HB) k_token_step(TokenStep a) {
    constexpr int LPR = N / 4, RPW = 64 / LPR;
    constexpr int HT = P * LPR < 256 ? P * LPR : 256;  // threads of a head
    constexpr int NT = HB * HT, NW = HT / 64, NR = P / (NW * RPW);
    static_assert(NW * RPW * NR == P, "the waves' rows tile the head");
    __shared__ float sx[HB * P], sB[N], sC[N];
    const int lane = threadIdx.x % 64, col = 4 * (lane % LPR);
    const int per = a.H / HB, row = blockIdx.x / per, h0 = blockIdx.x % per * HB;
    const int hs = __builtin_amdgcn_readfirstlane(threadIdx.x / HT), h = h0 + hs;
    const int64_t slot = row_slot(a.slots, a.positions, a.nslots, row);
    if (slot < 0) return;
    const int hpg = a.H / a.G, g = h / hpg;
    const int64_t pos = a.positions[row];
    const int d0 = wave_id() % NW * RPW * NR + lane / LPR;
    float* S = a.state + ((slot * a.H + h) * P + d0) * N + col;
    f32x4 m[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
        m[i] = pos == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : *(const f32x4*)(S + i * RPW * N);
    if (row_taken(a.slots, a.positions, slot, row, lane)) return;  // the whole workgroup
    const float A = -expf(a.A_log[h]), bias = a.dt_bias[h], Dh = a.D[h];
    T* ring = (T*)a.ring + slot * a.R * a.C;
    for (int t = 0; t < a.tokens; ++t) {
        const int64_t tok = (int64_t)row * a.tokens + t;
        const T* xr = (const T*)a.xBC + tok * a.C;
        if (t > 0) __syncthreads();
        for (int i = threadIdx.x; i < HB * P + 2 * N; i += NT) {
            const int c = i < HB * P ? h0 * P + i
                                     : (i < HB * P + N ? a.H * P + g * N + (i - HB * P)
                                                       : a.H * P + (a.G + g) * N + (i - HB * P - N));
            const T now = xr[c];
            const float* w = a.conv_w + (int64_t)c * a.W;
            float u = w[a.W - 1] * (float)now;
            for (int back = 1; back < a.W; ++back) {
                const int64_t src = pos + t - back;
                if (src < 0) break;
                const float xv = back <= t ? (float)xr[c - back * a.C]
                                           : (float)ring[(src % a.R) * a.C + c];
                u += w[a.W - 1 - back] * xv;
            }
            u = u * __builtin_amdgcn_rcpf(1.f + __expf(-u));
            (i < HB * P ? sx[i] : (i < HB * P + N ? sB[i - HB * P] : sC[i - HB * P - N])) = u;
            if (i < HB * P || h0 == g * hpg) ring[((pos + t) % a.R) * a.C + c] = now;
        }
        const float raw = (float)((const T*)a.dt_raw)[tok * a.H + h];
        const float dt = fminf(fmaxf(softplus_f(raw + bias), a.dt_min), a.dt_max);
        const float keep = expf(dt * A);
        __syncthreads();
        const f32x4 B = *(const f32x4*)(sB + col), C = *(const f32x4*)(sC + col);
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float x = sx[hs * P + d0 + i * RPW];
            m[i] = m[i] * keep + B * (dt * x);
            const f32x4 p = m[i] * C;
            const float o = lanes_sum<LPR>((p[0] + p[1]) + (p[2] + p[3])) + Dh * x;
            if (lane % LPR == i) mine = o;
        }
        if (lane % LPR < NR)
            ((T*)a.y)[(tok * a.H + h) * P + d0 + (lane % LPR) * RPW] = (T)mine;
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) *(f32x4*)(S + i * RPW * N) = m[i];
}

template <typename T, int P, int N>
static hipError_t token_step_shape(const TokenStep& a, hipStream_t s) {
    constexpr int HT = P * N / 4 < 256 ? P * N / 4 : 256;
    const int64_t blocks = (int64_t)a.rows * a.H;
    // Two heads to a workgroup share the convolved B and C (237 -> 224 us for 256
    // rows of 64 heads of 64 x 128 in 8 groups); with few workgroups
    // they only leave CUs idle.
    if (a.H / a.G % 2 == 0 && blocks >= 2048)
        return launch(k_token_step<T, P, N, 2>, dim3((unsigned)(blocks / 2)), dim3(2 * HT), s, a);
    return launch(k_token_step<T, P, N, 1>, dim3((unsigned)blocks), dim3(HT), s, a);
}

hipError_t launch_token_step(const TokenStep& a, int act, hipStream_t s) {
#define SSD_STEP(TT, PP, NN) \
    if (a.P == PP && a.N == NN) return token_step_shape<TT, PP, NN>(a, s);
#define SSD_STEP_F32(PP, NN) SSD_STEP(float, PP, NN)
#define SSD_STEP_BF16(PP, NN) SSD_STEP(bf16, PP, NN)
    if (act == SSD_F32) {
        SSD_F32_SHAPES(SSD_STEP_F32)
    } else {
        SSD_BF16_SHAPES(SSD_STEP_BF16)
    }
#undef SSD_STEP_F32
#undef SSD_STEP_BF16
#undef SSD_STEP
    return hipErrorInvalidValue;
}

}  // namespace ssd
