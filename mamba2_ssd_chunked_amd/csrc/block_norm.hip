// The norms around a block with its gate and residual scale (include/ssd_layer.h).
//
//   u = norm(y) w1 + b1,  m = u act(z),  r = alpha x + scale m,  h = norm(r) w2 + b2
// Backward, with G the whole gradient of r and n = norm(.):
//   e = dh w2,  G = dr + rstd (e - [center] mean(e) - n mean(e n)),  dx = alpha G,  dm = scale G
//   dz = dm u act'(z),  du = dm act(z),  dy as G's second term with y, du w1 for r, e
//   dw2 = sum dh n(r),  db2 = sum dh,  dscale = sum G m,  dw1 = sum du n(y),  db1 = sum du
//
// Bound by HBM: every tensor is read or written once.  A workgroup holds a row in registers, EL
// channels to a thread, between its statistics and its outputs; in the backward it goes over
// several rows and keeps the five sums of its channels in registers, which a second launch adds up
// in a fixed order.
#include "layer_internal.h"

namespace ssd {

__device__ __forceinline__ float bn_sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.f + __expf(-v));
}

// act(z) and, if asked for, its derivative.
__device__ __forceinline__ float bn_gate(int kind, float z, float* d) {
    if (kind == SSD_GATE_LINEAR) {
        if (d) *d = 1.f;
        return z;
    }
    const float s = bn_sigmoid(z);
    if (kind == SSD_GATE_SIGMOID) {
        if (d) *d = s * (1.f - s);
        return s;
    }
    if (d) *d = s * (1.f + z * (1.f - s));
    return z * s;
}

// The channels of thread `tid` of THR: EL in vectors of 8 (VEC) or one by one, neighbouring threads
// side by side.
template <int EL, bool VEC>
struct BnMap {
    int tid, thr, C;
    __device__ __forceinline__ int channel(int e) const {
        return VEC ? ((e / 8) * thr + tid) * 8 + e % 8 : e * thr + tid;
    }
    // 0 where there is no channel
    template <typename T>
    __device__ __forceinline__ void load(const T* p, float (&v)[EL]) const {
        if constexpr (VEC) {
            typedef typename Vec4<T>::type v4;
            typedef T v8 __attribute__((ext_vector_type(8)));
#pragma unroll
            for (int e = 0; e < EL; e += 8) {
                const int c = channel(e);
                v8 x = {};
                if (c < C) {
                    if constexpr (sizeof(T) == 2) {
                        x = *(const v8*)(p + c);
                    } else {
                        const v4 a = *(const v4*)(p + c), b = *(const v4*)(p + c + 4);
                        x = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[e + i] = (float)x[i];
            }
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) v[e] = channel(e) < C ? (float)p[channel(e)] : 0.f;
        }
    }
    __device__ __forceinline__ void load_or(const float* p, float other, float (&v)[EL]) const {
        if (p) {
            load(p, v);
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) v[e] = other;
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* p, const float (&v)[EL]) const {
        if constexpr (VEC) {
            typedef typename Vec4<T>::type v4;
            typedef T v8 __attribute__((ext_vector_type(8)));
#pragma unroll
            for (int e = 0; e < EL; e += 8) {
                const int c = channel(e);
                if (c >= C) continue;
                v8 x;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = (T)v[e + i];
                if constexpr (sizeof(T) == 2) {
                    *(v8*)(p + c) = x;
                } else {
                    *(v4*)(p + c) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
                    *(v4*)(p + c + 4) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e)
                if (channel(e) < C) p[channel(e)] = (T)v[e];
        }
    }
};

// Sums of a and b over the workgroup, the same for all threads.
__device__ __forceinline__ void bn_sum2(float& a, float& b, float* red) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        a += __shfl_xor(a, o, 64);
        b += __shfl_xor(b, o, 64);
    }
    const int waves = blockDim.x / 64;
    if (waves == 1) return;
    __syncthreads();  // the last sums are read
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = a, red[8 + threadIdx.x / 64] = b;
    __syncthreads();
    a = b = 0.f;
    for (int w = 0; w < waves; ++w) a += red[w], b += red[8 + w];
}

// n = norm(v) in place of v; returns 1 / deviation.  Channels beyond C stay 0.
template <int EL, bool VEC>
__device__ __forceinline__ float bn_norm(const BnMap<EL, VEC>& m, float (&v)[EL], int center, float eps,
                                         float* red) {
    const float inv = 1.f / (float)m.C;
    float s = 0.f, q = 0.f, none = 0.f;
    if (center) {
#pragma unroll
        for (int e = 0; e < EL; ++e) s += v[e];
        bn_sum2(s, none, red);
        s *= inv;
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = m.channel(e) < m.C ? v[e] - s : 0.f;
    }
    none = 0.f;
#pragma unroll
    for (int e = 0; e < EL; ++e) q += v[e] * v[e];
    bn_sum2(q, none, red);
    const float rstd = 1.f / sqrtf(q * inv + eps);
#pragma unroll
    for (int e = 0; e < EL; ++e) v[e] *= rstd;
    return rstd;
}

// Gradient of norm's input from that of its output, in place.
template <int EL, bool VEC>
__device__ __forceinline__ void bn_back(const BnMap<EL, VEC>& m, float (&g)[EL], const float (&n)[EL],
                                        float rstd, int center, float* red) {
    const float inv = 1.f / (float)m.C;
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int e = 0; e < EL; ++e) s += g[e], q += g[e] * n[e];
    bn_sum2(s, q, red);
    s = center ? s * inv : 0.f;
    q *= inv;
#pragma unroll
    for (int e = 0; e < EL; ++e) g[e] = rstd * (g[e] - s - n[e] * q);
}

template <typename T, typename R, int EL, bool VEC>
__global__ void __launch_bounds__(512) k_block_fwd(BlockArgs a) {
    __shared__ float red[16];
    const BnMap<EL, VEC> m = {(int)threadIdx.x, (int)blockDim.x, a.C};
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float u[EL], v[EL], w[EL];
        m.load((const T*)a.y + row * a.ys, u);
        m.load((const R*)a.x + row * a.xs, v);
        if (a.gate) m.load((const T*)a.z + row * a.zs, w);
        if (a.post) {
            bn_norm(m, u, a.center, a.eps, red);
            float p[EL];
            m.load(a.w1, p);
#pragma unroll
            for (int e = 0; e < EL; ++e) u[e] *= p[e];
            if (a.b1) {
                m.load(a.b1, p);
#pragma unroll
                for (int e = 0; e < EL; ++e) u[e] += p[e];
            }
        }
        if (a.gate)
#pragma unroll
            for (int e = 0; e < EL; ++e) u[e] *= bn_gate(a.gate, w[e], nullptr);
        m.load_or(a.scale, 1.f, w);
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = a.alpha * v[e] + w[e] * u[e];
        m.store((R*)a.r + row * a.rs, v);
        if (a.pre) {
            bn_norm(m, v, a.center, a.eps, red);
            m.load(a.w2, w);
#pragma unroll
            for (int e = 0; e < EL; ++e) v[e] *= w[e];
            if (a.b2) {
                m.load(a.b2, w);
#pragma unroll
                for (int e = 0; e < EL; ++e) v[e] += w[e];
            }
            m.store((T*)a.h + row * a.hs, v);
        }
    }
}

// part: [workgroup][5][C] sums of dscale, dw1, db1, dw2, db2.
template <typename T, typename R, int EL, bool VEC>
__global__ void __launch_bounds__(512) k_block_bwd(BlockArgs a, float* __restrict__ part) {
    __shared__ float red[16];
    const BnMap<EL, VEC> m = {(int)threadIdx.x, (int)blockDim.x, a.C};
    float ds[EL], dw1[EL], db1[EL], dw2[EL], db2[EL];
#pragma unroll
    for (int e = 0; e < EL; ++e) ds[e] = dw1[e] = db1[e] = dw2[e] = db2[e] = 0.f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float n[EL], u[EL], z[EL], v[EL], G[EL], s[EL], t[EL];
        m.load((const T*)a.y + row * a.ys, n);
        m.load((const R*)a.x + row * a.xs, v);
        if (a.gate) m.load((const T*)a.z + row * a.zs, z);
        if (a.dr) {
            m.load((const R*)a.dr + row * a.rs, G);
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) G[e] = 0.f;
        }
        if (a.pre) m.load((const T*)a.dh + row * a.hs, t);
        float rstd1 = 0.f;
        if (a.post) {
            rstd1 = bn_norm(m, n, a.center, a.eps, red);
            m.load(a.w1, u);
#pragma unroll
            for (int e = 0; e < EL; ++e) u[e] *= n[e];
            if (a.b1) {
                m.load(a.b1, s);
#pragma unroll
                for (int e = 0; e < EL; ++e) u[e] += s[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e) u[e] = n[e];
        }
        m.load_or(a.scale, 1.f, s);
        if (a.pre) {
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                const float f = a.gate ? bn_gate(a.gate, z[e], nullptr) : 1.f;
                v[e] = a.alpha * v[e] + s[e] * (u[e] * f);
            }
            const float rstd = bn_norm(m, v, a.center, a.eps, red);
#pragma unroll
            for (int e = 0; e < EL; ++e) dw2[e] += t[e] * v[e], db2[e] += t[e];
            float w[EL];
            m.load(a.w2, w);
#pragma unroll
            for (int e = 0; e < EL; ++e) t[e] *= w[e];
            bn_back(m, t, v, rstd, a.center, red);
#pragma unroll
            for (int e = 0; e < EL; ++e) G[e] += t[e];
        }
#pragma unroll
        for (int e = 0; e < EL; ++e) t[e] = a.alpha * G[e];
        m.store((R*)a.dx + row * a.dxs, t);
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            float f = 1.f, d = 0.f;
            if (a.gate) f = bn_gate(a.gate, z[e], &d);
            ds[e] += G[e] * (u[e] * f);
            const float dm = s[e] * G[e];
            z[e] = dm * u[e] * d;
            t[e] = dm * f;
        }
        if (a.gate) m.store((T*)a.dz + row * a.dzs, z);
        if (a.post) {
#pragma unroll
            for (int e = 0; e < EL; ++e) dw1[e] += t[e] * n[e], db1[e] += t[e];
            m.load(a.w1, u);
#pragma unroll
            for (int e = 0; e < EL; ++e) t[e] *= u[e];
            bn_back(m, t, n, rstd1, a.center, red);
        }
        m.store((T*)a.dy + row * a.dys, t);
    }
    const BnMap<EL, VEC>& c = m;
    float* p = part + (int64_t)blockIdx.x * 5 * a.C;
#pragma unroll
    for (int e = 0; e < EL; ++e)
        if (c.channel(e) < a.C) {
            float* q = p + c.channel(e);
            q[0] = ds[e];
            q[a.C] = dw1[e];
            q[2 * a.C] = db1[e];
            q[3 * a.C] = dw2[e];
            q[4 * a.C] = db2[e];
        }
}

// Adds up `n` workgroups' sums: 64 columns to a workgroup, its four waves a quarter of them each.
__global__ void __launch_bounds__(256) k_block_sums(BlockArgs a, const float* __restrict__ part, int n) {
    __shared__ float red[4][64];
    const int w = threadIdx.x / 64, lane = threadIdx.x % 64, all = 5 * a.C;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < all) {
        const int q = (n + 3) / 4, end = (w + 1) * q < n ? (w + 1) * q : n;
        for (int i = w * q; i < end; ++i) s += part[(int64_t)i * all + c];
    }
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < all) {
        float* const out[5] = {a.dscale, a.dw1, a.db1, a.dw2, a.db2};
        float* p = c / a.C == 0 ? out[0] : (c / a.C == 1 ? out[1] : (c / a.C == 2 ? out[2] : (c / a.C == 3 ? out[3] : out[4])));
        if (p) p[c % a.C] = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
    }
}

// Workgroups of the backward: enough to fill the CUs four times over, and few enough that their sums
// are a small part of the traffic.
static int bwd_blocks(const BlockArgs& a) { return (int)(a.rows < 1024 ? a.rows : 1024); }
size_t block_bwd_ws(const BlockArgs& a) { return align256((size_t)bwd_blocks(a) * 5 * a.C * 4); }

// Whether all rows can be read and written in vectors of 8 channels.
static bool vectors(const BlockArgs& a, int act, int res) {
    auto ok = [](const void* p, int64_t stride, int esz) {
        return !p || (((uintptr_t)p | (uintptr_t)(stride * esz)) & 15) == 0;
    };
    const int e = act == SSD_BF16 ? 2 : 4, f = res == SSD_BF16 ? 2 : 4;
    if (a.C % 8 != 0) return false;
    for (const float* p : {a.scale, a.w1, a.b1, a.w2, a.b2})
        if (!ok(p, 0, 4)) return false;
    return ok(a.x, a.xs, f) && ok(a.y, a.ys, e) && ok(a.z, a.zs, e) && ok(a.r, a.rs, f) && ok(a.dr, a.rs, f) &&
           ok(a.h, a.hs, e) && ok(a.dh, a.hs, e) && ok(a.dx, a.dxs, f) && ok(a.dy, a.dys, e) && ok(a.dz, a.dzs, e);
}

template <typename T, typename R, int EL, bool VEC>
static hipError_t go(const BlockArgs& a, float* part, int threads, hipStream_t s) {
    if (!part) {
        const int64_t blocks = a.rows < (1 << 22) ? a.rows : (1 << 22);
        return launch(k_block_fwd<T, R, EL, VEC>, dim3((unsigned)blocks), dim3(threads), s, a);
    }
    const int n = bwd_blocks(a);
    SSD_TRY(launch(k_block_bwd<T, R, EL, VEC>, dim3(n), dim3(threads), s, a, part));
    return launch(k_block_sums, dim3((5 * a.C + 63) / 64), dim3(256), s, a, part, n);
}

// 8 channels to a thread up to 512 threads, then 16 and 32.
template <typename T, typename R, bool VEC>
static hipError_t width(const BlockArgs& a, float* part, hipStream_t s) {
    const int threads = (a.C + 511) / 512 * 64;
    if (threads <= 512) return go<T, R, 8, VEC>(a, part, threads, s);
    if (threads <= 1024) return go<T, R, 16, VEC>(a, part, 512, s);
    return go<T, R, 32, VEC>(a, part, 512, s);
}
static hipError_t types(const BlockArgs& a, int act, int res, float* part, hipStream_t s) {
    const bool v = vectors(a, act, res);
    if (act == SSD_F32) return v ? width<float, float, true>(a, part, s) : width<float, float, false>(a, part, s);
    if (res == SSD_F32) return v ? width<bf16, float, true>(a, part, s) : width<bf16, float, false>(a, part, s);
    return v ? width<bf16, bf16, true>(a, part, s) : width<bf16, bf16, false>(a, part, s);
}

hipError_t launch_block_fwd(const BlockArgs& a, int act, int res, hipStream_t s) {
    return types(a, act, res, nullptr, s);
}
hipError_t launch_block_bwd(const BlockArgs& a, int act, int res, float* part, hipStream_t s) {
    return types(a, act, res, part, s);
}

}  // namespace ssd
