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
// in a fixed order.  16384 rows of 2048 bf16 channels with a float32 residual: forward 100 us, 4.7 TB/s; backward
// 203 us, 3.6 TB/s of its 740 MB, since a row's loads do not overlap the sums of the one before (below), and the
// second launch 13 us.  Its sums are what a thread's registers allow, 128 with 1024 threads: four channels a thread.
// Rows of more than 4096 channels have 8 or 16 and spill in the backward, without vectors in the forward too: 16384 x
// 5120 235 and 1138 us (one channel at a time 841 and 3073), 8192 x 10240 319 and 3916 (1764 and 21788).
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

// The channels of thread `tid` of THR: EL in vectors of 4 (VEC) or one by one, neighbouring threads
// side by side.
template <int EL, bool VEC>
struct BnMap {
    int tid, thr, C;
    float inv;  // 1 / C
    __device__ __forceinline__ int channel(int e) const {
        return VEC ? ((e / 4) * thr + tid) * 4 + e % 4 : e * thr + tid;
    }
    // a load in two steps: the raw values on their way, then as float32
    template <typename T>
    struct Raw {
        typename Vec4<T>::type v[VEC ? EL / 4 : 1];
    };
    template <typename T>
    __device__ __forceinline__ void ask(const T* p, Raw<T>& r) const {
#pragma unroll
        for (int e = 0; e < EL; e += 4) {
            typename Vec4<T>::type x = {};
            if (channel(e) < C) x = *(const typename Vec4<T>::type*)(p + channel(e));
            r.v[e / 4] = x;
        }
    }
    template <typename T>
    __device__ __forceinline__ void take(const Raw<T>& r, float (&v)[EL]) const {
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = (float)r.v[e / 4][e % 4];
    }
    // 0 where there is no channel
    template <typename T>
    __device__ __forceinline__ void load(const T* p, float (&v)[EL]) const {
        if constexpr (VEC) {
            typedef typename Vec4<T>::type v4;
#pragma unroll
            for (int e = 0; e < EL; e += 4) {
                const int c = channel(e);
                v4 x = {};
                if (c < C) x = *(const v4*)(p + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[e + i] = (float)x[i];
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
#pragma unroll
            for (int e = 0; e < EL; e += 4)
                if (channel(e) < C)
                    *(v4*)(p + channel(e)) = v4{(T)v[e], (T)v[e + 1], (T)v[e + 2], (T)v[e + 3]};
        } else {
#pragma unroll
            for (int e = 0; e < EL; ++e)
                if (channel(e) < C) p[channel(e)] = (T)v[e];
        }
    }
};

// Sum over the wave, the same for all lanes, without a trip through LDS.
__device__ __forceinline__ float bn_wave_sum(float v) {
    auto dpp = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    v += dpp(v, std::integral_constant<int, 0xb1>{});   // lanes 1 0 3 2 of four
    v += dpp(v, std::integral_constant<int, 0x4e>{});   // 2 3 0 1
    v += dpp(v, std::integral_constant<int, 0x141>{});  // eight mirrored
    v += dpp(v, std::integral_constant<int, 0x140>{});  // sixteen mirrored
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Sums over the workgroup, the same for all threads.
template <int N>
__device__ __forceinline__ void bn_sum(float (&v)[N], float (*red)[16]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = bn_wave_sum(v[i]);
    const int waves = blockDim.x / 64;
    if (waves == 1) return;
    __syncthreads();  // the last sums are read
    if (threadIdx.x % 64 == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[i][threadIdx.x / 64] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const f32x4* r = (const f32x4*)red[i];
        f32x4 s = r[0];
        for (int w = 4; w < waves; w += 4) s += r[w / 4];  // zeros behind the last wave
        v[i] = (s[0] + s[1]) + (s[2] + s[3]);
    }
}

// n = norm(v) in place of v; returns 1 / deviation.  Channels beyond C stay 0.
template <int EL, bool VEC>
__device__ __forceinline__ float bn_norm(const BnMap<EL, VEC>& m, float (&v)[EL], int center, float eps,
                                         float (*red)[16]) {
    if (center) {
        float s[1] = {0.f};
#pragma unroll
        for (int e = 0; e < EL; ++e) s[0] += v[e];
        bn_sum(s, red);
        s[0] *= m.inv;
#pragma unroll
        for (int e = 0; e < EL; ++e) v[e] = m.channel(e) < m.C ? v[e] - s[0] : 0.f;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int e = 0; e < EL; ++e) q[0] += v[e] * v[e];
    bn_sum(q, red);
    const float rstd = 1.f / sqrtf(q[0] * m.inv + eps);
#pragma unroll
    for (int e = 0; e < EL; ++e) v[e] *= rstd;
    return rstd;
}

// Gradient of norm's input from that of its output, in place.
template <int EL, bool VEC>
__device__ __forceinline__ void bn_back(const BnMap<EL, VEC>& m, float (&g)[EL], const float (&n)[EL],
                                        float rstd, int center, float (*red)[16]) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < EL; ++e) s[0] += g[e] * n[e], s[1] += g[e];
    if (center) {
        bn_sum(s, red);
    } else {
        float q[1] = {s[0]};
        bn_sum(q, red);
        s[0] = q[0], s[1] = 0.f;
    }
    s[0] *= m.inv, s[1] *= m.inv;
#pragma unroll
    for (int e = 0; e < EL; ++e) g[e] = rstd * (g[e] - s[1] - n[e] * s[0]);
}

template <typename T, typename R, int EL, bool VEC>
__global__ void __launch_bounds__(1024) k_block_fwd(BlockArgs a) {
    __shared__ __align__(16) float red[2][16];
    if (threadIdx.x < 32) red[threadIdx.x / 16][threadIdx.x % 16] = 0.f;
    __syncthreads();
    const BnMap<EL, VEC> m = {(int)threadIdx.x, (int)blockDim.x, a.C, 1.f / (float)a.C};
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
__global__ void __launch_bounds__(1024) k_block_bwd(BlockArgs a, float* __restrict__ part) {
    __shared__ __align__(16) float red[2][16];
    if (threadIdx.x < 32) red[threadIdx.x / 16][threadIdx.x % 16] = 0.f;
    __syncthreads();
    const BnMap<EL, VEC> m = {(int)threadIdx.x, (int)blockDim.x, a.C, 1.f / (float)a.C};
    float ds[EL], dw1[EL], db1[EL], dw2[EL], db2[EL];
#pragma unroll
    for (int e = 0; e < EL; ++e) ds[e] = dw1[e] = db1[e] = dw2[e] = db2[e] = 0.f;
    // Where registers allow, the next row is asked for before one is computed.  The loads' conditions (channels
    // beyond the row, a gate) leave the compiler no count of them, so that it waits for all before the first sum; it was
    // 237 us without and 221 so all the same.  The last row is asked for twice.
    constexpr bool AHEAD = VEC && EL == 4;
    typename BnMap<EL, VEC>::template Raw<T> ry, rz, rh;
    typename BnMap<EL, VEC>::template Raw<R> rx, rr;
    auto ask = [&](int64_t row) {
        if constexpr (AHEAD) {
            m.ask((const T*)a.y + row * a.ys, ry);
            m.ask((const R*)a.x + row * a.xs, rx);
            if (a.gate) m.ask((const T*)a.z + row * a.zs, rz);
            if (a.dr) m.ask((const R*)a.dr + row * a.rs, rr);
            if (a.pre) m.ask((const T*)a.dh + row * a.hs, rh);
        }
    };
    ask(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float n[EL], u[EL], z[EL], v[EL], G[EL], s[EL], t[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) G[e] = 0.f;
        if constexpr (AHEAD) {
            m.take(ry, n);
            m.take(rx, v);
            if (a.gate) m.take(rz, z);
            if (a.dr) m.take(rr, G);
            if (a.pre) m.take(rh, t);
            ask(row + gridDim.x < a.rows ? row + gridDim.x : row);  // the last row again: nobody takes it
        } else {
            m.load((const T*)a.y + row * a.ys, n);
            m.load((const R*)a.x + row * a.xs, v);
            if (a.gate) m.load((const T*)a.z + row * a.zs, z);
            if (a.dr) m.load((const R*)a.dr + row * a.rs, G);
            if (a.pre) m.load((const T*)a.dh + row * a.hs, t);
        }
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
        float f[EL];  // act(z); z becomes its derivative times u
#pragma unroll
        for (int e = 0; e < EL; ++e) {
            float d = 0.f;
            f[e] = 1.f;
            if (a.gate) f[e] = bn_gate(a.gate, z[e], &d);
            z[e] = d * u[e];
            u[e] *= f[e];
        }
        if (a.pre) {
#pragma unroll
            for (int e = 0; e < EL; ++e) v[e] = a.alpha * v[e] + s[e] * u[e];
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
            ds[e] += G[e] * u[e];
            const float dm = s[e] * G[e];
            z[e] *= dm;
            t[e] = dm * f[e];
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

// Adds up `n` workgroups' sums: 16 columns to a workgroup, whose 16 groups of lanes take every 16th of them
// (64 columns, a quarter of the sums to a wave: 81 us for 1024 of 5 x 2048).
__global__ void __launch_bounds__(256) k_block_sums(BlockArgs a, const float* __restrict__ part, int n) {
    __shared__ float red[16][17];
    const int g = threadIdx.x / 16, lane = threadIdx.x % 16, all = 5 * a.C;
    const int c = blockIdx.x * 16 + lane;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < all)
        for (int i = g; i < n; i += 128)
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i + 16 * u < n) s[u] += part[(int64_t)(i + 16 * u) * all + c];
    red[g][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    if (g == 0 && c < all) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += red[i][lane];
        float* const out[5] = {a.dscale, a.dw1, a.db1, a.dw2, a.db2};
        float* p = c / a.C == 0 ? out[0] : (c / a.C == 1 ? out[1] : (c / a.C == 2 ? out[2] : (c / a.C == 3 ? out[3] : out[4])));
        if (p) p[c % a.C] = v;
    }
}

static int block_threads(int C) {  // 4 channels to each, 8 or 16 where 1024 are not enough
    const int t = (C + 255) / 256 * 64;
    return t <= 1024 ? t : (t <= 2048 ? (t / 2 + 63) / 64 * 64 : 1024);
}
// Workgroups of the backward: as many as the CUs hold at once (1024 threads each), so that their sums are a
// small part of the traffic.
static int bwd_blocks(const BlockArgs& a) {
    const int64_t n = 256 * 1024 / block_threads(a.C);
    return (int)(a.rows < n ? a.rows : n);
}
size_t block_bwd_ws(const BlockArgs& a) { return align256((size_t)bwd_blocks(a) * 5 * a.C * 4); }

// Whether all rows can be read and written in vectors of 4 channels.
static bool vectors(const BlockArgs& a, int act, int res) {
    auto ok = [](const void* p, int64_t stride, int esz) {
        return !p || (((uintptr_t)p | (uintptr_t)(stride * esz)) & (4 * esz - 1)) == 0;
    };
    const int e = act == SSD_BF16 ? 2 : 4, f = res == SSD_BF16 ? 2 : 4;
    if (a.C % 4 != 0) return false;
    for (const float* p : {a.scale, a.w1, a.b1, a.w2, a.b2})
        if (!ok(p, 0, 4)) return false;
    return ok(a.x, a.xs, f) && ok(a.y, a.ys, e) && ok(a.z, a.zs, e) && ok(a.r, a.rs, f) && ok(a.dr, a.rs, f) &&
           ok(a.h, a.hs, e) && ok(a.dh, a.hs, e) && ok(a.dx, a.dxs, f) && ok(a.dy, a.dys, e) && ok(a.dz, a.dzs, e);
}

template <typename T, typename R, int EL, bool VEC>
static hipError_t go(const BlockArgs& a, float* part, int threads, hipStream_t s) {
    if (!part) {
        const int64_t blocks = a.rows < (1 << 21) ? a.rows : (1 << 21);
        return launch(k_block_fwd<T, R, EL, VEC>, dim3((unsigned)blocks), dim3(threads), s, a);
    }
    const int n = bwd_blocks(a);
    SSD_TRY(launch(k_block_bwd<T, R, EL, VEC>, dim3(n), dim3(threads), s, a, part));
    return launch(k_block_sums, dim3((5 * a.C + 15) / 16), dim3(256), s, a, part, n);
}

// (8 channels to a thread from the start take 128 registers and more in the backward: 300 us for 16384 rows
// of 2048, 255 with 4.)
template <typename T, typename R, bool VEC>
static hipError_t width(const BlockArgs& a, float* part, hipStream_t s) {
    const int threads = block_threads(a.C);
    if (a.C <= 4 * threads) return go<T, R, 4, VEC>(a, part, threads, s);
    if (a.C <= 8 * threads) return go<T, R, 8, VEC>(a, part, threads, s);
    return go<T, R, 16, VEC>(a, part, threads, s);
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
