// Group norm with an activation, channels last: forward and backward.
//
// With s the gate's SiLU and u = x s (gated before) or x:
//   n = (u - m) r,  r = 1 / sqrt(mean((u - m)^2) + eps),  lin = n w + b
//   y = lin, silu(lin) or lin s
// Backward, with e the gradient that reaches lin, g = e w:
//   du = r (g - [center] mean(g) - n mean(g n));  dw = sum e n, db = sum e.
//
// Bound by HBM: x, z (and dy) read once, y (dx, dz) written once.  A group of a row is held
// in registers by a team of lanes between its statistics and its outputs; a team keeps one
// group for all its rows, so that weight and bias, and the sums of dweight and dbias, stay
// in registers too (16384 rows of 2048 bf16 channels, gated before: 39 to 42 us forward, 4.7 to 5.1
// TB/s; 76 us backward, 4.5 TB/s).  Groups too wide for a team take the kernels that read a group again for
// every sweep (k_norm_*_any).
#include "mixer_internal.h"

namespace ssd {

__device__ __forceinline__ float sigm(float v) {
    return __builtin_amdgcn_rcpf(1.f + __expf(-v));
}

// Sum of v over the 256 threads, the same value for all.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    __syncthreads();
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// One workgroup per (row, group), the group's channels read again for every sweep.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_fwd_any(NormArgs a) {
    __shared__ float red[4];
    const int64_t items = a.rows * a.G;
    const float inv = 1.f / (float)a.gs;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t row = it / a.G;
        const int c0 = (int)(it % a.G) * a.gs;
        const T* x = (const T*)a.x + row * a.xs + c0;
        const T* z = (const T*)a.z + row * a.zs + c0;
        T* y = (T*)a.y + row * a.ys + c0;
        auto u = [&](int i) {
            float v = (float)x[i];
            if (a.mode == SSD_NORM_BEFORE) {
                const float zv = (float)z[i];
                v *= zv * sigm(zv);
            }
            return v;
        };
        float m = 0.f, q = 0.f;
        if (a.center) {
            for (int i = threadIdx.x; i < a.gs; i += 256) m += u(i);
            m = block_sum(m, red) * inv;
        }
        for (int i = threadIdx.x; i < a.gs; i += 256) {
            const float d = u(i) - m;
            q += d * d;
        }
        const float r = rsqrtf(block_sum(q, red) * inv + a.eps);
        for (int i = threadIdx.x; i < a.gs; i += 256) {
            float v = (u(i) - m) * r * a.w[c0 + i] + (a.b ? a.b[c0 + i] : 0.f);
            if (a.mode == SSD_NORM_SILU) v *= sigm(v);
            if (a.mode == SSD_NORM_AFTER) {
                const float zv = (float)z[i];
                v *= zv * sigm(zv);
            }
            y[i] = (T)v;
        }
    }
}

// Workgroup (block, group): rows block, block + blocks, ...; its partial sums of dw and
// db go to row `block` of part ([blocks][2][C]).
template <typename T>
__global__ void __launch_bounds__(256) k_norm_bwd_any(NormArgs a, float* __restrict__ part) {
    __shared__ float red[4];
    const int c0 = blockIdx.y * a.gs;
    const float inv = 1.f / (float)a.gs;
    float* pw = part + (int64_t)blockIdx.x * 2 * a.C + c0;
    float* pb = pw + a.C;
    for (int i = threadIdx.x; i < a.gs; i += 256) pw[i] = pb[i] = 0.f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = (const T*)a.x + row * a.xs + c0;
        const T* z = (const T*)a.z + row * a.zs + c0;
        const T* dy = (const T*)a.dy + row * a.ys + c0;
        T* dx = (T*)a.dx + row * a.dxs + c0;
        T* dz = (T*)a.dz + row * a.dzs + c0;
        auto u = [&](int i) {
            float v = (float)x[i];
            if (a.mode == SSD_NORM_BEFORE) {
                const float zv = (float)z[i];
                v *= zv * sigm(zv);
            }
            return v;
        };
        float m = 0.f, q = 0.f;
        if (a.center) {
            for (int i = threadIdx.x; i < a.gs; i += 256) m += u(i);
            m = block_sum(m, red) * inv;
        }
        for (int i = threadIdx.x; i < a.gs; i += 256) {
            const float d = u(i) - m;
            q += d * d;
        }
        const float r = rsqrtf(block_sum(q, red) * inv + a.eps);
        // gradient that reaches lin = n w + b at channel i
        auto grad = [&](int i, float n) {
            float e = (float)dy[i];
            if (a.mode == SSD_NORM_AFTER) {
                const float zv = (float)z[i];
                e *= zv * sigm(zv);
            } else if (a.mode == SSD_NORM_SILU) {
                const float lin = n * a.w[c0 + i] + (a.b ? a.b[c0 + i] : 0.f);
                const float sg = sigm(lin);
                e *= sg * (1.f + lin * (1.f - sg));
            }
            return e;
        };
        float sg = 0.f, sgn = 0.f;
        for (int i = threadIdx.x; i < a.gs; i += 256) {
            const float n = (u(i) - m) * r, e = grad(i, n), gw = e * a.w[c0 + i];
            sg += gw;
            sgn += gw * n;
            pw[i] += e * n;
            pb[i] += e;
        }
        sgn = block_sum(sgn, red) * inv;
        sg = a.center ? block_sum(sg, red) * inv : 0.f;
        for (int i = threadIdx.x; i < a.gs; i += 256) {
            const float n = (u(i) - m) * r, w = a.w[c0 + i];
            float du = r * (grad(i, n) * w - sg - n * sgn);
            if (a.mode >= SSD_NORM_BEFORE) {
                const float zv = (float)z[i], s = sigm(zv);
                const float ds = s * (1.f + zv * (1.f - s));
                float dzv;
                if (a.mode == SSD_NORM_BEFORE) {
                    dzv = du * (float)x[i] * ds;
                    du *= zv * s;
                } else {
                    dzv = (float)dy[i] * (n * w + (a.b ? a.b[c0 + i] : 0.f)) * ds;
                }
                dz[i] = (T)dzv;
            }
            dx[i] = (T)du;
        }
    }
}

// ---- teams --------------------------------------------------------------------------
//
// A team of `lpt` neighbouring lanes of a workgroup (a power of two; with WIDE several
// waves), holds EPL channels to a lane: vectors lane, lane + lpt, ... of the group.

constexpr int NORM_NT = 512;

// E channels at a time: 16 bytes where groups and tensors are aligned to it, otherwise two
// bf16, otherwise one channel (which still makes runs of whole cache lines for a wave).
template <typename T, int E>
struct NormVec {
    typedef T type __attribute__((ext_vector_type(E)));
};
template <typename T>
struct NormVec<T, 1> {
    struct type {
        T v;
        __device__ __forceinline__ T& operator[](int) { return v; }
        __device__ __forceinline__ const T& operator[](int) const { return v; }
    };
};

// Team sums of N values at once.  With WIDE every team of the workgroup calls it.
template <int N, bool WIDE>
__device__ __forceinline__ void team_sum(float (&v)[N], int lpt, float (*red)[NORM_NT / 64]) {
    for (int o = 1; o < (WIDE ? 64 : lpt); o <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], o, 64);
    if constexpr (WIDE) {
        __syncthreads();  // the last sums have been read
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[i][threadIdx.x / 64] = v[i];
        __syncthreads();
        const int w0 = threadIdx.x / lpt * (lpt / 64);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
        for (int k = 0; k < lpt / 64; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += red[i][w0 + k];
    }
}

// The same vector as far as the compiler knows anew: what was computed from it before is
// computed again, not held.
template <typename V>
__device__ __forceinline__ V forget(V v) {
    if constexpr (sizeof(V) == 16) {
        f32x4 h = __builtin_bit_cast(f32x4, v);
        asm volatile("" : "+v"(h));
        return __builtin_bit_cast(V, h);
    } else {
        return v;
    }
}

struct NormTeam {
    int lane, lpt;       // place in the team, its lanes
    int64_t item, step;  // first (row, group), distance to the next
    int c0, nv;          // the group's first channel and its vectors
    int turns;           // (row, group)s of the team, with WIDE of the workgroup's busiest
};
template <typename T, int E, bool WIDE>
__device__ __forceinline__ NormTeam norm_team(const NormArgs& a, int lpt) {
    NormTeam t;
    t.lpt = lpt;
    t.lane = threadIdx.x % t.lpt;
    const int per = NORM_NT / t.lpt;
    t.item = (int64_t)blockIdx.x * per + threadIdx.x / t.lpt;
    t.step = (int64_t)gridDim.x * per;  // a multiple of G: the group stays
    t.c0 = (int)(t.item % a.G) * a.gs;
    t.nv = a.gs / E;
    // the same for all teams of the workgroup, which meet in team_sum
    t.turns = (int)((a.rows * a.G - t.item + t.step - 1) / t.step);
    if (WIDE) {
        const int64_t first = (int64_t)blockIdx.x * per;
        t.turns = first < a.rows * a.G ? (int)((a.rows * a.G - first + t.step - 1) / t.step) : 0;
    }
    return t;
}

// weight or bias of the lane's channels; `otherwise` where there is none
template <int E, int EPL>
__device__ __forceinline__ void norm_params(const float* p, const NormTeam& t, float otherwise,
                                            float (&o)[EPL]) {
#pragma unroll
    for (int i = 0; i < EPL / E; ++i) {
        const int v = t.lane + i * t.lpt;
#pragma unroll
        for (int e = 0; e < E; ++e) o[i * E + e] = p && v < t.nv ? p[t.c0 + v * E + e] : otherwise;
    }
}

template <typename T, int E, int EPL>
__device__ __forceinline__ void norm_load(const T* row, const NormTeam& t,
                                          typename NormVec<T, E>::type (&o)[EPL / E]) {
    typedef typename NormVec<T, E>::type vt;
#pragma unroll
    for (int i = 0; i < EPL / E; ++i) {
        const int v = t.lane + i * t.lpt;
        o[i] = v < t.nv ? *(const vt*)(row + v * E) : vt{};
    }
}

// u, then n = (u - m) r, of the lane's channels (0 where it has none); returns r
template <typename T, int E, int EPL, int MODE, bool WIDE, bool TIGHT = false>
__device__ __forceinline__ float norm_n(const NormArgs& a, const NormTeam& t,
                                        const typename NormVec<T, E>::type (&x)[EPL / E],
                                        const typename NormVec<T, E>::type (&z)[EPL / E],
                                        float (&n)[EPL], float (*red)[NORM_NT / 64]) {
    const float inv = 1.f / (float)a.gs;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (TIGHT && i % 8 == 0) __builtin_amdgcn_sched_barrier(0);
        n[i] = (float)x[i / E][i % E];
        if (MODE == SSD_NORM_BEFORE) {
            const float zv = (float)z[i / E][i % E];
            n[i] *= zv * sigm(zv);
        }
    }
    if (a.center) {
        float m[1] = {0.f};
#pragma unroll
        for (int i = 0; i < EPL; ++i) m[0] += n[i];
        team_sum<1, WIDE>(m, t.lpt, red);
        m[0] *= inv;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (t.lane + (i / E) * t.lpt < t.nv) n[i] -= m[0];
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < EPL; ++i) q[0] += n[i] * n[i];
    team_sum<1, WIDE>(q, t.lpt, red);
    const float r = rsqrtf(q[0] * inv + a.eps);
#pragma unroll
    for (int i = 0; i < EPL; ++i) n[i] *= r;
    return r;
}

template <typename T, int E, int EPL, int MODE, bool WIDE>
__global__ void __launch_bounds__(NORM_NT) k_norm_fwd(NormArgs a, int lpt) {
    typedef typename NormVec<T, E>::type vt;
    constexpr int V = EPL / E;
    constexpr bool GATED = MODE >= SSD_NORM_BEFORE;
    __shared__ float red[1][NORM_NT / 64];
    const NormTeam t0 = norm_team<T, E, WIDE>(a, lpt);
    float w[EPL], b[EPL];
    norm_params<E, EPL>(a.w, t0, 0.f, w);
    norm_params<E, EPL>(a.b, t0, 0.f, b);
    NormTeam t = t0;
    for (int k = 0; k < t0.turns; ++k) {
        const int64_t it = t0.item + k * t0.step;
        if (WIDE && it >= a.rows * a.G) t.nv = 0;  // nothing to load or store, only to meet
        const int64_t row = WIDE && t.nv == 0 ? 0 : (uint32_t)it / (uint32_t)a.G;
        vt x[V], z[V];
        norm_load<T, E, EPL>((const T*)a.x + row * a.xs + t.c0, t, x);
        if (GATED) norm_load<T, E, EPL>((const T*)a.z + row * a.zs + t.c0, t, z);
        float n[EPL];
        norm_n<T, E, EPL, MODE, WIDE>(a, t, x, z, n, red);
        T* y = (T*)a.y + row * a.ys + t.c0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            vt o;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float v = n[i * E + e] * w[i * E + e] + b[i * E + e];
                if (MODE == SSD_NORM_SILU) v *= sigm(v);
                if (MODE == SSD_NORM_AFTER) {
                    const float zv = (float)z[i][e];
                    v *= zv * sigm(zv);
                }
                o[e] = (T)v;
            }
            if (t.lane + i * t.lpt < t.nv) *(vt*)(y + (t.lane + i * t.lpt) * E) = o;
        }
    }
}

// Partial sums of dw and db: row p of part ([np][2][C]).  Where the workgroup's teams hold
// whole sets of groups they are added in the workgroup first, team after team (`fold`).
template <typename T, int E, int EPL, int MODE, bool WIDE>
__global__ void __launch_bounds__(NORM_NT, EPL == 8 ? 4 : 2) k_norm_bwd(NormArgs a, int lpt, int fold,
                                                     float* __restrict__ part) {
    typedef typename NormVec<T, E>::type vt;
    constexpr int V = EPL / E;
    constexpr bool GATED = MODE >= SSD_NORM_BEFORE;
    __shared__ float red[2][NORM_NT / 64];
    extern __shared__ __align__(16) float sums[];  // fold
    const NormTeam t0 = norm_team<T, E, WIDE>(a, lpt);
    const float inv = 1.f / (float)a.gs;
    float w[EPL], b[MODE == SSD_NORM_SILU || MODE == SSD_NORM_AFTER ? EPL : 1];
    norm_params<E, EPL>(a.w, t0, 0.f, w);
    if constexpr (MODE == SSD_NORM_SILU || MODE == SSD_NORM_AFTER)
        norm_params<E, EPL>(a.b, t0, 0.f, b);
    float sw[EPL], sb[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) sw[i] = sb[i] = 0.f;
    NormTeam t = t0;
    for (int k = 0; k < t0.turns; ++k) {
        const int64_t it = t0.item + k * t0.step;
        if (WIDE && it >= a.rows * a.G) t.nv = 0;  // nothing to load or store, only to meet
        const int64_t row = WIDE && t.nv == 0 ? 0 : (uint32_t)it / (uint32_t)a.G;
        vt x[V], z[V], dy[V];
        norm_load<T, E, EPL>((const T*)a.x + row * a.xs + t.c0, t, x);
        if (GATED) norm_load<T, E, EPL>((const T*)a.z + row * a.zs + t.c0, t, z);
        norm_load<T, E, EPL>((const T*)a.dy + row * a.ys + t.c0, t, dy);
        float n[EPL], e[EPL];
        const float r = norm_n<T, E, EPL, MODE, WIDE, true>(a, t, x, z, n, red);
        float s[2] = {0.f, 0.f};  // sums of g n, g
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            // vector by vector: interleaved, their temporaries do not fit the registers
            if (i % 8 == 0) __builtin_amdgcn_sched_barrier(0);
            e[i] = (float)dy[i / E][i % E];
            if (MODE == SSD_NORM_AFTER) {
                const float zv = (float)z[i / E][i % E];
                e[i] *= zv * sigm(zv);
            }
            if (MODE == SSD_NORM_SILU) {
                const float lin = n[i] * w[i] + b[i];
                const float sg = sigm(lin);
                e[i] *= sg * (1.f + lin * (1.f - sg));
            }
            sw[i] += e[i] * n[i];
            sb[i] += e[i];
            e[i] *= w[i];
            s[0] += e[i] * n[i];
            s[1] += e[i];
        }
        team_sum<2, WIDE>(s, t.lpt, red);
        s[0] *= inv;
        s[1] = a.center ? s[1] * inv : 0.f;
        // at 16 channels to a lane the gate is computed again from z, not held across the sums
        if (EPL > 8)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                z[i] = forget(z[i]);
                x[i] = forget(x[i]);
                dy[i] = forget(dy[i]);
            }
        T* dx = (T*)a.dx + row * a.dxs + t.c0;
        T* dz = (T*)a.dz + row * a.dzs + t.c0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = t.lane + i * t.lpt;
            if (i * E % 8 == 0) __builtin_amdgcn_sched_barrier(0);
            vt ox, oz;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int c = i * E + j;
                float du = r * (e[c] - s[1] - n[c] * s[0]);
                if (GATED) {
                    const float zv = (float)z[i][j], g = sigm(zv);
                    const float ds = g * (1.f + zv * (1.f - g));
                    if constexpr (MODE == SSD_NORM_BEFORE) {
                        oz[j] = (T)(du * (float)x[i][j] * ds);
                        du *= zv * g;
                    } else if constexpr (MODE == SSD_NORM_AFTER) {
                        oz[j] = (T)((float)dy[i][j] * (n[c] * w[c] + b[c]) * ds);
                    }
                }
                ox[j] = (T)du;
            }
            if (v < t.nv) {
                *(vt*)(dx + v * E) = ox;
                if (GATED) *(vt*)(dz + v * E) = oz;
            }
        }
    }
    t = t0;
    const int team = threadIdx.x / t.lpt, per = NORM_NT / t.lpt;
    if (fold) {
        // [dw, db][group][quad of a lane][lane] in LDS: each access a run of 16-byte vectors
        const int gw = EPL * t.lpt, half = a.G * gw;
        f32x4* mine = (f32x4*)(sums + team % a.G * gw) + t.lane;
        for (int q = 0; q < per / a.G; ++q) {
            if (team / a.G == q) {
#pragma unroll
                for (int i = 0; i < EPL; i += 4) {
                    f32x4* p = mine + i / 4 * t.lpt;
                    f32x4 vw = {sw[i], sw[i + 1], sw[i + 2], sw[i + 3]};
                    f32x4 vb = {sb[i], sb[i + 1], sb[i + 2], sb[i + 3]};
                    if (q) vw += p[0], vb += p[half / 4];
                    p[0] = vw;
                    p[half / 4] = vb;
                }
            }
            __syncthreads();
        }
        float* p = part + (int64_t)blockIdx.x * 2 * a.C;
        for (int i = threadIdx.x; i < 2 * a.C; i += NORM_NT) {
            const int c = i % a.C, k = c % a.gs, v = k / E;  // vector v / lpt of lane v % lpt
            const int el = v / t.lpt * E + k % E;
            p[i] = sums[(i / a.C) * half + c / a.gs * gw + el / 4 * 4 * t.lpt + v % t.lpt * 4 + el % 4];
        }
    } else {
        float* p = part + ((int64_t)blockIdx.x * per + team) / a.G * 2 * a.C + t.c0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int v = t.lane + (i / E) * t.lpt;
            if (v < t.nv) {
                p[v * E + i % E] = sw[i];
                p[a.C + v * E + i % E] = sb[i];
            }
        }
    }
}

// dw and db from the partial sums, 16 rows of them side by side, each in its order.
__global__ void __launch_bounds__(1024) k_norm_reduce(const float* __restrict__ part, int np, int C,
                                                      float* __restrict__ dw,
                                                      float* __restrict__ db) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x % 64, k = threadIdx.x / 64;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < 2 * C)
#pragma unroll 8
        for (int p = k; p < np; p += 16) s += part[(int64_t)p * 2 * C + c];
    red[k][lane] = s;
    __syncthreads();
    if (k == 0 && c < 2 * C) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += red[i][lane];
        if (c < C) dw[c] = s;
        else if (db) db[c - C] = s;
    }
}

// How a problem is dealt out.
struct NormPlan {
    bool teams, wide, fold;
    int e, epl, lpt, blocks, np;  // channels at a time and of a lane, lanes of a team
};

static int64_t fold_lds(const NormArgs& a, const NormPlan& p) {
    return 2ll * a.G * p.epl * p.lpt * 4;
}

static int gcd_of(int a, int b) {
    while (b) {
        const int r = a % b;
        a = b;
        b = r;
    }
    return a;
}

// `e`: the channels at a time that the tensors' alignment allows
static NormPlan norm_plan(const NormArgs& a, bool bwd, int e) {
    NormPlan p = {};
    p.e = e;
    const int64_t items = a.rows * a.G;
    // The fewest lanes that hold the group, at 8, 16 or 32 channels to a lane.  Forward: many,
    // for bytes on their way and sums within a wave (16 channels of bf16 in two vectors rather
    // than 8 in one: 36 -> 19 us for 8192 rows of 32 groups of 64); with one channel at a time
    // 8, whose loads are as many.
    // Backward: 8 wherever 512 lanes hold the group, since it keeps five values of each
    // channel (16384 rows of 2048 bf16 channels: 74 us at 8, 190 at 16 and 228 at 32).  Wider groups
    // pay for it: 151 us for 4096 channels, 289 for 5120, 783 for 10240, whose 32 channels
    // to a lane spill.
    p.teams = a.gs <= 32 * NORM_NT;
    if (bwd || e == 1) p.epl = a.gs <= 8 * NORM_NT ? 8 : (a.gs <= 16 * NORM_NT ? 16 : 32);
    else p.epl = a.gs <= (e == 8 ? 8 : 8 * 64) ? 8 : (a.gs <= 16 * 64 ? 16 : 32);
    p.lpt = 1;
    while (p.lpt < NORM_NT && p.lpt * p.epl < a.gs) p.lpt *= 2;
    p.wide = p.lpt > 64;
    const int per = NORM_NT / p.lpt;          // teams per workgroup
    const int unit = a.G / gcd_of(a.G, per);  // workgroups whose teams hold whole sets of groups
    if (unit > 512) p.teams = false;          // thousands of groups, an odd number of them
    if (!p.teams) {
        const int64_t want = 1024 / a.G < 1 ? 1 : 1024 / a.G;
        p.np = (int)(a.rows < want ? a.rows : want);
        p.blocks = (int)(items < 65536 ? items : 65536);
        return p;
    }
    // The backward runs one workgroup per CU twice over (its partial sums grow with them);
    // the forward one for each two rows of a team, up to where the CUs are full many times.
    const int64_t need = (items + per - 1) / per;
    int64_t want = bwd ? 512 : (need + 1) / 2;
    if (!bwd && want < 512) want = 512;
    if (want > 16384) want = 16384;
    if (want > need) want = need;
    p.blocks = (int)((want + unit - 1) / unit) * unit;
    p.fold = per % a.G == 0 && per / a.G > 1 && fold_lds(a, p) <= 60 * 1024;
    p.np = p.fold ? p.blocks : (int)((int64_t)p.blocks * per / a.G);
    return p;
}

size_t norm_bwd_ws(const NormArgs& a, int) {
    return (size_t)norm_plan(a, true, 1).np * 2 * a.C * 4;  // the same for every e
}

static int norm_e(const NormArgs& a, int act, bool bwd) {
    const int esz = act == SSD_BF16 ? 2 : 4;
    auto fits = [&](int e) {
        auto ok = [&](const void* p, int64_t stride) {
            return p == nullptr || ((uintptr_t)p % (e * esz) == 0 && stride % e == 0);
        };
        if (a.gs % e || !ok(a.x, a.xs) || !ok(a.z, a.zs)) return false;
        return bwd ? ok(a.dy, a.ys) && ok(a.dx, a.dxs) && ok(a.dz, a.dzs) : ok(a.y, a.ys);
    };
    if (fits(16 / esz)) return 16 / esz;
    return esz == 2 && fits(2) ? 2 : 1;
}

template <typename T, int E, int EPL, int MODE>
static hipError_t norm_teams(const NormArgs& a, const NormPlan& p, float* part, hipStream_t s) {
    const dim3 grid((unsigned)p.blocks), block(NORM_NT);
    if (!part) {
        if (p.wide) return launch(k_norm_fwd<T, E, EPL, MODE, true>, grid, block, s, a, p.lpt);
        return launch(k_norm_fwd<T, E, EPL, MODE, false>, grid, block, s, a, p.lpt);
    }
    const int lds = p.fold ? (int)fold_lds(a, p) : 0;
    if (p.wide)
        return launch_lds(k_norm_bwd<T, E, EPL, MODE, true>, grid, block, lds, s, a, p.lpt,
                          (int)p.fold, part);
    if constexpr (EPL == 8)
        return launch_lds(k_norm_bwd<T, E, EPL, MODE, false>, grid, block, lds, s, a, p.lpt,
                          (int)p.fold, part);
    return hipErrorInvalidValue;  // more than 8 channels to a lane take 512 lanes
}

template <typename T, int E, int EPL>
static hipError_t norm_mode(const NormArgs& a, const NormPlan& p, float* part, hipStream_t s) {
    switch (a.mode) {
        case SSD_NORM_NONE: return norm_teams<T, E, EPL, SSD_NORM_NONE>(a, p, part, s);
        case SSD_NORM_SILU: return norm_teams<T, E, EPL, SSD_NORM_SILU>(a, p, part, s);
        case SSD_NORM_BEFORE: return norm_teams<T, E, EPL, SSD_NORM_BEFORE>(a, p, part, s);
        default: return norm_teams<T, E, EPL, SSD_NORM_AFTER>(a, p, part, s);
    }
}

template <typename T, int E>
static hipError_t norm_epl(const NormArgs& a, const NormPlan& p, float* part, hipStream_t s) {
    if (p.epl == 8) return norm_mode<T, E, 8>(a, p, part, s);
    if (p.epl == 16) return norm_mode<T, E, 16>(a, p, part, s);
    return norm_mode<T, E, 32>(a, p, part, s);
}

template <typename T>
static hipError_t norm_t(const NormArgs& a, const NormPlan& p, float* part, hipStream_t s) {
    if (!p.teams) {
        if (!part) return launch(k_norm_fwd_any<T>, dim3((unsigned)p.blocks), dim3(256), s, a);
        return launch(k_norm_bwd_any<T>, dim3((unsigned)p.np, (unsigned)a.G), dim3(256), s, a, part);
    }
    if (p.e == 1) return norm_epl<T, 1>(a, p, part, s);
    if constexpr (sizeof(T) == 2)
        if (p.e == 2) return norm_epl<T, 2>(a, p, part, s);
    return norm_epl<T, 16 / (int)sizeof(T)>(a, p, part, s);
}

hipError_t launch_norm_fwd(const NormArgs& a, int act, hipStream_t s) {
    const NormPlan p = norm_plan(a, false, norm_e(a, act, false));
    return act == SSD_BF16 ? norm_t<bf16>(a, p, nullptr, s) : norm_t<float>(a, p, nullptr, s);
}

hipError_t launch_norm_bwd(const NormArgs& a, int act, float* part, hipStream_t s) {
    const NormPlan p = norm_plan(a, true, norm_e(a, act, true));
    SSD_TRY(act == SSD_BF16 ? norm_t<bf16>(a, p, part, s) : norm_t<float>(a, p, part, s));
    return launch(k_norm_reduce, dim3((unsigned)((2 * (int64_t)a.C + 63) / 64)), dim3(1024), s,
                  (const float*)part, p.np, a.C, a.dw, a.db);
}

}  // namespace ssd
