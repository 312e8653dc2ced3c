// Group norm with an activation, channels last: forward and backward.
//
// With s the gate's SiLU and u = x s (gated before) or x:
//   n = (u - m) r,  r = 1 / sqrt(mean((u - m)^2) + eps),  lin = n w + b
//   y = lin, silu(lin) or lin s
// Backward, with e the gradient that reaches lin, g = e w:
//   du = r (g - [center] mean(g) - n mean(g n));  dw = sum e n, db = sum e.
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

// dw and db from the blocks' partial sums, in the blocks' order.
__global__ void __launch_bounds__(256) k_norm_reduce(const float* __restrict__ part, int blocks,
                                                    int C, float* __restrict__ dw,
                                                    float* __restrict__ db) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= C) return;
    float sw = 0.f, sb = 0.f;
    for (int i = 0; i < blocks; ++i) {
        sw += part[(int64_t)i * 2 * C + c];
        sb += part[(int64_t)i * 2 * C + C + c];
    }
    dw[c] = sw;
    if (db) db[c] = sb;
}

int norm_row_blocks(const NormArgs& a, int) {
    const int64_t want = 1024 / a.G < 1 ? 1 : 1024 / a.G;
    return (int)(a.rows < want ? a.rows : want);
}

hipError_t launch_norm_fwd(const NormArgs& a, int act, hipStream_t s) {
    const int64_t n = a.rows * a.G;
    const dim3 grid((unsigned)(n < 65536 ? n : 65536));
    if (act == SSD_BF16) return launch(k_norm_fwd_any<bf16>, grid, dim3(256), s, a);
    return launch(k_norm_fwd_any<float>, grid, dim3(256), s, a);
}

hipError_t launch_norm_bwd(const NormArgs& a, int act, float* part, hipStream_t s) {
    const int nb = norm_row_blocks(a, act);
    const dim3 grid((unsigned)nb, (unsigned)a.G);
    if (act == SSD_BF16)
        SSD_TRY(launch(k_norm_bwd_any<bf16>, grid, dim3(256), s, a, part));
    else
        SSD_TRY(launch(k_norm_bwd_any<float>, grid, dim3(256), s, a, part));
    return launch(k_norm_reduce, dim3((unsigned)((a.C + 255) / 256)), dim3(256), s,
                  (const float*)part, nb, a.C, a.dw, a.db);
}

}  // namespace ssd
