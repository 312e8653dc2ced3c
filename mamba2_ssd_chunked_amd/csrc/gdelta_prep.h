// T and P of every chunk of the gated delta rule, and its per-token factors.
//
// One workgroup of four waves per (chunk, head).  Wave w computes row tile w of K K^T and Q K^T (each
// tile transposed, so that a lane has four neighbouring columns of a row), then inverts
// the 16 x 16 diagonal block w of I + A by substitution, a column to a lane, and solves block column
// w below it with products of 16 x 16 blocks, all in float32: T_ij = -T_ii sum_{j<=k<i} A_ik T_kj.
// (Powers of A would be cheaper products, but lose all digits for keys that resemble each other.)
#pragma once

#include "gdelta.h"

namespace ssd {

// PT, PP: parts of T and P.  TAME: a key, g or beta that is not finite ends the chunk at its row (k and
// beta count as zero from there on, and `out` tells the rows); else it spreads over the chunk.
template <typename T, int DK, int PT, int PP, bool TAME>
__global__ void __launch_bounds__(256) k_gd_prep(GdArgs a, LaPlan plan) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    constexpr int SL = M::SL, KS = M::KS, KB = DK / KS, AP = GdRows<T, DK>::PITCH, FP = GD_Q + 4;
    constexpr int QB = GD_Q * AP * (int)sizeof(T), AB = GD_Q * FP * 4;
    __shared__ __align__(16) T sk[GD_Q * AP];
    __shared__ __align__(16) char both[QB > AB ? QB : AB];  // the queries, then A (four workgroups fit a CU)
    T* sq = (T*)both;
    float* A = (float*)both;
    __shared__ double c2[GD_Q];  // c in units of log 2
    __shared__ float sbeta[GD_Q];
    __shared__ int sbad;
    const int h = blockIdx.x % a.H;
    const LaSpan sp = la_span(a, plan, blockIdx.x / a.H);
    if (sp.s < 0 || sp.n <= 0) return;
    const int n = sp.n, wave = wave_id(), lane = threadIdx.x % 64, lr = lane % 16, lg = lane / 16;
    const int64_t t0 = sp.lo + sp.i0;
    const int hk = h / a.share;
    GdRows<T, DK> rk, rq;
    rk.load((const T*)a.k + (int64_t)hk * DK, a.k_ts, t0, n);
    rq.load((const T*)a.q + (int64_t)hk * DK, a.q_ts, t0, n);
    float g = 0.f, b = 0.f;
    if (wave == 0 && lane < n) {
        g = a.g[(t0 + lane) * a.g_ts + h];
        b = a.beta[(t0 + lane) * a.b_ts + h];
    }
    if (TAME && threadIdx.x == 0) sbad = GD_Q;
    rk.store(sk);
    rq.store(sq);
    if constexpr (TAME) {
        __syncthreads();
        int bad = rk.wild_row();
        if (wave == 0 && bad > lane && (!(g < INFINITY) || !(fabsf(b) < INFINITY))) bad = lane;
        if (bad < GD_Q) atomicMin(&sbad, bad);
        __syncthreads();
        bad = sbad;
        if (bad < GD_Q) {
            for (int x = threadIdx.x; x < (GD_Q - bad) * AP; x += 256) sk[bad * AP + x] = (T)0.f;
            if (lane >= bad) g = b = 0.f;
        }
    }
    const int64_t row0 = (int64_t)h * a.tokens + t0;
    if (wave == 0) {
        if constexpr (!TAME)
            if (lane < n && fabsf(b) < GD_BETA_MIN) b = copysignf(GD_BETA_MIN, b);
        // minus infinity is as good as any factor that float32 has no number for
        double c = (double)(g < -1e5f ? -1e5f : g) * 1.4426950408889634;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double up = __shfl_up(c, o, 64);
            if (lane >= o) c += up;
        }
        c2[lane] = c;
        sbeta[lane] = b;
        const double last = __shfl(c, 63, 64);
        if (lane < n) {
            const bool bad = TAME && lane >= sbad;
            a.in[row0 + lane] = __builtin_amdgcn_exp2f((float)c);
            a.out[row0 + lane] = bad ? -1.f : __builtin_amdgcn_exp2f((float)(last - c));
            a.beta_of[row0 + lane] = b;
            if constexpr (!TAME) a.c2[row0 + lane] = c;
        }
    }
    __syncthreads();

    // row tile `wave`; a lane has row i of every tile and its four columns j ..
    const int i = 16 * wave + lr;
    {
        Frag kf[KB], qf[KB];
#pragma unroll
        for (int q = 0; q < KB; ++q) {
            kf[q] = M::load(sk + i * AP + KS * q + SL * lg);
            qf[q] = M::load(sq + i * AP + KS * q + SL * lg);
        }
        __syncthreads();  // the queries are read
        const double ci = c2[i];
        const float bi = sbeta[i];
        const __amdgpu_buffer_rsrc_t rp = buf_rsrc((T*)a.P + row0 * (GD_Q * PP), n * GD_Q * PP * (int)sizeof(T));
        for (int kb = 0; kb <= wave / 2; ++kb) {
            f32x4 p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int jt = 2 * kb + e, j = 16 * jt + 4 * lg;
                f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qk = kk;
#pragma unroll
                for (int q = 0; q < KB; ++q) {
                    const Frag f = M::load(sk + (16 * jt + lr) * AP + KS * q + SL * lg);
                    kk = M::mma(f, kf[q], kk);
                    qk = M::mma(f, qf[q], qk);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float m = __builtin_amdgcn_exp2f((float)(ci - c2[j + r]));
                    kk[r] = j + r < i ? bi * m * kk[r] : 0.f;
                    p[e][r] = j + r <= i ? a.scale * m * qk[r] : 0.f;
                }
                *(f32x4*)(A + i * FP + j) = kk;
            }
            if constexpr (sizeof(T) == 2) {
                Frag f[PP];
                gd_split<T, PP>(p, f);
#pragma unroll
                for (int x = 0; x < PP; ++x)
                    buf_store(f[x], rp, (i * GD_Q * PP + x * GD_Q + 32 * kb + 8 * lg) * 2);
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) buf_store(p[e], rp, (i * GD_Q + 32 * kb + 16 * e + 4 * lg) * 4);
            }
        }
    }
    __syncthreads();

    // diagonal block `wave`: column lr of its inverse, the same in the four lane groups
    f32x4 x[GD_NT];  // block column `wave` of T
    {
        float y[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float v = r == lr ? 1.f : 0.f;
            const float* row = A + (16 * wave + r) * FP + 16 * wave;
#pragma unroll
            for (int c = 0; c < r; ++c) v -= row[c] * y[c];
            y[r] = v;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[0][r] = lg == 0 ? y[r] : (lg == 1 ? y[4 + r] : (lg == 2 ? y[8 + r] : y[12 + r]));
#pragma unroll
        for (int r = 0; r < 4; ++r) A[(16 * wave + 4 * lg + r) * FP + 16 * wave + lr] = x[0][r];
    }
    __syncthreads();
    auto block = [&](int ib, int jb) { return *(const f32x4*)(A + (16 * ib + lr) * FP + 16 * jb + 4 * lg); };
#pragma unroll
    for (int d = 1; d < GD_NT; ++d)
        if (wave + d < GD_NT) {
            f32x4 y = {0.f, 0.f, 0.f, 0.f}, z = y;
#pragma unroll
            for (int e = 0; e < d; ++e) y = Mma<float>::mma(block(wave + d, wave + e), x[e], y);
            x[d] = -Mma<float>::mma(block(wave + d, wave + d), y, z);
        }
    __syncthreads();
#pragma unroll
    for (int d = 1; d < GD_NT; ++d)
        if (wave + d < GD_NT) {
#pragma unroll
            for (int r = 0; r < 4; ++r) A[(16 * (wave + d) + 4 * lg + r) * FP + 16 * wave + lr] = x[d][r];
        }
    __syncthreads();
    const __amdgpu_buffer_rsrc_t rt = buf_rsrc((T*)a.T + row0 * (GD_Q * PT), n * GD_Q * PT * (int)sizeof(T));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int item = k * 256 + threadIdx.x, row = item / 8, b = item % 8 / 4, q = item % 4;
        if (b > row / 32) continue;  // above the diagonal: never read
        f32x4 v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) v[e] = *(const f32x4*)(A + row * FP + 32 * b + 16 * e + 4 * q);
        if constexpr (sizeof(T) == 2) {
            Frag f[PT];
            gd_split<T, PT>(v, f);
#pragma unroll
            for (int p = 0; p < PT; ++p)
                buf_store(f[p], rt, (row * GD_Q * PT + p * GD_Q + 32 * b + 8 * q) * 2);
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) buf_store(v[e], rt, (row * GD_Q + 32 * b + 16 * e + 4 * q) * 4);
        }
    }
}

}  // namespace ssd
