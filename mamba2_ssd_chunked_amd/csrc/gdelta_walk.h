// The walk of the gated delta rule from chunk to chunk (see gdelta.h): forward, and the same walk as
// the backward's recomputation (KEEP), which keeps entering states and u instead of outputs.
//
// A workgroup of four waves walks 64 CT value channels of a head over its sequence.  The rows of
// the next chunk are on their way into registers while a chunk is computed.
#pragma once

#include "gdelta.h"

namespace ssd {

template <typename T, int BD, int CT, int PT, bool KEEP>
constexpr int gd_walk_lds() {
    constexpr int e = sizeof(T);
    return GD_Q * (GdRows<T, BD>::PITCH * (KEEP ? 1 : 2) + GdRows<T, 64 * CT>::PITCH + GdMat<T, PT>::PITCH +
                   (KEEP ? 0 : GdMat<T, sizeof(T) == 2 ? 2 : 1>::PITCH)) * e +
           (int)sizeof(GdScalars) + 16;
}

// PT: parts of T, R, states and u on their way into states (2, or 3 where a state is asked for).
template <typename T, int BD, int CT, int PT, bool KEEP>
__global__ void __launch_bounds__(256) k_gd_walk(GdArgs a, LaPlan plan) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    constexpr int SL = M::SL, KS = M::KS, KB = BD / KS, TPK = LaCfg<T>::TPK, NK = GD_Q / KS;
    constexpr int BT = BD / 16, CDW = 64 * CT, PO = sizeof(T) == 2 ? 2 : 1;  // parts in outputs
    constexpr int PE = 1;  // q, k and v are exact
    typedef GdMat<T, PT> MatT;
    typedef GdMat<T, PO> MatP;
    constexpr int AP = GdRows<T, BD>::PITCH, CP = GdRows<T, CDW>::PITCH;
    __shared__ __align__(16) unsigned char lds[gd_walk_lds<T, BD, CT, PT, KEEP>()];
    T* sk = (T*)lds;
    T* sv = sk + GD_Q * AP;
    T* st = sv + GD_Q * CP;
    T* sq = st + GD_Q * MatT::PITCH;
    T* sp = sq + (KEEP ? 0 : GD_Q * AP);
    GdScalars* sc = (GdScalars*)(sp + (KEEP ? 0 : GD_Q * MatP::PITCH));

    const int nblk = a.valdim / CDW;
    const GdItem it = gd_item(a, nblk);
    if (it.s < 0) return;
    const int h = it.h, wave = wave_id(), lane = threadIdx.x % 64, lr = lane % 16, lg = lane / 16;
    const SeqRange sr = seq_range(a, it.s);
    const int64_t lo = sr.lo;
    const int len = (int)(sr.hi - sr.lo), nch = (len + GD_Q - 1) / GD_Q;
    const int c0 = it.cb * CDW, DV = a.valdim;
    const T* pq = (const T*)a.q + (int64_t)(h / a.share) * BD;
    const T* pk = (const T*)a.k + (int64_t)(h / a.share) * BD;
    const T* pv = (const T*)a.v + (int64_t)h * DV + c0;
    const int64_t hrow = (int64_t)h * a.tokens;

    GdRows<T, BD> rk, rq;
    GdRows<T, CDW> rv;
    GdRows<T, MatT::D> rt;
    GdRows<T, MatP::D> rp;
    f32x4 rs;
    auto tokens_of = [&](int k) { return len - k * GD_Q < GD_Q ? len - k * GD_Q : GD_Q; };
    auto load = [&](int k) {
        const int n = tokens_of(k);
        const int64_t t0 = lo + (int64_t)k * GD_Q;
        rk.load(pk, a.k_ts, t0, n);
        rv.load(pv, a.v_ts, t0, n);
        rt.load((const T*)a.T, MatT::D, hrow + t0, n);
        if constexpr (!KEEP) {
            rq.load(pq, a.q_ts, t0, n);
            rp.load((const T*)a.P, MatP::D, hrow + t0, n);
        }
        rs = f32x4{0.f, 0.f, 0.f, 0.f};
        if (threadIdx.x < n) rs = a.sc[hrow + t0 + threadIdx.x];
    };
    if (nch > 0) load(0);

    // this lane's elements of tile (t, u): channels of k from la_channel, channel `col` + 16 u of v
    f32x4 St[BT][CT];
    const int cw = wave * 16 * CT, col = c0 + cw + lr;
    const int64_t state_at = ((int64_t)it.s * a.H + h) * ((int64_t)BD * DV);
    auto at = [&](int t, int u) { return (col + 16 * u) * BD + la_channel<T>(t, lg); };
#pragma unroll
    for (int t = 0; t < BT; ++t)
#pragma unroll
        for (int u = 0; u < CT; ++u)
            St[t][u] = a.init ? *(const f32x4*)(a.init + state_at + at(t, u)) : f32x4{0.f, 0.f, 0.f, 0.f};

    for (int k = 0; k < nch; ++k) {
        const int n = tokens_of(k);
        const int64_t t0 = lo + (int64_t)k * GD_Q;
        __syncthreads();  // the last chunk's reads are done
        rk.store(sk);
        rv.store(sv);
        rt.store(st);
        if constexpr (!KEEP) {
            rq.store(sq);
            rp.store(sp);
        }
        if (wave == 0) gd_scalars_store(sc, rs);
        __syncthreads();
        load(k + 1 < nch ? k + 1 : k);
        const int bad = sc->bad;
        if (!KEEP && bad < GD_Q) {  // for the whole workgroup
            for (int x = threadIdx.x; x < (GD_Q - bad) * AP; x += 256) sk[bad * AP + x] = (T)0.f;
            __syncthreads();
        }
        if constexpr (KEEP)
            if (k > 0) {
                float* S = a.S + (la_place(a, plan, it.s, lo, k) * a.H + h) * ((int64_t)BD * DV);
#pragma unroll
                for (int t = 0; t < BT; ++t)
#pragma unroll
                    for (int u = 0; u < CT; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            S[(la_channel<T>(t, lg) + r) * DV + col + 16 * u] = St[t][u][r];
            }

        // X = K S^T and S Q^T
        f32x4 x[GD_NT][CT], o[GD_NT][CT];
#pragma unroll
        for (int t = 0; t < GD_NT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) x[t][u] = o[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < KB; ++q) {
            Frag sf[CT][PT];
#pragma unroll
            for (int u = 0; u < CT; ++u) {
                f32x4 tl[TPK];
#pragma unroll
                for (int e = 0; e < TPK; ++e) tl[e] = St[q * TPK + e][u];
                gd_split<T, PT>(tl, sf[u]);
            }
#pragma unroll
            for (int t = 0; t < GD_NT; ++t) {
                const Frag f = M::load(sk + (16 * t + lr) * AP + KS * q + SL * lg);
#pragma unroll
                for (int u = 0; u < CT; ++u) x[t][u] = gd_mma<T, PE, PT>(&f, sf[u], x[t][u]);
            }
            if constexpr (!KEEP)
#pragma unroll
                for (int t = 0; t < GD_NT; ++t) {
                    const Frag f = M::load(sq + (16 * t + lr) * AP + KS * q + SL * lg);
#pragma unroll
                    for (int u = 0; u < CT; ++u) o[t][u] = gd_mma<T, PO, PE>(sf[u], &f, o[t][u]);
                }
        }

        // R = B (V - e^c X).  A value of v that is not finite would reach the rows before its own: it
        // counts as zero, and its channel is made NaN from its row on further down.
        Frag rf[NK][CT][PT];
        int first[CT];
#pragma unroll
        for (int u = 0; u < CT; ++u) {
            float seen = 0.f;
            Frag vf[NK];
#pragma unroll
            for (int b = 0; b < NK; ++b) {
                vf[b] = XT<T>::load(sv, CP, KS * b, cw + 16 * u, lane);
#pragma unroll
                for (int s = 0; s < SL; ++s) seen += (float)vf[b][s] * 0.f;
            }
            first[u] = bad;
            if (!KEEP && __ballot(seen != 0.f)) {  // NaN is not equal to zero
#pragma unroll
                for (int b = NK - 1; b >= 0; --b)
#pragma unroll
                    for (int s = SL - 1; s >= 0; --s)
                        if (!(fabsf((float)vf[b][s]) < INFINITY)) {
                            const int j = KS * b + 16 * (s / 4) + 4 * lg + s % 4;
                            first[u] = j < first[u] ? j : first[u];
                            vf[b][s] = (T)0.f;
                        }
                // the least of the four lane groups' rows
#pragma unroll
                for (int m = 16; m < 64; m <<= 1) {
                    const int y = __shfl_xor(first[u], m, 64);
                    first[u] = y < first[u] ? y : first[u];
                }
            }
#pragma unroll
            for (int b = 0; b < NK; ++b) {
                f32x4 tl[TPK];
#pragma unroll
                for (int e = 0; e < TPK; ++e) {
                    const int t = b * TPK + e;
                    const f32x4 in = *(const f32x4*)(sc->in + 16 * t + 4 * lg);
                    const f32x4 be = *(const f32x4*)(sc->beta + 16 * t + 4 * lg);
#pragma unroll
                    for (int r = 0; r < 4; ++r) tl[e][r] = be[r] * ((float)vf[b][4 * e + r] - in[r] * x[t][u][r]);
                }
                gd_split<T, PT>(tl, rf[b][u]);
            }
        }

        // U = T R
#pragma unroll
        for (int t = 0; t < GD_NT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) x[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < NK; ++b)
#pragma unroll
            for (int t = b * TPK; t < GD_NT; ++t) {
                Frag tf[PT];
#pragma unroll
                for (int p = 0; p < PT; ++p) tf[p] = MatT::row(st, t, b, p, lane);
#pragma unroll
                for (int u = 0; u < CT; ++u) x[t][u] = gd_mma<T, PT, PT>(tf, rf[b][u], x[t][u]);
            }

        if constexpr (KEEP) {
            const __amdgpu_buffer_rsrc_t r = buf_rsrc(a.U + (hrow + t0) * DV, n * DV * 4);
#pragma unroll
            for (int t = 0; t < GD_NT; ++t)
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        __builtin_amdgcn_raw_buffer_store_b32(
                            __float_as_uint(x[t][u][q]), r, ((16 * t + 4 * lg + q) * DV + col + 16 * u) * 4, 0, 0);
        } else {
            // O = scale e^c Q S^T + P U, a lane has row 16 t + lr and channels 4 lg ..
#pragma unroll
            for (int t = 0; t < GD_NT; ++t) {
                const float f = a.scale * sc->in[16 * t + lr];
#pragma unroll
                for (int u = 0; u < CT; ++u) o[t][u] *= f;
            }
#pragma unroll
            for (int b = 0; b < NK; ++b) {
                Frag uf[CT][PO];
#pragma unroll
                for (int u = 0; u < CT; ++u) {
                    f32x4 tl[TPK];
#pragma unroll
                    for (int e = 0; e < TPK; ++e) tl[e] = x[b * TPK + e][u];
                    gd_split<T, PO>(tl, uf[u]);
                }
#pragma unroll
                for (int t = b * TPK; t < GD_NT; ++t) {
                    Frag pf[PO];
#pragma unroll
                    for (int p = 0; p < PO; ++p) pf[p] = MatP::row(sp, t, b, p, lane);
#pragma unroll
                    for (int u = 0; u < CT; ++u) o[t][u] = gd_mma<T, PO, PO>(uf[u], pf, o[t][u]);
                }
            }
#pragma unroll
            for (int u = 0; u < CT; ++u)
                if (__ballot(first[u] < GD_Q)) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int f = __shfl(first[u], 4 * lg + r, 64);
#pragma unroll
                        for (int t = 0; t < GD_NT; ++t)
                            if (16 * t + lr >= f) o[t][u][r] = NAN;
                    }
                }
            const int out_bytes = (int)a.o_ts * (int)sizeof(T);
            const __amdgpu_buffer_rsrc_t r =
                buf_rsrc((T*)a.o + t0 * a.o_ts + (int64_t)h * DV + c0, n * out_bytes);
            if constexpr (sizeof(T) == 2) {
                const int half = lg & 1, c8 = cw + 8 * (lg >> 1);
                if constexpr (CT == 2) {
#pragma unroll
                    for (int t = 0; t < GD_NT; ++t)
                        buf_store(la_pair(o[t][0], o[t][1]), r,
                                  (16 * t + lr) * out_bytes + (c8 + 16 * half) * 2);
                } else {
#pragma unroll
                    for (int t = 0; t < GD_NT; t += 2)
                        buf_store(la_pair(o[t][0], o[t + 1][0]), r,
                                  (16 * (t + half) + lr) * out_bytes + c8 * 2);
                }
            } else {
#pragma unroll
                for (int t = 0; t < GD_NT; ++t)
#pragma unroll
                    for (int u = 0; u < CT; ++u)
                        buf_store(o[t][u], r, (16 * t + lr) * out_bytes + (cw + 16 * u + 4 * lg) * 4);
            }
        }

        // S <- e^C S + sum_j e^(C - c_j) u_j k_j^T
        const float keep = sc->in[n - 1];
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) St[t][u] *= keep;
#pragma unroll
        for (int b = 0; b < NK; ++b) {
            Frag uf[CT][PT];
#pragma unroll
            for (int u = 0; u < CT; ++u) {
                f32x4 tl[TPK];
#pragma unroll
                for (int e = 0; e < TPK; ++e)
                    tl[e] = x[b * TPK + e][u] * *(const f32x4*)(sc->out + 16 * (b * TPK + e) + 4 * lg);
                gd_split<T, PT>(tl, uf[u]);
            }
#pragma unroll
            for (int t = 0; t < BT; ++t) {
                const Frag f = la_bt<T>(sk, AP, KS * b, t, lane);
#pragma unroll
                for (int u = 0; u < CT; ++u) St[t][u] = gd_mma<T, PE, PT>(&f, uf[u], St[t][u]);
            }
        }
        if (!KEEP)
#pragma unroll
            for (int u = 0; u < CT; ++u)
                if (first[u] < GD_Q)
#pragma unroll
                    for (int t = 0; t < BT; ++t) St[t][u] = f32x4{NAN, NAN, NAN, NAN};
    }
    if (!KEEP && a.fin) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) *(f32x4*)(a.fin + state_at + at(t, u)) = St[t][u];
    }
}

}  // namespace ssd
