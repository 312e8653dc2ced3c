// Backward of the gated delta rule (see gdelta.h): the walk from the last chunk to the first and the
// chunks' gradients.
#pragma once

#include "gdelta.h"

namespace ssd {

template <typename T, int BD, int NW, int PT>
struct GdBackLds {
    static constexpr int k = 0, q = k + GdTile<T, BD>::BYTES, d = q + GdTile<T, BD>::BYTES,
                         t = d + GdTile<T, 16 * NW>::BYTES, p = t + GdMat<T, PT>::BYTES,
                         sc = p + GdMat<T, PT>::BYTES, bytes = (sc + (int)sizeof(GdScalars) + 1023) / 1024 * 1024;
    static constexpr int buffers = 2 * bytes <= 160 * 1024 ? 2 : 1;
};

// The gradient G of the state, as the forward walk keeps S: a wave owns columns of G^T.
template <typename T, int BD, int NW, int PT>
__global__ void __launch_bounds__(64 * NW) k_gd_back(GdArgs a, LaPlan plan) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    typedef GdBackLds<T, BD, NW, PT> L;
    typedef GdTile<T, BD> Tile;
    typedef GdTile<T, 16 * NW> TileV;
    typedef GdMat<T, PT> Mat;
    constexpr int KS = M::KS, KB = BD / KS, TPK = LaCfg<T>::TPK, NK = GD_Q / KS;
    constexpr int BT = BD / 16, CDW = 16 * NW;
    __shared__ __align__(1024) char lds[L::buffers * L::bytes];

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
    const T* pd = (const T*)a.dout + (int64_t)h * DV + c0;
    const int64_t hrow = (int64_t)h * a.tokens;

    auto tokens_of = [&](int k) { return len - k * GD_Q < GD_Q ? len - k * GD_Q : GD_Q; };
    // as in the forward walk
    struct Next {
        gd_i4 k, d, t, q, p;
        int64_t row;
        int n;
        unsigned to;
    };
    auto next_of = [&](int k, int buffer) {
        Next x;
        const int64_t t0 = lo + (int64_t)k * GD_Q;
        x.n = tokens_of(k);
        x.row = hrow + t0;
        x.to = gd_lds(lds + (L::buffers == 2 && buffer % 2 ? L::bytes : 0));
        auto rows = [&](const T* base, int64_t ts) { return gd_rsrc(base + t0 * ts, x.n * (int)ts * (int)sizeof(T)); };
        x.k = rows(pk, a.k_ts);
        x.q = rows(pq, a.q_ts);
        x.d = rows(pd, a.o_ts);
        x.t = gd_rsrc((const T*)a.T + x.row * Mat::D, x.n * Mat::ROW);
        x.p = gd_rsrc((const T*)a.P + x.row * Mat::D, x.n * Mat::ROW);
        return x;
    };
    constexpr int FR = gd_share(Tile::FETCHES, NW), FM = gd_share(Mat::FETCHES, NW), FV = gd_share(TileV::FETCHES, NW);
    constexpr int NF = 2 * FR + 2 * FM + FV + gd_share(3, NW);
    auto fetch = [&](const Next& x, auto I) {
        constexpr int i = decltype(I)::value, at_d = FR, at_p = at_d + FV, at_t = at_p + FM, at_q = at_t + FM, at_s = at_q + FR;
        const int es = (int)sizeof(T);
        if constexpr (i < at_d) Tile::fetch(x.k, (int)a.k_ts * es, x.to + L::k, gd_mine<Tile::FETCHES, NW>(i, wave), lane);
        else if constexpr (i < at_p) TileV::fetch(x.d, (int)a.o_ts * es, x.to + L::d, gd_mine<TileV::FETCHES, NW>(i - at_d, wave), lane);
        else if constexpr (i < at_t) Mat::fetch(x.p, x.to + L::p, gd_mine<Mat::FETCHES, NW>(i - at_p, wave), lane);
        else if constexpr (i < at_q) Mat::fetch(x.t, x.to + L::t, gd_mine<Mat::FETCHES, NW>(i - at_t, wave), lane);
        else if constexpr (i < at_s) Tile::fetch(x.q, (int)a.q_ts * es, x.to + L::q, gd_mine<Tile::FETCHES, NW>(i - at_q, wave), lane);
        else gd_scalars_fetch(a, x.row, x.n, x.to + L::sc, gd_mine<3, NW>(i - at_s, wave), lane);
    };
    auto stage_all = [&](int k) {
        const Next x = next_of(k, k);
        gd_for<NF>([&](auto I) { fetch(x, I); });
    };
    if (L::buffers == 2 && nch > 0) stage_all(nch - 1);

    f32x4 G[BT];
    const int cw = wave * 16, col = c0 + cw + lr;
    const int64_t state_at = ((int64_t)it.s * a.H + h) * ((int64_t)BD * DV);
    auto at = [&](int t) { return col * BD + la_channel<T>(t, lg); };
#pragma unroll
    for (int t = 0; t < BT; ++t)
        G[t] = a.dfin ? *(const f32x4*)(a.dfin + state_at + at(t)) : f32x4{0.f, 0.f, 0.f, 0.f};

    for (int k = nch - 1; k >= 0; --k) {
        const int n = tokens_of(k);
        const int64_t t0 = lo + (int64_t)k * GD_Q;
        if constexpr (L::buffers == 1) {
            __syncthreads();  // the last chunk's reads are done
            stage_all(k);
        }
        // behind this chunk's fetches stand only the last chunk's stores of Z
        if (L::buffers == 2 && k + 1 < nch) gd_wait<16>();
        else gd_wait<0>();
        __syncthreads();
        if (k + 1 < nch) {  // the gradient behind chunk k is kept where the state that enters k + 1 is
            float* g = a.G + (la_place(a, plan, it.s, lo, k + 1) * a.H + h) * ((int64_t)BD * DV);
#pragma unroll
            for (int t = 0; t < BT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) g[(la_channel<T>(t, lg) + r) * DV + col] = G[t][r];
        }
        const Next nx = next_of(k > 0 ? k - 1 : 0, k + 1);
        constexpr int PLACES = KB + 2 * NK;
        auto ahead = [&](auto I) {
            constexpr int i = decltype(I)::value, from = i * NF / PLACES, to = (i + 1) * NF / PLACES;
            if constexpr (L::buffers == 2) gd_for<to - from>([&](auto J) { fetch(nx, std::integral_constant<int, from + decltype(J)::value>{}); });
        };
        const char* buf = lds + (L::buffers == 2 && k % 2 ? L::bytes : 0);
        const char *sk = buf + L::k, *sq = buf + L::q, *sd = buf + L::d, *st = buf + L::t, *sp = buf + L::p;
        const GdScalars* sc = (const GdScalars*)(buf + L::sc);

        // P^T do + e^(C - c) K G^T
        f32x4 x[GD_NT], y[GD_NT];
#pragma unroll
        for (int t = 0; t < GD_NT; ++t) x[t] = y[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        Frag df[NK];
#pragma unroll
        for (int b = 0; b < NK; ++b) df[b] = TileV::xt(sd, KS * b, cw, lane);
        Frag f[KB][GD_NT];
#pragma unroll
        for (int q = 0; q < KB; ++q)
#pragma unroll
            for (int t = 0; t < GD_NT; ++t) f[q][t] = Tile::row(sk, t, q, lane);
        if constexpr (sizeof(T) == 2) __builtin_amdgcn_sched_barrier(0);
        gd_for<KB>([&](auto Q) {
            constexpr int q = decltype(Q)::value;
            Frag gf[PT];
            f32x4 tl[TPK];
#pragma unroll
            for (int e = 0; e < TPK; ++e) tl[e] = G[q * TPK + e];
            gd_split<T, PT>(tl, gf);
#pragma unroll
            for (int p = PT - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < GD_NT; ++t) y[t] = M::mma(f[q][t], gf[p], y[t]);
            ahead(Q);
        });
        gd_for<NK>([&](auto B) {
            constexpr int b = decltype(B)::value;
            Frag pf[GD_NT][PT];
#pragma unroll
            for (int t = 0; t < (b + 1) * TPK; ++t)
#pragma unroll
                for (int p = 0; p < PT; ++p) pf[t][p] = Mat::col(sp, t, b, p, lane);
            ahead(std::integral_constant<int, KB + b>{});
#pragma unroll
            for (int p = PT - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < (b + 1) * TPK; ++t) x[t] = M::mma(pf[t][p], df[b], x[t]);
        });
#pragma unroll
        for (int t = 0; t < GD_NT; ++t) {
            const f32x4 w = *(const f32x4*)(sc->out + 16 * t + 4 * lg);
            x[t] += w * y[t];
        }

        // Z = T^T of that
        f32x4 z[GD_NT];
#pragma unroll
        for (int t = 0; t < GD_NT; ++t) z[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        gd_for<NK>([&](auto B) {
            constexpr int b = NK - 1 - decltype(B)::value;
            Frag xf[PT];
            f32x4 tl[TPK];
#pragma unroll
            for (int e = 0; e < TPK; ++e) tl[e] = x[b * TPK + e];
            gd_split<T, PT>(tl, xf);
            Frag tf[GD_NT][PT];
#pragma unroll
            for (int t = 0; t < (b + 1) * TPK; ++t)
#pragma unroll
                for (int p = 0; p < PT; ++p) tf[t][p] = Mat::col(st, t, b, p, lane);
            ahead(std::integral_constant<int, KB + NK + decltype(B)::value>{});
#pragma unroll
            for (int s = PT - 1; s >= 0; --s)
#pragma unroll
                for (int p = 0; p <= s; ++p)
#pragma unroll
                    for (int t = 0; t < (b + 1) * TPK; ++t) z[t] = M::mma(tf[t][p], xf[s - p], z[t]);
        });
        const __amdgpu_buffer_rsrc_t r = buf_rsrc(a.Z + (hrow + t0) * DV, n * DV * 4);
#pragma unroll
        for (int t = 0; t < GD_NT; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                __builtin_amdgcn_raw_buffer_store_b32(
                    __float_as_uint(z[t][q]), r, ((16 * t + 4 * lg + q) * DV + col) * 4, 0, 0);

        // G <- e^C G + scale (e^c do)^T Q - (e^c B Z)^T K
        const float keep = sc->in[n - 1];
#pragma unroll
        for (int t = 0; t < BT; ++t) G[t] *= keep;
        gd_for<NK>([&](auto B) {
            constexpr int b = decltype(B)::value;
            Frag wf[PT], zf[PT];
            f32x4 tl[TPK], tz[TPK];
#pragma unroll
            for (int e = 0; e < TPK; ++e) {
                const int t = b * TPK + e;
                const f32x4 in = *(const f32x4*)(sc->in + 16 * t + 4 * lg);
                const f32x4 be = *(const f32x4*)(sc->beta + 16 * t + 4 * lg);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    tl[e][i] = a.scale * in[i] * (float)df[b][4 * e + i];
                    tz[e][i] = -in[i] * be[i] * z[t][i];
                }
            }
            gd_split<T, PT>(tl, wf);
            gd_split<T, PT>(tz, zf);
            Frag fb[BT];
#pragma unroll
            for (int t = 0; t < BT; ++t) fb[t] = Tile::bt(sq, KS * b, t, lane);
#pragma unroll
            for (int p = PT - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < BT; ++t) G[t] = M::mma(fb[t], wf[p], G[t]);
#pragma unroll
            for (int t = 0; t < BT; ++t) fb[t] = Tile::bt(sk, KS * b, t, lane);
#pragma unroll
            for (int p = PT - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < BT; ++t) G[t] = M::mma(fb[t], zf[p], G[t]);
        });
    }
    gd_wait<0>();  // a workgroup's LDS is another's once its waves have ended
    if (a.dinit) {
#pragma unroll
        for (int t = 0; t < BT; ++t) *(f32x4*)(a.dinit + state_at + at(t)) = G[t];
    }
}

// Parts of U, Z and E in a chunk's gradients: U and E reach dg, which is float32, Z only dk.
template <typename T> struct GdParts { static constexpr int U = 3, Z = 2, E = 3, N = 2; };
template <> struct GdParts<float> { static constexpr int U = 1, Z = 1, E = 1, N = 1; };

template <typename T, int DK, int DV>
struct GdChunkLds {
    typedef GdParts<T> P;
    static constexpr int AP = GdRows<T, DK, DK * 4>::PITCH, VP = DV + 16 / (int)sizeof(T);
    static constexpr int EP = GdRowsMat<T, P::E>::PITCH, NP = GdRowsMat<T, P::N>::PITCH;
    static constexpr bool DO = sizeof(T) == 2;  // rows of do are staged too
    // E and N take the place of U and Z
    static constexpr int uz = GD_Q * VP * (P::U + P::Z), en = GD_Q * (EP + NP);
    static constexpr int rows = GD_Q * AP * 2 + (DO ? GD_Q * VP : 0) + (uz > en ? uz : en);
    static constexpr int NW = DK / 16;
    static constexpr int bytes = rows * (int)sizeof(T);
};

// Gradients of one chunk of the heads that share a key head.  A wave owns 16 key channels: dq^T and dk^T
// [bd][token], summed over the heads in registers, in their order.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(DK * 4) k_gd_chunk(GdArgs a, LaPlan plan) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    typedef GdParts<T> P;
    typedef GdChunkLds<T, DK, DV> L;
    typedef GdRowsMat<T, P::E> MatE;
    typedef GdRowsMat<T, P::N> MatN;
    constexpr int SL = M::SL, KS = M::KS, TPK = LaCfg<T>::TPK, NK = GD_Q / KS, KV = DV / KS;
    constexpr int NW = L::NW, NTHR = DK * 4, AP = L::AP, VP = L::VP;
    constexpr int TILES = NK * (NK + 1) / 2 * TPK * TPK;  // of E: whole k blocks on and below the diagonal
    constexpr int PER = (TILES + NW - 1) / NW;
    __shared__ __align__(16) unsigned char lds[L::bytes];
    __shared__ double c2[GD_Q];
    __shared__ float s_in[GD_Q], s_out[GD_Q], s_beta[GD_Q], zv[GD_Q], red[NW][GD_Q], tot[NW];
    T* sk = (T*)lds;
    T* sq = sk + GD_Q * AP;
    T* sd = sq + GD_Q * AP;
    T* su = sd + (L::DO ? GD_Q * VP : 0);
    T* sz = su + GD_Q * VP * P::U;
    T* se = su;
    T* sn = se + GD_Q * L::EP;

    // a workgroup takes the heads of a key head in turn, or (a.sums) one head, whose dq and dk it leaves in float32
    const int heads = a.sums ? 1 : a.share, items = a.H / heads;
    const int h0 = (int)(blockIdx.x % items) * heads, hk = h0 / a.share;
    const LaSpan sp = la_span(a, plan, blockIdx.x / items);
    if (sp.s < 0 || sp.n <= 0) return;
    const int n = sp.n, wave = wave_id(), lane = threadIdx.x % 64, lr = lane % 16, lg = lane / 16;
    const int64_t t0 = sp.lo + sp.i0;
    const int b0 = 16 * wave;
    GdRows<T, DK, NTHR> rk, rq;
    rk.load((const T*)a.k + (int64_t)hk * DK, a.k_ts, t0, n);
    rq.load((const T*)a.q + (int64_t)hk * DK, a.q_ts, t0, n);
    f32x4 DQ[GD_NT], DKt[GD_NT];
#pragma unroll
    for (int t = 0; t < GD_NT; ++t) DQ[t] = DKt[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int m = 0; m < heads; ++m) {
        const int h = h0 + m;
        const int64_t row0 = (int64_t)h * a.tokens + t0;
        if (m > 0) __syncthreads();  // the last head's reads are done
        // All that a head reads is asked for at once, but for G: one wait where each piece would have its own
        // (8192 chunks of 128 x 128: 930 us, 885 so, 915 with rates as given; 23 chunks of 64 x 64: 49, 41).
        typedef T t4 __attribute__((ext_vector_type(4)));
        constexpr int VPR = DV / 8, NX = GD_Q * VPR / NTHR;  // runs of eight value channels of a row, of a thread
        static_assert(GD_Q * VPR % NTHR == 0, "the threads tile the rows");
        const __amdgpu_buffer_rsrc_t ru = buf_rsrc(a.U + row0 * DV, n * DV * 4), rz = buf_rsrc(a.Z + row0 * DV, n * DV * 4);
        const __amdgpu_buffer_rsrc_t rv = buf_rsrc((const T*)a.v + t0 * a.v_ts + (int64_t)h * DV, n * (int)a.v_ts * (int)sizeof(T));
        const T* pd = (const T*)a.dout + t0 * a.o_ts + (int64_t)h * DV;
        const bool live = threadIdx.x < n;
        const float rin = live ? a.in[row0 + threadIdx.x] : 0.f, rout = live ? a.out[row0 + threadIdx.x] : 0.f;
        const float rbeta = live ? a.beta[(t0 + threadIdx.x) * a.b_ts + h] : 1.f;
        const double rc = live ? a.c2[row0 + threadIdx.x] : -1e30;  // no factor of a row without a token
        GdRows<T, DV, NTHR> rd;
        if constexpr (L::DO) rd.load((const T*)a.dout + (int64_t)h * DV, a.o_ts, t0, n);
        f32x4 u[NX][2], z[NX][2];
        t4 vv[NX][2];
        float be[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int y = i * NTHR + threadIdx.x, row = y / VPR, c = y % VPR * 8;
            be[i] = row < n ? a.beta[(t0 + row) * a.b_ts + h] : 1.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                u[i][e] = buf_load<f32x4>(ru, (row * DV + c + 4 * e) * 4);
                z[i][e] = buf_load<f32x4>(rz, (row * DV + c + 4 * e) * 4);
                vv[i][e] = buf_load<t4>(rv, (row * (int)a.v_ts + c + 4 * e) * (int)sizeof(T));
            }
        }
        // S and G of this wave's key channels: a lane has channel b0 + lr and value channels in k order
        const int64_t state = ((int64_t)sp.s * a.H + h) * ((int64_t)DK * DV);
        const float *pS = nullptr, *pG = nullptr;  // kept ones: [bd][cd]
        if (sp.i0 > 0) pS = a.S + (la_place(a, plan, sp.s, sp.lo, sp.j) * a.H + h) * ((int64_t)DK * DV);
        if (!sp.last) pG = a.G + (la_place(a, plan, sp.s, sp.lo, sp.j + 1) * a.H + h) * ((int64_t)DK * DV);
        auto channels = [&](const float* kept, const float* given, int q, f32x4 (&v)[TPK]) {
#pragma unroll
            for (int e = 0; e < TPK; ++e) {
                const int c = KS * q + SL * lg + 4 * e;
                if (kept) {
                    v[e] = *(const f32x4*)(kept + (b0 + lr) * DV + c);
                } else if (given) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[e][r] = given[state + (int64_t)(c + r) * DK + b0 + lr];
                } else {
                    v[e] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            }
        };
        f32x4 s[KV][TPK];
#pragma unroll
        for (int q = 0; q < KV; ++q) channels(pS, a.init, q, s[q]);
        __builtin_amdgcn_sched_barrier(0);
        if (m == 0) {
            rk.store(sk);
            rq.store(sq);
        }
        if (threadIdx.x < GD_Q) {
            s_in[threadIdx.x] = rin;
            s_out[threadIdx.x] = rout;
            s_beta[threadIdx.x] = rbeta;
            c2[threadIdx.x] = rc;
        }
        if constexpr (L::DO) rd.store(sd);
        // U and Z in parts; dv, dbeta and v . dv from them
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int y = i * NTHR + threadIdx.x, row = y / VPR, c = y % VPR * 8;
            float zu = 0.f, vz = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                t4 o;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    zu += z[i][e][r] * u[i][e][r];
                    const float dv = be[i] * z[i][e][r];
                    vz += dv * (float)vv[i][e][r];
                    o[r] = (T)dv;
                }
                if (row < n) *(t4*)((T*)a.dv + (t0 + row) * a.dv_ts + (int64_t)h * DV + c + 4 * e) = o;
            }
#pragma unroll
            for (int o = 1; o < VPR; o <<= 1) {
                zu += __shfl_xor(zu, o, 64);
                vz += __shfl_xor(vz, o, 64);
            }
            if (y % VPR == 0) {
                zv[row] = vz;
                if (row < n) a.dbeta[(t0 + row) * a.H + h] = zu / (fabsf(be[i]) < GD_BETA_MIN ? copysignf(GD_BETA_MIN, be[i]) : be[i]);
            }
            // U of a beta smaller than the walk's, so that all of dk that is this token's has the given one as a factor
            const float share = fabsf(be[i]) < GD_BETA_MIN ? fabsf(be[i]) * (1.f / GD_BETA_MIN) : 1.f;
            u[i][0] *= share, u[i][1] *= share;
            if constexpr (sizeof(T) == 2) {
                Frag f[P::U], g[P::Z];
                gd_split<T, P::U>(u[i], f);
                gd_split<T, P::Z>(z[i], g);
#pragma unroll
                for (int p = 0; p < P::U; ++p) *(Frag*)(su + (p * GD_Q + row) * VP + c) = f[p];
#pragma unroll
                for (int p = 0; p < P::Z; ++p) *(Frag*)(sz + (p * GD_Q + row) * VP + c) = g[p];
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    *(f32x4*)(su + row * VP + c + 4 * e) = u[i][e];
                    *(f32x4*)(sz + row * VP + c + 4 * e) = z[i][e];
                }
            }
        }
        f32x4 g[KV][TPK];
#pragma unroll
        for (int q = 0; q < KV; ++q) channels(pG, a.dfin, q, g[q]);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();

        // k operands of value channels: rows of do, U, Z
        const __amdgpu_buffer_rsrc_t rdo = buf_rsrc(pd, n * (int)a.o_ts * (int)sizeof(T));
        auto d_row = [&](int t, int q) {
            if constexpr (L::DO) return M::load(sd + (16 * t + lr) * VP + KS * q + SL * lg);
            else return buf_load<Frag>(rdo, ((16 * t + lr) * (int)a.o_ts + KS * q + SL * lg) * (int)sizeof(T));
        };
        auto u_row = [&](int t, int q, int p) { return M::load(su + (p * GD_Q + 16 * t + lr) * VP + KS * q + SL * lg); };
        auto z_row = [&](int t, int q, int p) { return M::load(sz + (p * GD_Q + 16 * t + lr) * VP + KS * q + SL * lg); };

        // tiles of E and N, transposed: a lane has row i and columns j ..
        f32x4 E[PER], N[PER];
        auto tile_of = [&](int y, int* ti, int* tj) {  // of whole k blocks: rows b TPK .., columns up to there
            int b = 0, left = y;
            while (left >= (b + 1) * TPK * TPK) left -= (b + 1) * TPK * TPK, ++b;
            *ti = b * TPK + left / ((b + 1) * TPK);
            *tj = left % ((b + 1) * TPK);
        };
#pragma unroll
        for (int y = 0; y < PER; ++y) {
            E[y] = N[y] = f32x4{0.f, 0.f, 0.f, 0.f};
            const int no = y * NW + wave;
            if (no >= TILES) continue;
            int ti, tj;
            tile_of(no, &ti, &tj);
            if (tj > ti) continue;
#pragma unroll
            for (int q = 0; q < KV; ++q) {
                Frag uf[P::U], zf[P::Z];
#pragma unroll
                for (int p = 0; p < P::U; ++p) uf[p] = u_row(tj, q, p);
#pragma unroll
                for (int p = 0; p < P::Z; ++p) zf[p] = z_row(ti, q, p);
                const Frag d = d_row(ti, q);
                E[y] = gd_mma<T, P::U, 1>(uf, &d, E[y]);
                N[y] = gd_mma<T, P::Z, P::Z>(uf, zf, N[y]);
            }
            const int i = 16 * ti + lr, j = 16 * tj + 4 * lg;
            const float bi = s_beta[i];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float f = j + r <= i ? __builtin_amdgcn_exp2f((float)(c2[i] - c2[j + r])) : 0.f;
                E[y][r] = j + r <= i ? a.scale * f * E[y][r] : 0.f;
                N[y][r] = j + r < i ? bi * f * N[y][r] : 0.f;
            }
        }

        f32x4 dq[GD_NT], gu[GD_NT], sz_[GD_NT];
#pragma unroll
        for (int t = 0; t < GD_NT; ++t) dq[t] = gu[t] = sz_[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        float dot = 0.f;
#pragma unroll
        for (int q = 0; q < KV; ++q) {
#pragma unroll
            for (int e = 0; e < TPK; ++e)
#pragma unroll
                for (int r = 0; r < 4; ++r) dot += s[q][e][r] * g[q][e][r];
            Frag sf[P::U], gf[P::U];
            gd_split<T, P::U>(s[q], sf);
            gd_split<T, P::U>(g[q], gf);
#pragma unroll
            for (int t = 0; t < GD_NT; ++t) {
                Frag uf[P::U], zf[P::Z];
#pragma unroll
                for (int p = 0; p < P::U; ++p) uf[p] = u_row(t, q, p);
#pragma unroll
                for (int p = 0; p < P::Z; ++p) zf[p] = z_row(t, q, p);
                const Frag d = d_row(t, q);
                dq[t] = gd_mma<T, P::U, 1>(sf, &d, dq[t]);
                gu[t] = gd_mma<T, P::U, P::U>(gf, uf, gu[t]);
                sz_[t] = gd_mma<T, P::Z, P::Z>(sf, zf, sz_[t]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // <G, S behind> = e^C <G, S> + sum_j e^(C - c_j) k_j . (G u_j)
        dot *= s_in[n - 1];
#pragma unroll
        for (int t = 0; t < GD_NT; ++t) {
            const int i = 16 * t + lr;
            const t4 kv = *(const t4*)(sk + i * AP + b0 + 4 * lg);
            const float in = s_in[i], be = s_beta[i];
            gu[t] *= s_out[i];
#pragma unroll
            for (int r = 0; r < 4; ++r) dot += (float)kv[r] * gu[t][r];
            dq[t] *= a.scale * in;
            gu[t] -= sz_[t] * (in * be);
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o, 64);
        if (lane == 0) tot[wave] = dot;
        __syncthreads();  // U and Z are read
#pragma unroll
        for (int y = 0; y < PER; ++y) {
            const int no = y * NW + wave;
            if (no >= TILES) continue;
            int ti, tj;
            tile_of(no, &ti, &tj);
            T* pe = se + (16 * ti + lr) * L::EP + MatE::at(tj, lg);
            T* pn = sn + (16 * ti + lr) * L::NP + MatN::at(tj, lg);
            if constexpr (sizeof(T) == 2) {
                f32x4 two[2] = {E[y], N[y]};
                Frag f[P::E];
                gd_split<T, P::E>(two, f);  // the first four of a part are E's
#pragma unroll
                for (int p = 0; p < P::E; ++p) {
                    *(bf16x4*)(pe + p * GD_Q) = __builtin_shufflevector(f[p], f[p], 0, 1, 2, 3);
                    if (p < P::N) *(bf16x4*)(pn + p * GD_Q) = __builtin_shufflevector(f[p], f[p], 4, 5, 6, 7);
                }
            } else {
                *(f32x4*)pe = E[y];
                *(f32x4*)pn = N[y];
            }
        }
        __syncthreads();
        // dq += E K; dk += E^T Q - (N + N^T) K
#pragma unroll
        for (int b = 0; b < NK; ++b) {
            const Frag kf = XT<T>::load(sk, AP, KS * b, b0, lane), qf = XT<T>::load(sq, AP, KS * b, b0, lane);
            Frag nk = kf;
#pragma unroll
            for (int s = 0; s < SL; ++s) nk[s] = -kf[s];
#pragma unroll
            for (int t = b * TPK; t < GD_NT; ++t) {
                Frag ef[P::E], nf[P::N];
#pragma unroll
                for (int p = 0; p < P::E; ++p) ef[p] = MatE::row(se, t, b, p, lane);
#pragma unroll
                for (int p = 0; p < P::N; ++p) nf[p] = MatN::row(sn, t, b, p, lane);
                dq[t] = gd_mma<T, 1, P::E>(&kf, ef, dq[t]);
                gu[t] = gd_mma<T, 1, P::N>(&nk, nf, gu[t]);
            }
#pragma unroll
            for (int t = 0; t < (b + 1) * TPK; ++t) {
                Frag ef[P::N], nf[P::N];
#pragma unroll
                for (int p = 0; p < P::N; ++p) {
                    ef[p] = MatE::col(se, t, b, p, lane);
                    nf[p] = MatN::col(sn, t, b, p, lane);
                }
                gu[t] = gd_mma<T, 1, P::N>(&qf, ef, gu[t]);
                gu[t] = gd_mma<T, 1, P::N>(&nk, nf, gu[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < GD_NT; ++t) {
            const t4 qv = *(const t4*)(sq + (16 * t + lr) * AP + b0 + 4 * lg);
            float d = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) d += (float)qv[r] * dq[t][r];
            d += __shfl_xor(d, 16, 64);
            d += __shfl_xor(d, 32, 64);
            if (lg == 0) red[wave][16 * t + lr] = d;
            DQ[t] += dq[t];
            DKt[t] += gu[t];
        }
        __syncthreads();
        if (wave == 0) {  // dg_t: the sum from t on; zero, not the sum's roundings, where nothing before t is kept
            double d = -(double)zv[lane], all = 0.0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                d += (double)red[w][lane];
                all += (double)tot[w];
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double down = __shfl_down(d, o, 64);
                if (lane + o < 64) d += down;
            }
            const float keep = __builtin_amdgcn_exp2f((float)(c2[lane] - (lane > 0 ? c2[lane - 1] : 0.0)));
            if (lane < n) a.dg[(t0 + lane) * a.H + h] = keep == 0.f ? 0.f : (float)(d + all);
        }
    }

    if (a.sums) {
        const __amdgpu_buffer_rsrc_t r = buf_rsrc(a.sums + ((int64_t)h0 * a.tokens + t0) * (2 * DK), n * 2 * DK * 4);
#pragma unroll
        for (int t = 0; t < GD_NT; ++t) {
            buf_store(DQ[t], r, ((16 * t + lr) * 2 * DK + b0 + 4 * lg) * 4);
            buf_store(DKt[t], r, ((16 * t + lr) * 2 * DK + DK + b0 + 4 * lg) * 4);
        }
        return;
    }
    auto write = [&](const f32x4 (&v)[GD_NT], void* out, int64_t ts) {
        const int bytes = (int)ts * (int)sizeof(T);
        const __amdgpu_buffer_rsrc_t r = buf_rsrc((T*)out + t0 * ts + (int64_t)hk * DK, n * bytes);
        if constexpr (sizeof(T) == 2) {
            const int half = lg & 1, c8 = b0 + 8 * (lg >> 1);
#pragma unroll
            for (int t = 0; t < GD_NT; t += 2)
                buf_store(la_pair(v[t], v[t + 1]), r, (16 * (t + half) + lr) * bytes + c8 * 2);
        } else {
#pragma unroll
            for (int t = 0; t < GD_NT; ++t) buf_store(v[t], r, (16 * t + lr) * bytes + (b0 + 4 * lg) * 4);
        }
    };
    write(DQ, a.dq, a.dq_ts);
    write(DKt, a.dk, a.dk_ts);
}

// dq and dk of the tokens of all sequences, the sums of their heads' in order; four channels to a lane.
template <typename T>
__global__ void __launch_bounds__(256) k_gd_sum(GdArgs a) {
    const int64_t lo = seq_range(a, 0).lo, hi = seq_range(a, a.nseq - 1).hi;
    const int DK = a.keydim, quads = 2 * DK / 4, groups = a.H / a.share;
    typedef typename Vec4<T>::type vt;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < (hi - lo) * groups * quads; i += gridDim.x * 256ll) {
        const int c = (int)(i % quads) * 4, hk = (int)(i / quads % groups);
        const int64_t t = lo + i / quads / groups;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        for (int m = 0; m < a.share; ++m)
            v += *(const f32x4*)(a.sums + (((int64_t)hk * a.share + m) * a.tokens + t) * (2 * DK) + c);
        T* out = c < DK ? (T*)a.dq + t * a.dq_ts + hk * DK + c : (T*)a.dk + t * a.dk_ts + hk * DK + c - DK;
        *(vt*)out = vt{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    }
}

}  // namespace ssd
