// The walk of the gated delta rule from chunk to chunk (see gdelta.h): forward, and the same walk as
// the backward's recomputation (KEEP), which keeps entering states and u instead of outputs.
//
// A workgroup of NW waves walks 16 CT NW value channels of a head over its sequence.  The waves meet once
// per chunk, where the next chunk's operands have arrived; between, each goes its own way.  With one
// wave to a SIMD nothing hides an LDS read but the wave's own work: the operands of a product are read
// while the one before it runs, and the splitting of a result into parts is dealt out between the
// matrix instructions of the next product (gd_weave).
#pragma once

#include "gdelta.h"

namespace ssd {

template <typename T, int BD, int CT, int NW, int PT, bool KEEP>
struct GdWalkLds {
    static constexpr int PO = sizeof(T) == 2 ? 2 : 1;  // parts of P and of what else only meets outputs
    static constexpr int k = 0, v = k + GdTile<T, BD>::BYTES, t = v + GdTile<T, 16 * CT * NW>::BYTES,
                         sc = t + GdMat<T, PT>::BYTES, q = sc + (int)sizeof(GdScalars),
                         p = q + (KEEP ? 0 : GdTile<T, BD>::BYTES),
                         bytes = (p + (KEEP ? 0 : GdMat<T, PO>::BYTES) + 1023) / 1024 * 1024;
    static constexpr int buffers = 2 * bytes <= 160 * 1024 ? 2 : 1;
};

// PT: parts of T, R, states and u on their way into states (2, or 3 where a state is asked for).
template <typename T, int BD, int CT, int NW, int PT, bool KEEP>
__global__ void __launch_bounds__(64 * NW) k_gd_walk(GdArgs a, LaPlan plan) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    typedef GdWalkLds<T, BD, CT, NW, PT, KEEP> L;
    typedef GdTile<T, BD> Tile;
    typedef GdTile<T, 16 * CT * NW> TileV;
    constexpr int SL = M::SL, KS = M::KS, KB = BD / KS, TPK = LaCfg<T>::TPK, NK = GD_Q / KS;
    constexpr int BT = BD / 16, CDW = 16 * CT * NW, PO = L::PO, PE = 1;  // q, k and v are exact
    typedef GdMat<T, PT> MatT;
    typedef GdMat<T, PO> MatP;
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
    const T* pv = (const T*)a.v + (int64_t)h * DV + c0;
    const int64_t hrow = (int64_t)h * a.tokens;

    auto tokens_of = [&](int k) { return len - k * GD_Q < GD_Q ? len - k * GD_Q : GD_Q; };
    // The operands of chunk k, a fetch of each wave at a time: all at once they would hold up the waves
    // until the CU has accepted them.  The last chunk fetches itself again, so that no branch parts the code.
    struct Next {
        gd_i4 k, v, t, q, p;
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
        x.v = rows(pv, a.v_ts);
        x.t = gd_rsrc((const T*)a.T + x.row * MatT::D, x.n * MatT::ROW);
        if constexpr (!KEEP) {
            x.q = rows(pq, a.q_ts);
            x.p = gd_rsrc((const T*)a.P + x.row * MatP::D, x.n * MatP::ROW);
        }
        return x;
    };
    constexpr int FK = gd_share(Tile::FETCHES, NW), FT_ = gd_share(MatT::FETCHES, NW), FV = gd_share(TileV::FETCHES, NW);
    constexpr int FP = KEEP ? 0 : gd_share(MatP::FETCHES, NW), FQ_ = KEEP ? 0 : FK;
    constexpr int NF = FK + FT_ + FV + FP + FQ_ + gd_share(3, NW);
    auto fetch = [&](const Next& x, auto I) {
        constexpr int i = decltype(I)::value, at_t = FK, at_v = at_t + FT_, at_p = at_v + FV, at_q = at_p + FP, at_s = at_q + FQ_;
        const int es = (int)sizeof(T);
        if constexpr (i < at_t) Tile::fetch(x.k, (int)a.k_ts * es, x.to + L::k, gd_mine<Tile::FETCHES, NW>(i, wave), lane);
        else if constexpr (i < at_v) MatT::fetch(x.t, x.to + L::t, gd_mine<MatT::FETCHES, NW>(i - at_t, wave), lane);
        else if constexpr (i < at_p) TileV::fetch(x.v, (int)a.v_ts * es, x.to + L::v, gd_mine<TileV::FETCHES, NW>(i - at_v, wave), lane);
        else if constexpr (i < at_q) MatP::fetch(x.p, x.to + L::p, gd_mine<MatP::FETCHES, NW>(i - at_p, wave), lane);
        else if constexpr (i < at_s) Tile::fetch(x.q, (int)a.q_ts * es, x.to + L::q, gd_mine<Tile::FETCHES, NW>(i - at_q, wave), lane);
        else gd_scalars_fetch(a, x.row, x.n, x.to + L::sc, gd_mine<3, NW>(i - at_s, wave), lane);
    };
    auto stage_all = [&](int k) {
        const Next x = next_of(k, k);
        gd_for<NF>([&](auto I) { fetch(x, I); });
    };
    if (L::buffers == 2 && nch > 0) stage_all(0);

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
        if constexpr (L::buffers == 1) {
            __syncthreads();  // the last chunk's reads are done
            stage_all(k);
        }
        // behind this chunk's fetches stand only the last chunk's stores of u or of outputs
        constexpr int STORES = (KEEP ? 16 : (sizeof(T) == 2 ? 2 : 4)) * CT;
        if (L::buffers == 2 && k > 0) gd_wait<STORES>();
        else gd_wait<0>();
        __syncthreads();
        if (KEEP && k > 0) {
            float* S = a.S + (la_place(a, plan, it.s, lo, k) * a.H + h) * ((int64_t)BD * DV);
#pragma unroll
            for (int t = 0; t < BT; ++t)
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[(la_channel<T>(t, lg) + r) * DV + col + 16 * u] = St[t][u][r];
        }
        char* buf = lds + (L::buffers == 2 && k % 2 ? L::bytes : 0);
        char* sk = buf + L::k;
        const char *sv = buf + L::v, *st = buf + L::t, *sq = buf + L::q, *sp = buf + L::p;
        const GdScalars* sc = (const GdScalars*)(buf + L::sc);

        // A value of v that is not finite would reach the rows before its own: it counts as zero, and its
        // channel is made NaN from its row on further down; so is every channel from a row that prep
        // found bad, whose keys count as zero from there on (mend: for the whole workgroup).
        Frag vf[NK][CT];
        int first[CT];
        unsigned long long bad = 0;
        bool tame = true;
        auto mend = [&] {
            const int row = __ffsll(bad) - 1;
            __syncthreads();  // another wave may still read the flags, or these rows
            for (int i = threadIdx.x; i < (GD_Q - row) * Tile::RB / 16; i += 64 * NW)
                *(f32x4*)(sk + row * Tile::RB + i * 16) = f32x4{0.f, 0.f, 0.f, 0.f};
            __syncthreads();
        };
        auto check = [&] {
            float seen[2] = {0.f, 0.f};
#pragma unroll
            for (int b = 0; b < NK; ++b)
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int s = 0; s < SL; ++s) seen[s % 2] = __builtin_fmaf((float)vf[b][u][s], 0.f, seen[s % 2]);
            tame = !bad && __ballot(seen[0] + seen[1] != 0.f) == 0;  // NaN is not equal to zero
            if (tame) return;
#pragma unroll
            for (int u = 0; u < CT; ++u) {
                first[u] = bad ? __ffsll(bad) - 1 : GD_Q;
#pragma unroll
                for (int b = NK - 1; b >= 0; --b)
#pragma unroll
                    for (int s = SL - 1; s >= 0; --s)
                        if (!(fabsf((float)vf[b][u][s]) < INFINITY)) {
                            const int j = KS * b + 16 * (s / 4) + 4 * lg + s % 4;
                            first[u] = j < first[u] ? j : first[u];
                            vf[b][u][s] = (T)0.f;
                        }
                // the least of the four lane groups' rows
#pragma unroll
                for (int m = 16; m < 64; m <<= 1) {
                    const int y = __shfl_xor(first[u], m, 64);
                    first[u] = y < first[u] ? y : first[u];
                }
            }
        };

        f32x4 x[GD_NT][CT], o[GD_NT][CT];
#pragma unroll
        for (int t = 0; t < GD_NT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) x[t][u] = o[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (sizeof(T) == 2 && CT == 1) {
            // The products in turn, each with the work that the next ones need dealt out between its
            // instructions (fetch: also the next chunk's).
            unsigned c1 = 0x0000bf80u, c2 = 0xbf800000u;
            asm("" : "+s"(c1), "+s"(c2));
            constexpr int FX = KEEP ? NF / 2 : NF / 3;               // fetches during X
            constexpr int FQ = KEEP ? 0 : NF / 5, FT = NF - FX - FQ;  // during Q S^T, during T R
            // what later products read from LDS is asked for a product before
            Frag f[KB][GD_NT];
            auto keys = [&] {
#pragma unroll
                for (int q = 0; q < KB; ++q)
#pragma unroll
                    for (int t = 0; t < GD_NT; ++t) f[q][t] = Tile::row(sk, t, q, lane);
            };
            const float flag = KEEP ? 0.f : sc->out[lane];
            keys();
#pragma unroll
            for (int b = 0; b < NK; ++b) vf[b][0] = TileV::xt(sv, KS * b, cw, lane);
            f32x4 in[GD_NT], be[GD_NT], ou[GD_NT];
            float row[GD_NT];
#pragma unroll
            for (int t = 0; t < GD_NT; ++t) {
                in[t] = *(const f32x4*)(sc->in + 16 * t + 4 * lg);
                be[t] = *(const f32x4*)(sc->beta + 16 * t + 4 * lg);
                ou[t] = *(const f32x4*)(sc->out + 16 * t + 4 * lg);
                if (!KEEP) row[t] = sc->in[16 * t + lr];
            }
            const float keep = sc->in[n - 1];
            __builtin_amdgcn_sched_barrier(0);
            const Next nx = next_of(k + 1 < nch ? k + 1 : k, k + 1);
            auto get = [&](auto I) { fetch(nx, I); };
            GdSplit<PT> s[KB];
            s[0].set(St[0][0], St[1][0]);
            gd_for<GdSplit<PT>::STEPS>([&](auto I) { s[0].template step<decltype(I)::value>(c1, c2); });
            if constexpr (!KEEP) {
                bad = __ballot(flag < 0.f);
                if (bad) {
                    mend();
                    keys();
                }
            }
            __builtin_amdgcn_sched_barrier(0);

            // X = K S^T; between: the parts of the next k block's states
            Frag tf[2][PT], tg[2][NK][PT], pf[GD_NT][PO], kt[BT];
            auto read_tg = [&](auto I) {
                constexpr int e = decltype(I)::value / (NK * PT), b = decltype(I)::value / PT % NK, p = decltype(I)::value % PT;
                tg[e][b][p] = MatT::row(st, 2 + e, b, p, lane);
            };
            constexpr int TG = 2 * NK * PT;
            gd_for<KB>([&](auto Q) {
                constexpr int q = decltype(Q)::value, more = q + 1 < KB;
                constexpr int f0 = q * FX / KB, f1 = (q + 1) * FX / KB, ns = more ? GdSplit<PT>::STEPS : 0;
                if constexpr (more) s[more ? q + 1 : 0].set(St[(more ? q + 1 : 0) * 2][0], St[(more ? q + 1 : 0) * 2 + 1][0]);
                gd_weave<4 * PT, ns + f1 - f0, 0>(
                    [&](auto I) {
                        constexpr int t = decltype(I)::value % 4, p = PT - 1 - decltype(I)::value / 4;
                        x[t][0] = M::mma(f[q][t], s[q].f[p], x[t][0]);
                    },
                    [&](auto I) {
                        constexpr int i = decltype(I)::value;
                        if constexpr (i < ns) s[more ? q + 1 : 0].template step<i>(c1, c2);
                        else get(std::integral_constant<int, f0 + i - ns>{});
                    });
                if constexpr (!KEEP)
#pragma unroll
                    for (int t = 0; t < GD_NT; ++t) f[q][t] = Tile::row(sq, t, q, lane);
                if constexpr (q == KB - 2)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int p = 0; p < PT; ++p) tf[e][p] = MatT::row(st, e, 0, p, lane);
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (!KEEP) check();

            // S Q^T; between: R = B (V - e^c X) and its parts
            GdSplit<PT> r[NK];
            auto rest = [&](auto I) {  // R's steps: per block 8 values, then their parts
                constexpr int i = decltype(I)::value, per = 8 + GdSplit<PT>::STEPS, b = i / per, j = i % per;
                if constexpr (j < 8) {
                    constexpr int t = 2 * b + j / 4, e = j % 4;
                    r[b].x[j] = be[t][e] * ((float)vf[b][0][j] - in[t][e] * x[t][0][e]);
                } else {
                    r[b].template step<j - 8>(c1, c2);
                }
            };
            constexpr int RS = NK * (8 + GdSplit<PT>::STEPS);
            if constexpr (KEEP) {
                gd_for<TG>([&](auto I) { read_tg(I); });
                gd_for<RS>([&](auto I) { rest(I); });
            } else {
                gd_weave<4 * PO * KB, RS + FQ + TG, 2>(
                    [&](auto I) {
                        constexpr int q = decltype(I)::value / (4 * PO), j = decltype(I)::value % (4 * PO), t = j % 4, p = PO - 1 - j / 4;
                        o[t][0] = M::mma(s[q].f[p], f[q][t], o[t][0]);
                    },
                    [&](auto I) {
                        constexpr int i = decltype(I)::value;
                        if constexpr (i < RS) rest(I);
                        else if constexpr (i < RS + FQ) get(std::integral_constant<int, FX + i - RS>{});
                        else read_tg(std::integral_constant<int, i - RS - FQ>{});
                    });
            }

            // U = T R, row tiles 0 and 1; between: S <- e^C S, O <- scale e^c O
            typedef GdPairs<PT> Pairs;
            f32x4 y[GD_NT];
#pragma unroll
            for (int t = 0; t < GD_NT; ++t) y[t] = f32x4{0.f, 0.f, 0.f, 0.f};
            constexpr int SS = BT * 2 + (KEEP ? 0 : GD_NT * 2), FT0 = FT / 3;  // pieces of two products each
            constexpr int PF = KEEP ? 0 : GD_NT * PO;
            gd_weave<2 * Pairs::N, SS + FT0 + PF, 0>(
                [&](auto I) {
                    constexpr int e = decltype(I)::value % 2, j = decltype(I)::value / 2;
                    y[e] = M::mma(tf[e][Pairs::a(j)], r[0].f[Pairs::b(j)], y[e]);
                },
                [&](auto I) {
                    constexpr int i = decltype(I)::value, t = i / 2, e = i % 2 * 2;
                    if constexpr (i < 2 * BT) {
                        St[t][0][e] *= keep;
                        St[t][0][e + 1] *= keep;
                    } else if constexpr (i < SS) {
                        constexpr int u = t - BT;
                        if constexpr (e == 0) row[u] *= a.scale;
                        o[u][0][e] *= row[u];
                        o[u][0][e + 1] *= row[u];
                    } else if constexpr (i < SS + FT0) {
                        get(std::integral_constant<int, FX + FQ + i - SS>{});
                    } else {
                        constexpr int j = i - SS - FT0;
                        pf[j / PO][j % PO] = MatP::row(sp, j / PO, 0, j % PO, lane);
                    }
                });

            // row tiles 2 and 3; between: the parts of the first two tiles of U, weighted for S and plain for O
            GdSplit<PT> w;
            GdSplit<PO> v;
            auto parts = [&](auto I, int t) {  // of tiles t, t + 1: weighted ones, then plain ones
                constexpr int i = decltype(I)::value, WS = 8 + GdSplit<PT>::STEPS;
                if constexpr (i < 8) w.x[i] = y[t + i / 4][i % 4] * ou[t + i / 4][i % 4];
                else if constexpr (i < WS) w.template step<i - 8>(c1, c2);
                else if constexpr (i < WS + 1) v.set(y[t], y[t + 1]);
                else v.template step<i - WS - 1>(c1, c2);
            };
            constexpr int WS = 8 + GdSplit<PT>::STEPS, US = WS + (KEEP ? 0 : 1 + GdSplit<PO>::STEPS);
            gd_weave<4 * Pairs::N, US + FT - FT0 + BT, 0>(
                [&](auto I) {
                    constexpr int b = decltype(I)::value / (2 * Pairs::N), i = decltype(I)::value % (2 * Pairs::N), e = i % 2, j = i / 2;
                    y[2 + e] = M::mma(tg[e][b][Pairs::a(j)], r[b].f[Pairs::b(j)], y[2 + e]);
                },
                [&](auto I) {
                    constexpr int i = decltype(I)::value;
                    if constexpr (i < US) parts(I, 0);
                    else if constexpr (i < US + FT - FT0) get(std::integral_constant<int, FX + FQ + FT0 + i - US>{});
                    else kt[i - US - FT + FT0] = Tile::bt(sk, 0, i - US - FT + FT0, lane);
                });
            if constexpr (KEEP) {
                const __amdgpu_buffer_rsrc_t ru = buf_rsrc(a.U + (hrow + t0) * DV, n * DV * 4);
#pragma unroll
                for (int t = 0; t < GD_NT; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[t][q]), ru,
                                                              ((16 * t + 4 * lg + q) * DV + col) * 4, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);

            // O += P U and S += K^T U over the first block of tokens; between: the parts of the others
            GdSplit<PT> w0 = w;
            Frag pg[2][PO], kn[BT];
            if constexpr (!KEEP) {
                GdSplit<PO> v0 = v;
                gd_weave<4 * GdPairs<PO>::N, 8 + 2 * PO, 0>(
                    [&](auto I) {
                        constexpr int t = decltype(I)::value % 4, j = decltype(I)::value / 4;
                        o[t][0] = M::mma(v0.f[GdPairs<PO>::a(j)], pf[t][GdPairs<PO>::b(j)], o[t][0]);
                    },
                    [&](auto I) {
                        constexpr int i = decltype(I)::value;
                        if constexpr (i < 8) parts(I, 2);
                        else pg[(i - 8) / PO][(i - 8) % PO] = MatP::row(sp, 2 + (i - 8) / PO, 1, (i - 8) % PO, lane);
                    });
            }
            constexpr int done = KEEP ? 0 : 8;
            gd_weave<BT * PT, US - done + BT, 0>(
                [&](auto I) {
                    constexpr int t = decltype(I)::value % BT, p = PT - 1 - decltype(I)::value / BT;
                    St[t][0] = M::mma(kt[t], w0.f[p], St[t][0]);
                },
                [&](auto I) {
                    constexpr int i = decltype(I)::value;
                    if constexpr (i < BT) kn[i] = Tile::bt(sk, KS, i, lane);
                    else parts(std::integral_constant<int, i - BT + done>{}, 2);
                });
            // and over the second; between: the outputs
            if constexpr (!KEEP)
                gd_for<2 * GdPairs<PO>::N>([&](auto I) {
                    constexpr int e = decltype(I)::value % 2, j = decltype(I)::value / 2;
                    o[2 + e][0] = M::mma(v.f[GdPairs<PO>::a(j)], pg[e][GdPairs<PO>::b(j)], o[2 + e][0]);
                });
            gd_for<BT * PT>([&](auto I) {
                constexpr int t = decltype(I)::value % BT, p = PT - 1 - decltype(I)::value / BT;
                St[t][0] = M::mma(kn[t], w.f[p], St[t][0]);
            });
        } else {
        const Next nx = next_of(k + 1 < nch ? k + 1 : k, k + 1);
        // the fetches of the I-th of N places in what follows
        constexpr int PLACES = KEEP ? KB + 3 : 2 * KB + 3 + 2 * NK;
        auto ahead = [&](auto I) {
            constexpr int i = decltype(I)::value, from = i * NF / PLACES, to = (i + 1) * NF / PLACES;
            if constexpr (L::buffers == 2) gd_for<to - from>([&](auto J) { fetch(nx, std::integral_constant<int, from + decltype(J)::value>{}); });
        };
        if constexpr (!KEEP) {
            bad = __ballot(sc->out[lane] < 0.f);
            if (bad) mend();
        }
#pragma unroll
        for (int b = 0; b < NK; ++b)
#pragma unroll
            for (int u = 0; u < CT; ++u) vf[b][u] = TileV::xt(sv, KS * b, cw + 16 * u, lane);
        if constexpr (!KEEP) check();
        // X = K S^T and S Q^T
        Frag sf[KB][CT][PT], f[KB][GD_NT];
#pragma unroll
        for (int q = 0; q < KB; ++q)
#pragma unroll
            for (int t = 0; t < GD_NT; ++t) f[q][t] = Tile::row(sk, t, q, lane);
        if constexpr (sizeof(T) == 2) __builtin_amdgcn_sched_barrier(0);
        gd_for<KB>([&](auto Q) {
            constexpr int q = decltype(Q)::value;
#pragma unroll
            for (int u = 0; u < CT; ++u) {
                f32x4 tl[TPK];
#pragma unroll
                for (int e = 0; e < TPK; ++e) tl[e] = St[q * TPK + e][u];
                gd_split<T, PT>(tl, sf[q][u]);
            }
#pragma unroll
            for (int p = PT - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < GD_NT; ++t)
#pragma unroll
                    for (int u = 0; u < CT; ++u) x[t][u] = M::mma(f[q][t], sf[q][u][p], x[t][u]);
            if constexpr (!KEEP)
#pragma unroll
                for (int t = 0; t < GD_NT; ++t) f[q][t] = Tile::row(sq, t, q, lane);
            ahead(Q);
        });
        if constexpr (!KEEP)
            gd_for<KB>([&](auto Q) {
                constexpr int q = decltype(Q)::value;
#pragma unroll
                for (int p = PO - 1; p >= 0; --p)
#pragma unroll
                    for (int t = 0; t < GD_NT; ++t)
#pragma unroll
                        for (int u = 0; u < CT; ++u) o[t][u] = M::mma(sf[q][u][p], f[q][t], o[t][u]);
                ahead(std::integral_constant<int, KB + q>{});
            });
        constexpr int AFTER = KEEP ? KB : 2 * KB;

        // R = B (V - e^c X), U = T R
        Frag rf[NK][CT][PT];
#pragma unroll
        for (int b = 0; b < NK; ++b)
#pragma unroll
            for (int u = 0; u < CT; ++u) {
                f32x4 tl[TPK];
#pragma unroll
                for (int e = 0; e < TPK; ++e) {
                    const int t = b * TPK + e;
                    const f32x4 in = *(const f32x4*)(sc->in + 16 * t + 4 * lg);
                    const f32x4 be = *(const f32x4*)(sc->beta + 16 * t + 4 * lg);
#pragma unroll
                    for (int r = 0; r < 4; ++r) tl[e][r] = be[r] * ((float)vf[b][u][4 * e + r] - in[r] * x[t][u][r]);
                }
                gd_split<T, PT>(tl, rf[b][u]);
            }
#pragma unroll
        for (int t = 0; t < GD_NT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) x[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
        // two row tiles at a time, so that neighbouring instructions do not wait for each other
        gd_for<2>([&](auto H) {
            constexpr int h2 = 2 * decltype(H)::value;
#pragma unroll
            for (int b = 0; b * TPK <= h2 + 1; ++b) {
                Frag tf[2][PT];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (b * TPK <= h2 + e)
#pragma unroll
                        for (int p = 0; p < PT; ++p) tf[e][p] = MatT::row(st, h2 + e, b, p, lane);
#pragma unroll
                for (int s = PT - 1; s >= 0; --s)
#pragma unroll
                    for (int p = 0; p <= s; ++p)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (b * TPK <= h2 + e)
#pragma unroll
                                for (int u = 0; u < CT; ++u)
                                    x[h2 + e][u] = M::mma(tf[e][p], rf[b][u][s - p], x[h2 + e][u]);
            }
            ahead(std::integral_constant<int, AFTER + decltype(H)::value>{});
        });
        ahead(std::integral_constant<int, AFTER + 2>{});
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
            gd_for<NK>([&](auto B) {
                constexpr int b = decltype(B)::value;
                Frag uf[CT][PO];
#pragma unroll
                for (int u = 0; u < CT; ++u) {
                    f32x4 tl[TPK];
#pragma unroll
                    for (int e = 0; e < TPK; ++e) tl[e] = x[b * TPK + e][u];
                    gd_split<T, PO>(tl, uf[u]);
                }
                Frag pf[GD_NT][PO];
#pragma unroll
                for (int t = b * TPK; t < GD_NT; ++t)
#pragma unroll
                    for (int p = 0; p < PO; ++p) pf[t][p] = MatP::row(sp, t, b, p, lane);
#pragma unroll
                for (int s = PO - 1; s >= 0; --s)
#pragma unroll
                    for (int p = 0; p <= s; ++p)
#pragma unroll
                        for (int t = b * TPK; t < GD_NT; ++t)
#pragma unroll
                            for (int u = 0; u < CT; ++u) o[t][u] = M::mma(uf[u][p], pf[t][s - p], o[t][u]);
                ahead(std::integral_constant<int, AFTER + 3 + b>{});
            });
        }

        // S <- e^C S + sum_j e^(C - c_j) u_j k_j^T
        const float keep = sc->in[n - 1];
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) St[t][u] *= keep;
        gd_for<NK>([&](auto B) {
            constexpr int b = decltype(B)::value;
            Frag uf[CT][PT];
#pragma unroll
            for (int u = 0; u < CT; ++u) {
                f32x4 tl[TPK];
#pragma unroll
                for (int e = 0; e < TPK; ++e)
                    tl[e] = x[b * TPK + e][u] * *(const f32x4*)(sc->out + 16 * (b * TPK + e) + 4 * lg);
                gd_split<T, PT>(tl, uf[u]);
            }
            Frag f[BT];
#pragma unroll
            for (int t = 0; t < BT; ++t) f[t] = Tile::bt(sk, KS * b, t, lane);
            if constexpr (!KEEP) ahead(std::integral_constant<int, AFTER + 3 + NK + b>{});
#pragma unroll
            for (int p = PT - 1; p >= 0; --p)
#pragma unroll
                for (int t = 0; t < BT; ++t)
#pragma unroll
                    for (int u = 0; u < CT; ++u) St[t][u] = M::mma(f[t], uf[u][p], St[t][u]);
        });

        }

        if constexpr (!KEEP) {
            if (!tame) {
#pragma unroll
                for (int u = 0; u < CT; ++u) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int f = __shfl(first[u], 4 * lg + r, 64);
#pragma unroll
                        for (int t = 0; t < GD_NT; ++t)
                            if (16 * t + lr >= f) o[t][u][r] = NAN;
                    }
                    if (first[u] < GD_Q)
#pragma unroll
                        for (int t = 0; t < BT; ++t) St[t][u] = f32x4{NAN, NAN, NAN, NAN};
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
    }
    gd_wait<0>();  // a workgroup's LDS is another's once its waves have ended
    if (!KEEP && a.fin) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) *(f32x4*)(a.fin + state_at + at(t, u)) = St[t][u];
    }
}

}  // namespace ssd
