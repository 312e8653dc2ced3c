// The walks of the gated delta rule (see gdelta.h) by teams: the four waves of a workgroup share 16 value
// channels, where a wave each would leave most of the chip idle.
//
// One wave issues some thousand instructions per chunk and 16 channels, so that the shard's 256 column tiles
// (2 rows, 32 heads of 64 channels) keep 256 of 1024 SIMDs busy for 460 us; teams take 300.  Here wave w owns a quarter
// of the state's key channels and token tile w of X, R, U and O, and what one has and all need
// goes through LDS in parts, as operands:
//   parts of S  |  X_w = K_w S^T, parts of R_w  |  U_w = T_w R, its parts  |  O_w, its channels of S
// with a barrier at each bar.  An operand is fetched into LDS as soon as its place is free: a chunk
// ahead of its use at most.
#pragma once

#include "gdelta.h"

namespace ssd {

// Operands of one column tile in parts: tile t of a [k][16] matrix, 4 rows to a lane, is half of k block
// t / 2 (float32: all of block t).
template <typename T, int P>
struct GdShared {
    typedef typename Mma<T>::Frag Frag;
    static constexpr int TPK = LaCfg<T>::TPK;
    static constexpr int bytes(int tiles) { return tiles / TPK * P * 1024; }
    __device__ static __forceinline__ void put(char* m, int t, f32x4 v, int lane) {
        if constexpr (sizeof(T) == 4) {
            *(f32x4*)(m + t * 1024 + lane * 16) = v;
        } else {
            typedef __bf16 b2 __attribute__((ext_vector_type(2)));
            unsigned first = 0x0000bf80u, second = 0xbf800000u;
            asm("" : "+s"(first), "+s"(second));
            char* at = m + t / 2 * (P * 1024) + lane * 16 + t % 2 * 8;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const b2 x = {(bf16)v[0], (bf16)v[1]}, y = {(bf16)v[2], (bf16)v[3]};
                *(bf16x4*)(at + p * 1024) = bf16x4{x[0], x[1], y[0], y[1]};
                if (p < P - 1) {
                    v[0] = __builtin_amdgcn_fdot2_f32_bf16(x, __builtin_bit_cast(b2, first), v[0], false);
                    v[1] = __builtin_amdgcn_fdot2_f32_bf16(x, __builtin_bit_cast(b2, second), v[1], false);
                    v[2] = __builtin_amdgcn_fdot2_f32_bf16(y, __builtin_bit_cast(b2, first), v[2], false);
                    v[3] = __builtin_amdgcn_fdot2_f32_bf16(y, __builtin_bit_cast(b2, second), v[3], false);
                }
            }
        }
    }
    __device__ static __forceinline__ Frag get(const char* m, int b, int p, int lane) {
        return *(const Frag*)(m + (b * P + p) * 1024 + lane * 16);
    }
};

template <typename T, int BD, int PT, bool KEEP>
struct GdTeamLds {
    static constexpr int PO = sizeof(T) == 2 ? 2 : 1;
    static constexpr int k = 0, sc = k + 2 * GdTile<T, BD>::BYTES, t = sc + 2 * 1024, q = t + GdMat<T, PT>::BYTES,
                         v = q + (KEEP ? 0 : GdTile<T, BD>::BYTES), p = v + GdTile<T, 16>::BYTES,
                         sx = p + (KEEP ? 0 : GdMat<T, PO>::BYTES), rx = sx + GdShared<T, PT>::bytes(BD / 16),
                         ux = rx + GdShared<T, PT>::bytes(4), up = ux + GdShared<T, PT>::bytes(4),
                         wild = up + (KEEP ? 0 : GdShared<T, PO>::bytes(4)), bytes = wild + 256;
};

// As k_gd_walk: forward, or the backward's recomputation (KEEP).
template <typename T, int BD, int PT, bool KEEP>
__global__ void __launch_bounds__(256) k_gd_team(GdArgs a, LaPlan plan) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    typedef GdTeamLds<T, BD, PT, KEEP> L;
    typedef GdTile<T, BD> Tile;
    typedef GdTile<T, 16> TileV;
    constexpr int KS = M::KS, KB = BD / KS, TPK = LaCfg<T>::TPK, NK = GD_Q / KS, PO = L::PO;
    constexpr int OT = BD / 64;  // tiles of S^T of a wave
    typedef GdMat<T, PT> MatT;
    typedef GdMat<T, PO> MatP;
    typedef GdShared<T, PT> ShT;
    typedef GdShared<T, PO> ShO;
    __shared__ __align__(1024) char lds[L::bytes];
    int* wild = (int*)(lds + L::wild);  // [2]: some value of v is not finite; [2][16]: its first row

    const int DV = a.valdim;
    const GdItem it = gd_item(a, DV / 16);
    if (it.s < 0) return;
    const int h = it.h, w = wave_id(), lane = threadIdx.x % 64, lr = lane % 16, lg = lane / 16;
    const SeqRange sr = seq_range(a, it.s);
    const int64_t lo = sr.lo;
    const int len = (int)(sr.hi - sr.lo), nch = (len + GD_Q - 1) / GD_Q;
    const int c0 = it.cb * 16, col = c0 + lr;
    const T* pq = (const T*)a.q + (int64_t)(h / a.share) * BD;
    const T* pk = (const T*)a.k + (int64_t)(h / a.share) * BD;
    const T* pv = (const T*)a.v + (int64_t)h * DV + c0;
    const int64_t hrow = (int64_t)h * a.tokens;
    const int es = (int)sizeof(T);

    // fetches of a wave
    constexpr int FK = gd_share(Tile::FETCHES, 4), FT = gd_share(MatT::FETCHES, 4), FV = gd_share(TileV::FETCHES, 4);
    constexpr int FP = KEEP ? 0 : gd_share(MatP::FETCHES, 4), FQ = KEEP ? 0 : FK;
    auto tokens_of = [&](int k) { return len - k * GD_Q < GD_Q ? len - k * GD_Q : GD_Q; };
    auto rows = [&](const T* base, int64_t ts, int k) {
        return gd_rsrc(base + (lo + (int64_t)k * GD_Q) * ts, tokens_of(k) * (int)ts * es);
    };
    auto get_k = [&](int k, int buffer) {
        const gd_i4 r = rows(pk, a.k_ts, k);
        const unsigned to = gd_lds(lds + L::k + buffer % 2 * Tile::BYTES);
        gd_for<FK>([&](auto I) { Tile::fetch(r, (int)a.k_ts * es, to, gd_mine<Tile::FETCHES, 4>(decltype(I)::value, w), lane); });
        gd_scalars_fetch(a, hrow + lo + (int64_t)k * GD_Q, tokens_of(k), gd_lds(lds + L::sc + buffer % 2 * 1024),
                         gd_mine<3, 4>(0, w), lane);
    };
    auto get_qv = [&](int k) {
        if constexpr (!KEEP) {
            const gd_i4 r = rows(pq, a.q_ts, k);
            gd_for<FQ>([&](auto I) {
                Tile::fetch(r, (int)a.q_ts * es, gd_lds(lds + L::q), gd_mine<Tile::FETCHES, 4>(decltype(I)::value, w), lane);
            });
        }
        const gd_i4 r = rows(pv, a.v_ts, k);
        gd_for<FV>([&](auto I) {
            TileV::fetch(r, (int)a.v_ts * es, gd_lds(lds + L::v), gd_mine<TileV::FETCHES, 4>(decltype(I)::value, w), lane);
        });
    };
    auto get_t = [&](int k) {
        const gd_i4 r = gd_rsrc((const T*)a.T + (hrow + lo + (int64_t)k * GD_Q) * MatT::D, tokens_of(k) * MatT::ROW);
        gd_for<FT>([&](auto I) { MatT::fetch(r, gd_lds(lds + L::t), gd_mine<MatT::FETCHES, 4>(decltype(I)::value, w), lane); });
    };
    auto get_p = [&](int k) {
        if constexpr (!KEEP) {
            const gd_i4 r = gd_rsrc((const T*)a.P + (hrow + lo + (int64_t)k * GD_Q) * MatP::D, tokens_of(k) * MatP::ROW);
            gd_for<FP>([&](auto I) { MatP::fetch(r, gd_lds(lds + L::p), gd_mine<MatP::FETCHES, 4>(decltype(I)::value, w), lane); });
        }
    };
    if (nch > 0) {
        get_k(0, 0);
        get_qv(0);
        get_t(0);
    }
    if (!KEEP && threadIdx.x < 34) wild[threadIdx.x] = threadIdx.x < 2 ? 0 : GD_Q;

    // this wave's tiles of S^T: channels la_channel(OT w + i, lg) .. of k, channel `col` of v
    f32x4 St[OT];
    const int64_t state_at = ((int64_t)it.s * a.H + h) * ((int64_t)BD * DV);
    auto at = [&](int i) { return col * BD + la_channel<T>(OT * w + i, lg); };
#pragma unroll
    for (int i = 0; i < OT; ++i)
        St[i] = a.init ? *(const f32x4*)(a.init + state_at + at(i)) : f32x4{0.f, 0.f, 0.f, 0.f};

    for (int k = 0; k < nch; ++k) {
        const int n = tokens_of(k), next = k + 1 < nch ? k + 1 : k, par = k % 2;
        const int64_t t0 = lo + (int64_t)k * GD_Q;
        char* sk = lds + L::k + par * Tile::BYTES;
        const GdScalars* sc = (const GdScalars*)(lds + L::sc + par * 1024);
        // ---- parts of S
#pragma unroll
        for (int i = 0; i < OT; ++i) ShT::put(lds + L::sx, OT * w + i, St[i], lane);
        // behind the keys, queries and values of this chunk: T, and the last chunk's stores of u or outputs
        if (k > 0) gd_wait<FT + (KEEP ? 4 : 1)>();
        else gd_wait<FT>();
        __syncthreads();
        if (KEEP && k > 0) {
            float* S = a.S + (la_place(a, plan, it.s, lo, k) * a.H + h) * ((int64_t)BD * DV);
#pragma unroll
            for (int i = 0; i < OT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[(la_channel<T>(OT * w + i, lg) + r) * DV + col] = St[i][r];
        }
        unsigned long long bad = 0;
        if constexpr (!KEEP) {
            if (threadIdx.x < 17) wild[threadIdx.x == 16 ? 1 - par : 2 + 16 * (1 - par) + threadIdx.x] = threadIdx.x == 16 ? 0 : GD_Q;
            bad = __ballot(sc->out[lane] < 0.f);
            if (bad) {  // for the whole workgroup: keys count as zero from the row on that prep found bad
                const int row = __ffsll(bad) - 1;
                for (int i = threadIdx.x; i < (GD_Q - row) * Tile::RB / 16; i += 256)
                    *(f32x4*)(sk + row * Tile::RB + i * 16) = f32x4{0.f, 0.f, 0.f, 0.f};
                __syncthreads();
            }
        }
        get_p(k);
        get_k(next, k + 1);

        // ---- X_w = K_w S^T (token rows), O_w = S Q_w^T (channel rows), R_w = B (V - e^c X)
        f32x4 x = {0.f, 0.f, 0.f, 0.f}, x2 = x, o = x, o2 = x;
        {
            Frag kf[KB], qf[KB];
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                kf[q] = Tile::row(sk, w, q, lane);
                if (!KEEP) qf[q] = Tile::row(lds + L::q, w, q, lane);
            }
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                Frag s[PT];
#pragma unroll
                for (int p = 0; p < PT; ++p) s[p] = ShT::get(lds + L::sx, q, p, lane);
#pragma unroll
                for (int p = PT - 1; p >= 0; --p) {
                    f32x4& y = q % 2 ? x2 : x;
                    y = M::mma(kf[q], s[p], y);
                    if (!KEEP && p < PO) {
                        f32x4& z = q % 2 ? o2 : o;
                        z = M::mma(s[p], qf[q], z);
                    }
                }
            }
        }
        x += x2;
        o += o2;
        const f32x4 in = *(const f32x4*)(sc->in + 16 * w + 4 * lg), be = *(const f32x4*)(sc->beta + 16 * w + 4 * lg);
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * w + 4 * lg + r;
            v[r] = (float)*(const T*)(lds + L::v + TileV::at(row, lr * es / 16) + lr * es % 16);
        }
        if constexpr (!KEEP) {
            // a value that is not finite counts as zero and makes its channel NaN from its row on
            const float seen = (v[0] * 0.f + v[1] * 0.f) + (v[2] * 0.f + v[3] * 0.f);
            if (__ballot(seen != 0.f)) {
#pragma unroll
                for (int r = 3; r >= 0; --r)
                    if (!(fabsf(v[r]) < INFINITY)) {
                        v[r] = 0.f;
                        atomicMin(wild + 2 + 16 * par + lr, 16 * w + 4 * lg + r);
                        wild[par] = 1;
                    }
            }
        }
        ShT::put(lds + L::rx, w, be * (v - in * x), lane);
        gd_wait<FP + FK + 1>();  // T is there; behind it P and the next keys
        __syncthreads();
        get_qv(next);

        // ---- U_w = T_w R
        const int nb = w / TPK + 1;
        f32x4 u = {0.f, 0.f, 0.f, 0.f}, u2 = u;
#pragma unroll
        for (int b = 0; b < NK; ++b)
            if (b < nb) {
                Frag t[PT], r[PT];
#pragma unroll
                for (int p = 0; p < PT; ++p) {
                    t[p] = *(const Frag*)(lds + L::t + (MatT::tb(w, b) * PT + p) * 1024 + MatT::slot(lg, lr) * 16);
                    r[p] = ShT::get(lds + L::rx, b, p, lane);
                }
#pragma unroll
                for (int j = 0; j < GdPairs<PT>::N; ++j) {
                    f32x4& y = j % 2 ? u2 : u;
                    y = M::mma(t[GdPairs<PT>::a(j)], r[GdPairs<PT>::b(j)], y);
                }
            }
        u += u2;
        ShT::put(lds + L::ux, w, u * *(const f32x4*)(sc->out + 16 * w + 4 * lg), lane);
        if constexpr (KEEP) {
            const __amdgpu_buffer_rsrc_t r = buf_rsrc(a.U + (hrow + t0) * DV, n * DV * 4);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(u[q]), r, ((16 * w + 4 * lg + q) * DV + col) * 4, 0, 0);
        } else {
            ShO::put(lds + L::up, w, u, lane);
            gd_wait<FK + 1 + FQ + FV>();  // P is there
        }
        const float keep = sc->in[n - 1], row = KEEP ? 0.f : sc->in[16 * w + lr];
        __syncthreads();
        get_t(next);

        // ---- its channels of S, O_w
        Frag kt[OT][NK];
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
            for (int b = 0; b < NK; ++b) kt[i][b] = Tile::bt(sk, KS * b, OT * w + i, lane);
#pragma unroll
        for (int i = 0; i < OT; ++i) St[i] *= keep;
#pragma unroll
        for (int b = 0; b < NK; ++b) {
            Frag f[PT];
#pragma unroll
            for (int p = 0; p < PT; ++p) f[p] = ShT::get(lds + L::ux, b, p, lane);
#pragma unroll
            for (int p = PT - 1; p >= 0; --p)
#pragma unroll
                for (int i = 0; i < OT; ++i) St[i] = M::mma(kt[i][b], f[p], St[i]);
        }
        if constexpr (!KEEP) {
            o *= a.scale * row;
#pragma unroll
            for (int b = 0; b < NK; ++b)
                if (b < nb) {
                    Frag p_[PO], f[PO];
#pragma unroll
                    for (int p = 0; p < PO; ++p) {
                        p_[p] = *(const Frag*)(lds + L::p + (MatP::tb(w, b) * PO + p) * 1024 + MatP::slot(lg, lr) * 16);
                        f[p] = ShO::get(lds + L::up, b, p, lane);
                    }
                    o = gd_mma<T, PO, PO>(f, p_, o);
                }
            const bool any = __builtin_amdgcn_readfirstlane(wild[par]);
            if (any || bad) {
                const int from = bad ? __ffsll(bad) - 1 : GD_Q;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int f = wild[2 + 16 * par + 4 * lg + r];
                    if (16 * w + lr >= (f < from ? f : from)) o[r] = NAN;
                }
                const int f = wild[2 + 16 * par + lr];
                if ((f < from ? f : from) < GD_Q)
#pragma unroll
                    for (int i = 0; i < OT; ++i) St[i] = f32x4{NAN, NAN, NAN, NAN};
            }
            const int out_bytes = (int)a.o_ts * es;
            const __amdgpu_buffer_rsrc_t r = buf_rsrc((T*)a.o + t0 * a.o_ts + (int64_t)h * DV + c0, n * out_bytes);
            const int off = (16 * w + lr) * out_bytes + 4 * lg * es;
            if constexpr (sizeof(T) == 2) buf_store(bf16x4{(bf16)o[0], (bf16)o[1], (bf16)o[2], (bf16)o[3]}, r, off);
            else buf_store(o, r, off);
        }
    }
    gd_wait<0>();  // a workgroup's LDS is another's once its waves have ended
    if (!KEEP && a.fin) {
#pragma unroll
        for (int i = 0; i < OT; ++i) *(f32x4*)(a.fin + state_at + at(i)) = St[i];
    }
}

}  // namespace ssd
