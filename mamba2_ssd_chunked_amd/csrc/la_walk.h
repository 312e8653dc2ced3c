// The chunked walk of linear attention with a decay per head (bf16 and float32 MFMA).
//
//   M_t = l M_(t-1) + s c_t b_t^T,   out_t = f M_t a_t
//
// is computed chunk by chunk.  With i, j token places in a chunk of n <= Q tokens and M the
// state that enters it:
//   out_i = inter l^(i+1) M a_i + intra sum_{j<=i} l^(i-j) (b_j . a_i) c_j
//   M     <- l^n M + s sum_j l^(n-1-j) c_j b_j^T
// so the work is three matrix products per chunk, and M never leaves the registers: wave w
// of the workgroup keeps columns w CD/4 .. of M^T [BD][CD] in float32 accumulators.
//
// A sequence is walked by as many workgroups as it has spans of `span` tokens (LaPlan).
// Where a sequence has more than one, a first launch (OUT = false) leaves the state that
// each span adds, a second one composes them into the states that enter the spans, and the
// walk proper starts from those.
//
// Operand layouts (see Mma in ssd_internal.h).  Every product is formed transposed so that
// its result is the next product's operand or is stored with four neighbouring channels to
// a lane:
//   scores^T [j][i] = b a^T : operands are rows of a and b with 8 (float32: 4) of BD to a
//       lane; the result's lane holds four j of one i, two stacked tiles are a k operand
//   out^T [cd][i] = M^T^T a^T + c^T scores^T : M^T's accumulators are a k operand as they
//       are; c is read from LDS transposed (XT)
//   M^T [bd][cd] = b^T (w c) : b is read transposed too, c's fragments are the ones above,
//       weighted in registers
// A bf16 k operand takes its 32 channels as 4g .. 4g+3 and 16+4g .. of lane group g (two
// stacked tiles); rows of a and b stand in LDS with their channels in that order, so that
// an operand is one 16-byte read.
//
// Precision.  Scores and the entering state are rounded to bf16 once as operands.  The
// weighted c are not: a state is a float32 result, and one rounding would leave 2^-9 of it.
// They enter as a sum of two bf16 (2^-17 of a term), of three (2^-24) where the state is
// an output or is handed to other spans.
#pragma once

#include "mixer_internal.h"
#include "xt.h"

namespace ssd {

template <typename T> struct LaCfg;
template <> struct LaCfg<bf16> {
    static constexpr int Q = 64;    // tokens per chunk
    static constexpr int TPK = 2;   // 16-wide tiles per k operand
};
template <> struct LaCfg<float> {
    static constexpr int Q = 32;
    static constexpr int TPK = 1;
};

// The spans of all sequences, numbered so that no scan over the lengths is needed:
// sequence s owns the numbers lo_s / span + s .. (as many as it has spans, and at least
// one), of which the ones behind its last span are idle.
struct LaPlan {
    int span;       // tokens per span, a multiple of the chunk
    int64_t slots;  // numbers handed out
    bool split;     // some sequence may have more than one span
};

struct LaSpan {
    int s, j;         // sequence, span of it; s < 0: idle
    int64_t lo, hi;   // tokens of the sequence
    int i0, n;        // first visited place, tokens of the span
    bool last;
};

__device__ __forceinline__ LaSpan la_span(const LaWalk& w, const LaPlan& p, int64_t slot) {
    int a = 0, b = w.nseq - 1;  // the last sequence whose numbers start at or below slot
    while (a < b) {
        const int m = (a + b + 1) / 2;
        if (seq_range(w, m).lo / p.span + m <= slot) a = m;
        else b = m - 1;
    }
    const SeqRange r = seq_range(w, a);
    const int64_t j = slot - (r.lo / p.span + a), len = r.hi - r.lo;
    LaSpan s;
    s.s = j < 0 || (j > 0 && j * p.span >= len) ? -1 : a;
    s.j = (int)j;
    s.lo = r.lo;
    s.hi = r.hi;
    s.i0 = (int)(j * p.span);
    s.n = (int)(len - s.i0 < p.span ? len - s.i0 : p.span);
    s.last = (j + 1) * p.span >= len;
    return s;
}

// Rows of one operand on their way into LDS: 16-byte vectors of D channels per token.
template <typename T, int D>
struct LaRows {
    static constexpr int Q = LaCfg<T>::Q, VEC = 16 / (int)sizeof(T), VPR = D / VEC;
    static constexpr int RPP = 256 / VPR, NP = Q / RPP;  // rows per pass, passes
    static constexpr int PITCH = D + VEC;
    typedef T vt __attribute__((ext_vector_type(VEC)));
    vt v[NP];

    // rows of the n tokens from t0 (in memory order), visited backwards if `rev`; rows
    // behind them are zero
    __device__ __forceinline__ void load(const T* base, int64_t ts, int64_t t0, int n, bool rev) {
        const T* p = base + t0 * ts;
        const int r0 = threadIdx.x / VPR, c = (threadIdx.x % VPR) * VEC;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int r = r0 + i * RPP;
            const int row = r < n ? (rev ? n - 1 - r : r) : 0;
            v[i] = *(const vt*)at32(p, (uint32_t)row * (uint32_t)ts + c);
            if (r >= n) v[i] = vt{};
        }
    }
    __device__ __forceinline__ void store(T* lds) const {
        const int r0 = threadIdx.x / VPR, c = (threadIdx.x % VPR) * VEC;
#pragma unroll
        for (int i = 0; i < NP; ++i) *(vt*)(lds + (r0 + i * RPP) * PITCH + c) = v[i];
    }
    // the same with the channels in k operand order
    __device__ __forceinline__ void store_k(T* lds) const {
        if constexpr (sizeof(T) == 4) {
            store(lds);
        } else {
            const int r0 = threadIdx.x / VPR, q = threadIdx.x % VPR, m = q % 4;
            T* p = lds + r0 * PITCH + 32 * (q / 4) + 16 * (m & 1) + 4 * (m >> 1);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                *(bf16x4*)(p + i * RPP * PITCH) = __builtin_shufflevector(v[i], v[i], 0, 1, 2, 3);
                *(bf16x4*)(p + i * RPP * PITCH + 8) = __builtin_shufflevector(v[i], v[i], 4, 5, 6, 7);
            }
        }
    }
};

// b^T as the row operand of M^T: rows are channels 16 t .., k the tokens from jb, b's rows
// being stored with channels in k operand order.
template <typename T>
__device__ __forceinline__ typename Mma<T>::Frag la_bt(const T* b, int pitch, int jb, int t,
                                                       int lane) {
    if constexpr (sizeof(T) == 4) {
        return XT<float>::load(b, pitch, jb, 16 * t, lane);
    } else {
        const int q = lane % 16, g = lane / 16;
        const bf16* a = b + (jb + 4 * g + q / 4) * pitch + 32 * (t / 2) + 8 * (q % 4) + 4 * (t % 2);
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s4 lds_s4;
        const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)a));
        const bf16x4 hi =
            __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(a + 16 * pitch)));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
}

// A k operand from TPK stacked accumulator tiles.
template <typename T>
__device__ __forceinline__ typename Mma<T>::Frag la_frag(const f32x4* tiles) {
    if constexpr (sizeof(T) == 4) {
        return tiles[0];
    } else {
        typename Mma<T>::Frag f;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (bf16)tiles[e / 4][e % 4];
        return f;
    }
}

// l^e, the exponent's product taken in float64 so that only exp2's own ulp is left.
__device__ __forceinline__ float la_pow(double l2, int e) {
    return e == 0 ? 1.f : __builtin_amdgcn_exp2f((float)(l2 * (double)e));
}

template <typename T, int BD, int CD, bool OUT>
constexpr int la_lds_bytes() {
    constexpr int Q = LaCfg<T>::Q, V = 16 / (int)sizeof(T), NT = Q / 16;
    return Q * (BD + V) * (int)sizeof(T) * (OUT ? 2 : 1) + Q * (CD + V) * (int)sizeof(T) +
           (OUT ? NT * (NT / LaCfg<T>::TPK) * 1024 : 0);
}

// Workgroup of four waves per (span, head).  SPLITS: bf16 terms per weighted c (1 for
// float32).  `ws`: the spans' states, [slot][H][wave][tile][lane] f32x4.
template <typename T, int BD, int CD, bool OUT, int SPLITS>
__global__ void __launch_bounds__(256, 2) k_la_walk(LaWalk w, LaPlan plan, f32x4* __restrict__ ws) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    constexpr int Q = LaCfg<T>::Q, TPK = LaCfg<T>::TPK, NT = Q / 16, NK = NT / TPK;
    constexpr int SL = M::SL, KS = M::KS, KB = BD / KS;
    constexpr int BT = BD / 16, CW = CD / 4, CT = CW / 16;  // tiles of M^T of one wave
    constexpr int AP = LaRows<T, BD>::PITCH, CP = LaRows<T, CD>::PITCH;
    __shared__ __align__(16) unsigned char lds[la_lds_bytes<T, BD, CD, OUT>()];
    T* sb = (T*)lds;
    T* sc = sb + Q * AP;
    T* sa = sc + Q * CP;
    Frag* sp = (Frag*)(sa + Q * AP);  // scores, [row tile][k block][lane]

    const int64_t nblk = gridDim.x;
    const int64_t item = nblk % 8 == 0 ? (blockIdx.x % 8) * (nblk / 8) + blockIdx.x / 8 : blockIdx.x;
    const int h = (int)(item % w.H);
    const int64_t slot = item / w.H;
    const LaSpan sp_ = la_span(w, plan, slot);
    if (sp_.s < 0 || (!OUT && sp_.last)) return;
    const int wave = wave_id(), lane = threadIdx.x % 64, lr = lane % 16, lg = lane / 16;
    const T* pa = (const T*)w.a + (int64_t)(h / w.a_div) * BD;
    const T* pb = (const T*)w.b + (int64_t)(h / w.b_div) * BD;
    const T* pc = (const T*)w.c + (int64_t)(h / w.c_div) * CD;
    const int64_t state_at = ((int64_t)sp_.s * w.H + h) * (BD * CD);
    f32x4* mine = ws + (((slot * w.H + h) * 4 + wave) * (BT * CT)) * 64 + lane;

    const int nch = (sp_.n + Q - 1) / Q;
    // tokens of chunk k in memory order: [t0, t0 + n)
    auto first_token = [&](int k, int n) {
        const int64_t i = sp_.i0 + (int64_t)k * Q;
        return w.reverse ? sp_.hi - i - n : sp_.lo + i;
    };
    auto tokens_of = [&](int k) { return sp_.n - k * Q < Q ? sp_.n - k * Q : Q; };
    LaRows<T, BD> ra, rb;
    LaRows<T, CD> rc;
    auto load = [&](int k) {
        const int n = tokens_of(k);
        const int64_t t0 = first_token(k, n);
        if constexpr (OUT) ra.load(pa, w.a_ts, t0, n, w.reverse);
        rb.load(pb, w.b_ts, t0, n, w.reverse);
        rc.load(pc, w.c_ts, t0, n, w.reverse);
    };
    if (nch > 0) load(0);

    // the state that enters the span
    f32x4 St[BT][CT];
    const bool given = sp_.j == 0;
#pragma unroll
    for (int t = 0; t < BT; ++t)
#pragma unroll
        for (int u = 0; u < CT; ++u) {
            const int bd = 16 * t + 4 * lg, cd = wave * CW + 16 * u + lr;
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            if (given) {
                if (w.init) {
                    const float* p = w.init + state_at;
                    if (w.trans) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = p[(bd + r) * CD + cd];
                    } else {
                        v = *(const f32x4*)(p + cd * BD + bd);
                    }
                }
            } else if constexpr (OUT) {
                v = mine[(t * CT + u) * 64];
            }
            St[t][u] = v;
        }

    const float ld = w.log_decay[h];
    const double l2 = (double)ld * 1.4426950408889634;
    // l^(i - j) of a lane's four j in the diagonal score tile, and l^(16 + i - j) for the
    // tiles below it, whose further factor l^(16 (d - 1)) the whole wave shares
    float dg[4], lw[4], far[NT > 2 ? NT - 2 : 1];
    if constexpr (OUT) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = lr - (4 * lg + r);
            dg[r] = w.intra * la_pow(l2, d > 0 ? d : 0);
            lw[r] = w.intra * la_pow(l2, 16 + d);
        }
#pragma unroll
        for (int d = 0; d < (NT > 2 ? NT - 2 : 1); ++d) far[d] = la_pow(l2, 16 * (d + 1));
    }
    const float lq = (float)exp((double)Q * (double)ld);  // compounded per chunk: exact to 2^-25
    float wk[NK][SL];  // s l^(n-1-j) of the lane's k slots
    auto weights = [&](int n) {
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int s = 0; s < SL; ++s) {
                const int j = KS * k + 16 * (s / 4) + 4 * lg + s % 4;
                wk[k][s] = j < n ? w.state_scale * la_pow(l2, n - 1 - j) : 0.f;
            }
    };
    weights(Q);
    float row[NT];  // inter l^(i+1)
#pragma unroll
    for (int t = 0; t < NT; ++t) row[t] = w.inter * la_pow(l2, 16 * t + lr + 1);

    for (int k = 0; k < nch; ++k) {
        const int n = tokens_of(k);
        const bool late = w.reverse && given && k == 0;  // the given state is not decayed yet
        __syncthreads();  // the last chunk's reads are done
        if constexpr (OUT) ra.store_k(sa);
        rb.store_k(sb);
        rc.store(sc);
        __syncthreads();
        if (k + 1 < nch) load(k + 1);
        if (n != Q) weights(n);

        f32x4 o[NT][CT];
        if constexpr (OUT) {
            // scores of row tile `wave`: k blocks up to the diagonal
            if (wave < NT) {
                Frag af[KB];
#pragma unroll
                for (int q = 0; q < KB; ++q)
                    af[q] = M::load(sa + (16 * wave + lr) * AP + KS * q + SL * lg);
#pragma unroll
                for (int kb = 0; kb < NK; ++kb) {
                    f32x4 tl[TPK];
#pragma unroll
                    for (int e = 0; e < TPK; ++e) {
                        const int jt = kb * TPK + e;
                        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
                        if (jt <= wave) {
#pragma unroll
                            for (int q = 0; q < KB; ++q)
                                acc = M::mma(M::load(sb + (16 * jt + lr) * AP + KS * q + SL * lg),
                                             af[q], acc);
                            if (jt == wave) {
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    acc[r] = 4 * lg + r <= lr ? acc[r] * dg[r] : 0.f;
                            } else {
                                const int d = wave - jt;
                                const float f = d == 1 ? 1.f : far[d - 2 < NT - 2 ? d - 2 : 0];
#pragma unroll
                                for (int r = 0; r < 4; ++r) acc[r] *= lw[r] * f;
                            }
                        }
                        tl[e] = acc;
                    }
                    sp[(wave * NK + kb) * 64 + lane] = la_frag<T>(tl);
                }
            }
            // M a_i
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < CT; ++u) o[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                Frag sf[CT];
#pragma unroll
                for (int u = 0; u < CT; ++u) {
                    f32x4 tl[TPK];
#pragma unroll
                    for (int e = 0; e < TPK; ++e) tl[e] = St[q * TPK + e][u];
                    sf[u] = la_frag<T>(tl);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const Frag a = M::load(sa + (16 * t + lr) * AP + KS * q + SL * lg);
#pragma unroll
                    for (int u = 0; u < CT; ++u) o[t][u] = M::mma(sf[u], a, o[t][u]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float f = late ? w.inter * la_pow(l2, 16 * t + lr) : row[t];
#pragma unroll
                for (int u = 0; u < CT; ++u) o[t][u] *= f;
            }
            __syncthreads();  // the scores are there
        }

        Frag cf[NK][CT];
#pragma unroll
        for (int kb = 0; kb < NK; ++kb)
#pragma unroll
            for (int u = 0; u < CT; ++u)
                cf[kb][u] = XT<T>::load(sc, CP, KS * kb, wave * CW + 16 * u, lane);
        if constexpr (OUT) {
            bool wild = false;  // a sum is not finite
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int kb = 0; kb <= t / TPK; ++kb) {
                    const Frag p = sp[(t * NK + kb) * 64 + lane];
#pragma unroll
                    for (int u = 0; u < CT; ++u) o[t][u] = M::mma(cf[kb][u], p, o[t][u]);
                }
#pragma unroll
                for (int u = 0; u < CT; ++u) {
                    const f32x4 v = o[t][u];
                    wild = wild || !(fabsf((v[0] + v[1]) + (v[2] + v[3])) < INFINITY);
                }
            }
            if (__ballot(wild)) {
                // A c_j that is not finite times a masked score's 0 is NaN in the outputs
                // before j too.  Row by row, with the later c taken out, it is not.
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    f32x4 base[CT];
#pragma unroll
                    for (int u = 0; u < CT; ++u) base[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < KB; ++q)
#pragma unroll
                        for (int u = 0; u < CT; ++u) {
                            f32x4 tl[TPK];
#pragma unroll
                            for (int e = 0; e < TPK; ++e) tl[e] = St[q * TPK + e][u];
                            base[u] = M::mma(la_frag<T>(tl),
                                             M::load(sa + (16 * t + lr) * AP + KS * q + SL * lg),
                                             base[u]);
                        }
                    const float f = late ? w.inter * la_pow(l2, 16 * t + lr) : row[t];
                    for (int i = 0; i < 16; ++i)
#pragma unroll
                        for (int u = 0; u < CT; ++u) {
                            f32x4 v = base[u] * f;
#pragma unroll
                            for (int kb = 0; kb <= t / TPK; ++kb) {
                                Frag c = cf[kb][u];
#pragma unroll
                                for (int s = 0; s < SL; ++s)
                                    if (KS * kb + 16 * (s / 4) + 4 * lg + s % 4 > 16 * t + i)
                                        c[s] = (T)0.f;
                                v = M::mma(c, sp[(t * NK + kb) * 64 + lane], v);
                            }
                            if (lr == i) o[t][u] = v;
                        }
                }
            }
        }

        // M <- l^n M + b^T (w c)
        const float keep = late ? (float)exp((double)(n - 1) * (n > 1 ? (double)ld : 0.0))
                                : (n == Q ? lq : (float)exp((double)n * (double)ld));
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) St[t][u] *= keep;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            Frag wc[SPLITS][CT];
#pragma unroll
            for (int u = 0; u < CT; ++u)
#pragma unroll
                for (int s = 0; s < SL; ++s) {
                    float x = (float)cf[kb][u][s] * wk[kb][s];
#pragma unroll
                    for (int p = 0; p < SPLITS; ++p) {
                        wc[p][u][s] = (T)x;
                        x -= (float)wc[p][u][s];
                    }
                }
#pragma unroll
            for (int t = 0; t < BT; ++t) {
                const Frag bt = la_bt<T>(sb, AP, KS * kb, t, lane);
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int p = SPLITS - 1; p >= 0; --p)
                        St[t][u] = M::mma(bt, wc[p][u], St[t][u]);
            }
        }

        if constexpr (OUT) {
            // a lane holds channels 4 lg .. of token lr of every tile
            const int64_t t0 = first_token(k, n);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int i = 16 * t + lr;
                if (i < n) {
                    const int64_t tok = t0 + (w.reverse ? n - 1 - i : i);
                    const int64_t at = tok * w.out_ts + (int64_t)h * CD + wave * CW + 4 * lg;
#pragma unroll
                    for (int u = 0; u < CT; ++u) {
                        if (w.out_f32) {
                            *(f32x4*)((float*)w.out + at + 16 * u) = o[t][u];
                        } else {
                            typename Vec4<T>::type v;
#pragma unroll
                            for (int r = 0; r < 4; ++r) v[r] = (T)o[t][u][r];
                            *(typename Vec4<T>::type*)((T*)w.out + at + 16 * u) = v;
                        }
                    }
                }
            }
        }
    }

    if constexpr (!OUT) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) mine[(t * CT + u) * 64] = St[t][u];
    } else if (w.fin && sp_.last) {
        const float keep = w.reverse && sp_.n > 0 ? (float)exp((double)ld) : 1.f;
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) {
                const int bd = 16 * t + 4 * lg, cd = wave * CW + 16 * u + lr;
                float* p = w.fin + state_at;
                const f32x4 v = St[t][u] * keep;
                if (w.trans) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[(bd + r) * CD + cd] = v[r];
                } else {
                    *(f32x4*)(p + cd * BD + bd) = v;
                }
            }
    }
}

}  // namespace ssd
