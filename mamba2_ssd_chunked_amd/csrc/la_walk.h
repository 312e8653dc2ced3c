// The chunked walk of linear attention with a decay per head (bf16 and float32 MFMA).
//
//   M_t = l M_(t-1) + s c_t b_t^T,   out_t = f M_t a_t
//
// is computed chunk by chunk.  With i, j token places in a chunk of n <= Q tokens and M the
// state that enters it:
//   out_i = inter l^(i+1) M a_i + intra sum_{j<=i} l^(i-j) (b_j . a_i) c_j
//   M     <- l^n M + s sum_j l^(n-1-j) c_j b_j^T
// so the work is three matrix products per chunk, and M never leaves the registers: a
// workgroup has 64 columns of M^T [BD][CD], each of its four waves 16 of them in float32
// accumulators.  (Where CD is 128, two neighbouring workgroups form the same scores and read
// the same a and b, the second time from L2.)
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
// They come through bounded buffer loads, which give zeros for rows without a token and
// need no branch or select: the n tokens of a last chunk take its last rows, so that the
// weights l^(Q-1-j) of its rows are every chunk's.
template <typename T, int D, bool REV>
struct LaRows {
    static constexpr int Q = LaCfg<T>::Q, VEC = 16 / (int)sizeof(T), VPR = D / VEC;
    static constexpr int RPP = 256 / VPR, NP = Q / RPP;  // rows per pass, passes
    static constexpr int PITCH = D + VEC;
    typedef T vt __attribute__((ext_vector_type(VEC)));
    vt v[NP];

    // rows of the n tokens from t0 (in memory order), `ts` elements apart, visited backwards
    // if REV; a row without a token is beyond the bound (forwards by its negative offset)
    __device__ __forceinline__ void load(const T* base, int ts, int64_t t0, int n) {
        const int bytes = ts * (int)sizeof(T);
        const __amdgpu_buffer_rsrc_t r = buf_rsrc(base + t0 * ts, n * bytes);
        const int r0 = threadIdx.x / VPR, c = (threadIdx.x % VPR) * 16;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int row = r0 + i * RPP;
            v[i] = buf_load<vt>(r, (REV ? Q - 1 - row : row - (Q - n)) * bytes + c);
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

enum LaOut { LA_STATE = 0, LA_ACT = 1, LA_F32 = 2 };  // what a walk leaves behind

template <typename T, int BD, int OUT>
constexpr int la_lds_bytes() {
    constexpr int Q = LaCfg<T>::Q, V = 16 / (int)sizeof(T), NT = Q / 16;
    return Q * (BD + V) * (int)sizeof(T) * (OUT ? 2 : 1) + Q * (64 + V) * (int)sizeof(T) +
           (OUT ? NT * (NT / LaCfg<T>::TPK) * 1024 : 0);
}

// Workgroup of four waves per (span, head, 64 columns).  SPLITS: bf16 terms per weighted c
// (1 for float32).  `ws`: the spans' states, [slot][H][CD / 64][wave][tile][lane] f32x4.
template <typename T, int BD, bool REV, int OUT, int SPLITS>
__global__ void __launch_bounds__(256, BD == 64 ? 3 : 2) k_la_walk(LaWalk w, LaPlan plan, f32x4* __restrict__ ws) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    constexpr int Q = LaCfg<T>::Q, TPK = LaCfg<T>::TPK, NT = Q / 16, NK = NT / TPK;
    constexpr int SL = M::SL, KS = M::KS, KB = BD / KS;
    constexpr int BT = BD / 16;  // tiles of M^T of one wave
    constexpr int AP = LaRows<T, BD, REV>::PITCH, CP = LaRows<T, 64, REV>::PITCH;
    __shared__ __align__(16) unsigned char lds[la_lds_bytes<T, BD, OUT>()];
    T* sb = (T*)lds;
    T* sc = sb + Q * AP;
    T* sa = sc + Q * CP;
    Frag* sp = (Frag*)(sa + Q * AP);  // scores, [row tile][k block][lane]

    // consecutive items (the column halves and heads that share rows) go to one XCD
    const int64_t nblk = gridDim.x;
    int64_t item = nblk % 8 == 0 ? (blockIdx.x % 8) * (nblk / 8) + blockIdx.x / 8 : blockIdx.x;
    const int CD = w.cd, nct = CD / 64;
    const int ct = (int)(item % nct);
    item /= nct;
    const int h = (int)(item % w.H);
    const int64_t slot = item / w.H;
    const LaSpan sp_ = la_span(w, plan, slot);
    if (sp_.s < 0 || (!OUT && sp_.last)) return;
    const int wave = wave_id(), lane = threadIdx.x % 64, lr = lane % 16, lg = lane / 16;
    const T* pa = (const T*)w.a + (int64_t)(h / w.a_div) * BD;
    const T* pb = (const T*)w.b + (int64_t)(h / w.b_div) * BD;
    const T* pc = (const T*)w.c + (int64_t)(h / w.c_div) * CD + ct * 64;
    const int ats = (int)w.a_ts, bts = (int)w.b_ts, cts = (int)w.c_ts;
    const int nch = (sp_.n + Q - 1) / Q;

    // tokens of chunk k in memory order: [t0, t0 + n)
    auto first_token = [&](int k, int n) {
        const int64_t i = sp_.i0 + (int64_t)k * Q;
        return REV ? sp_.hi - i - n : sp_.lo + i;
    };
    auto tokens_of = [&](int k) { return sp_.n - k * Q < Q ? sp_.n - k * Q : Q; };
    LaRows<T, BD, REV> ra, rb;
    LaRows<T, 64, REV> rc;
    auto load = [&](int k) {
        const int n = tokens_of(k);
        const int64_t t0 = first_token(k, n);
        rb.load(pb, bts, t0, n);
        rc.load(pc, cts, t0, n);
        if constexpr (OUT) ra.load(pa, ats, t0, n);
    };
    if (nch > 0) load(0);

    // the state that enters the span; this lane's elements of tile t are channels
    // 16 t + 4 lg .. of b and channel `col` of c
    f32x4 St[BT];
    const int col = ct * 64 + wave * 16 + lr;
    const bool given = sp_.j == 0;
    f32x4* mine = ws + (((slot * w.H + h) * nct + ct) * 4 + wave) * (BT * 64) + lane;
    const int64_t state_at = ((int64_t)sp_.s * w.H + h) * ((int64_t)BD * CD) +
                             (w.trans ? (int64_t)4 * lg * CD + col : (int64_t)col * BD + 4 * lg);
    if (OUT && !given) {
#pragma unroll
        for (int t = 0; t < BT; ++t) St[t] = mine[t * 64];
    } else if (given && w.init && !w.trans) {
#pragma unroll
        for (int t = 0; t < BT; ++t) St[t] = *(const f32x4*)(w.init + state_at + 16 * t);
    } else if (given && w.init) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) St[t][r] = w.init[state_at + (int64_t)(16 * t + r) * CD];
    } else {
#pragma unroll
        for (int t = 0; t < BT; ++t) St[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const float ld = w.log_decay[h];
    const double l2 = (double)ld * 1.4426950408889634;
    // l^(i - j) of a lane's four j in the diagonal score tile, and l^(16 + i - j) for the
    // tiles below it, whose further factor l^(16 (d - 1)) the whole wave shares
    float dg[4], lw[4];
    const float l16 = la_pow(l2, 16), l32 = la_pow(l2, 32);
    if constexpr (OUT) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = lr - (4 * lg + r);
            dg[r] = w.intra * la_pow(l2, d > 0 ? d : 0);
            lw[r] = w.intra * la_pow(l2, 16 + d);
        }
    }
    float wk[NK][SL];  // s l^(Q-1-j) of the lane's k slots
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int s = 0; s < SL; ++s)
            wk[k][s] = w.state_scale *
                       la_pow(l2, Q - 1 - (KS * k + 16 * (s / 4) + 4 * lg + s % 4));
    // The given state of a REV walk is not decayed before its first use.
    const bool late = REV && given;
    // l^n, compounded from chunk to chunk: the exact power, rounded once
    auto power = [&](int e) { return e == 0 ? 1.f : (float)exp((double)e * (double)ld); };
    const int nlast = sp_.n - (nch - 1) * Q;
    const float lq = power(Q), lfirst = late ? power(Q - 1) : lq,
                llast = power(late && nch == 1 ? nlast - 1 : nlast);
    float row[NT];  // inter l^(i+1)
#pragma unroll
    for (int t = 0; t < NT; ++t) row[t] = w.inter * la_pow(l2, 16 * t + lr + (late ? 0 : 1));
    const float l1 = la_pow(l2, 1);
    const int out_bytes = (int)w.out_ts * (OUT == LA_F32 ? 4 : (int)sizeof(T));

    for (int k = 0; k < nch; ++k) {
        const int n = tokens_of(k);
        __syncthreads();  // the last chunk's reads are done
        rb.store_k(sb);
        rc.store(sc);
        if constexpr (OUT) ra.store_k(sa);
        __syncthreads();
        // the last chunk's prefetch repeats it: no branch, so no full waits at a join
        load(k + 1 < nch ? k + 1 : k);
        const float keep = k + 1 == nch ? llast : (k == 0 ? lfirst : lq);
        if (OUT && n != Q) {  // the last chunk's tokens begin at row Q - n
            int i0 = lr - (Q - n) + (late && k == 0 ? 0 : 1);
            asm volatile("" : "+v"(i0));  // computed here, not held from before the loop
#pragma unroll
            for (int t = 0; t < NT; ++t)
                row[t] = w.inter * la_pow(l2, 16 * t + i0 > 0 ? 16 * t + i0 : 0);
        }

        f32x4 o[NT];
        if constexpr (OUT) {
            // scores of row tile `wave`: k blocks up to the diagonal
            if (wave < NT) {
                Frag af[KB];
#pragma unroll
                for (int q = 0; q < KB; ++q)
                    af[q] = M::load(sa + (16 * wave + lr) * AP + KS * q + SL * lg);
#pragma unroll
                for (int kb = 0; kb < NK; ++kb) {
                    if (kb * TPK > wave) break;
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
                                const float f = wave - jt == 1 ? 1.f : (wave - jt == 2 ? l16 : l32);
#pragma unroll
                                for (int r = 0; r < 4; ++r) acc[r] *= lw[r] * f;
                            }
                        }
                        tl[e] = acc;
                    }
                    sp[(wave * NK + kb) * 64 + lane] = la_frag<T>(tl);
                }
            }
            // l^(i+1) M a_i
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                const Frag sf = la_frag<T>(&St[q * TPK]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    o[t] = M::mma(sf, M::load(sa + (16 * t + lr) * AP + KS * q + SL * lg), o[t]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] *= row[t];
            __syncthreads();  // the scores are there
        }

        Frag cf[NK];
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) cf[kb] = XT<T>::load(sc, CP, KS * kb, wave * 16, lane);
        // w_j c_j, and whether one of this wave's c is not finite
        float x[NK][SL], all = 0.f;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb)
#pragma unroll
            for (int s = 0; s < SL; ++s) {
                x[kb][s] = (float)cf[kb][s] * wk[kb][s];
                all += x[kb][s];
            }
        if constexpr (OUT) {
            // A c_j that is not finite times a masked score's 0 would be NaN in the outputs
            // before j too.  It is taken out of the product, and the outputs of its channel
            // from j on are set.
            const bool wild = __ballot(!(fabsf(all) < INFINITY)) != 0;
            int from[4];
            if (wild) {
                int j0 = Q;
                int g4 = 4 * lg;
                asm volatile("" : "+v"(g4));
#pragma unroll
                for (int kb = NK - 1; kb >= 0; --kb)
#pragma unroll
                    for (int s = SL - 1; s >= 0; --s)
                        if (!(fabsf((float)cf[kb][s]) < INFINITY)) {
                            j0 = KS * kb + 16 * (s / 4) + s % 4 + g4;
                            cf[kb][s] = (T)0.f;
                        }
                j0 = min(j0, __shfl_xor(j0, 16, 64));
                j0 = min(j0, __shfl_xor(j0, 32, 64));
#pragma unroll
                for (int r = 0; r < 4; ++r) from[r] = __shfl(j0, 4 * lg + r, 64);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int kb = 0; kb <= t / TPK; ++kb)
                    o[t] = M::mma(cf[kb], sp[(t * NK + kb) * 64 + lane], o[t]);
            if (wild) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * t + lr >= from[r]) o[t][r] = NAN;
            }
        }

        // M <- l^n M + b^T (w c)
#pragma unroll
        for (int t = 0; t < BT; ++t) St[t] *= keep;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            Frag wc[SPLITS];
#pragma unroll
            for (int s = 0; s < SL; ++s) {
#pragma unroll
                for (int p = 0; p < SPLITS; ++p) {
                    wc[p][s] = (T)x[kb][s];
                    x[kb][s] -= (float)wc[p][s];
                }
            }
#pragma unroll
            for (int t = 0; t < BT; ++t) {
                const Frag bt = la_bt<T>(sb, AP, KS * kb, t, lane);
#pragma unroll
                for (int p = SPLITS - 1; p >= 0; --p) St[t] = M::mma(bt, wc[p], St[t]);
            }
        }

        if constexpr (OUT) {
            // a lane holds channels 4 lg .. of row lr of every tile; rows without a token are
            // beyond the buffer's bound
            typedef typename std::conditional<OUT == LA_F32, float, T>::type OT;
            typedef typename Vec4<OT>::type ov;
            const __amdgpu_buffer_rsrc_t r =
                buf_rsrc((OT*)w.out + first_token(k, n) * w.out_ts + (int64_t)h * CD + ct * 64,
                         n * out_bytes);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int i = 16 * t + lr;
                ov v;
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = (OT)o[t][c];
                buf_store(v, r, (REV ? Q - 1 - i : i - (Q - n)) * out_bytes +
                                    (wave * 16 + 4 * lg) * (int)sizeof(OT));
            }
        }
        if (late && k == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) row[t] *= l1;
        }
    }

    if constexpr (!OUT) {
#pragma unroll
        for (int t = 0; t < BT; ++t) mine[t * 64] = St[t];
    } else if (w.fin && sp_.last) {
        const float keep = REV && sp_.n > 0 ? (float)exp((double)ld) : 1.f;
#pragma unroll
        for (int t = 0; t < BT; ++t) {
            const f32x4 v = St[t] * keep;
            if (w.trans) {
#pragma unroll
                for (int r = 0; r < 4; ++r) w.fin[state_at + (int64_t)(16 * t + r) * CD] = v[r];
            } else {
                *(f32x4*)(w.fin + state_at + 16 * t) = v;
            }
        }
    }
}

}  // namespace ssd
