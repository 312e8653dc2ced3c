// The chunked walk of linear attention with a decay per head (bf16 and float32 MFMA).
//
//   M_t = l M_(t-1) + s c_t b_t^T,   out_t = f M_t a_t
//
// is computed chunk by chunk.  With i, j token places in a chunk of n <= Q tokens and M the
// state that enters it:
//   out_i = inter l^(i+1) M a_i + intra sum_{j<=i} l^(i-j) (b_j . a_i) c_j
//   M     <- l^n M + s sum_j l^(n-1-j) c_j b_j^T
// so the work is three matrix products per chunk, and M never leaves the registers: each of
// the four waves of a workgroup keeps CD/4 columns of M^T [BD][CD] in float32 accumulators.
//
// A sequence is walked by as many workgroups as it has spans of `span` tokens (LaPlan).
// Where a sequence has more than one, a first launch (OUT = false) leaves the state that
// each span adds, a second one composes them into the states that enter the spans, and the
// walk proper starts from those.
//
// What bounds it.  With a state of 128 x 64 the walk runs at 3.8 to 4.6 TB/s (2 x 8192 tokens,
// 32 heads: 87 to 105 us), with one of 128 x 128 it issues instructions for most of its time:
// 32768 tokens of 32 heads take 276 to 325 us, with MFMA 33 %, VALU 34 % and LDS 31 % busy at two
// workgroups per CU.  The figures that follow compare variants while scores and states were one
// bf16 (walks of 80 and 250 us at the quickest, 285 on average; see Precision): without any memory
// traffic nine tenths of the 128 x 128 walk's time were left.  Chunks of 64
// tokens: 128 gained nothing in the pass that only forms states (110 us to 135 in the backward)
// and double the scores' share.  Four waves: eight read each tile of LDS twice as often (338 us
// instead of 285 for 128 x 128).
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
// A bf16 k operand holds 8 neighbouring channels of 32 to a lane, so the two accumulator
// tiles that form one hold them 4 and 4: row 4g + r of tile t of M^T is channel
// 32 (t / 2) + 8 g + 4 (t % 2) + r (la_channel).  That costs nothing, since the transposed
// reads of b address their channels in quads of any order.
//
// Precision.  No float32 value is rounded to bf16 as an operand, since each such rounding adds
// 2^-9 to the one that an output has of its own (scores and entering states rounded once: root
// mean square error 1.41 times that of the rounded exact result; quickest walks of 80 instead of
// 87 us for 128 x 64 and of 250 instead of 287 for 128 x 128).  Scores and entering states are
// sums of two bf16 (LaCfg::PARTS), weighted c of two (2^-17 of a term left out) where they only
// reach bf16 outputs, and of three (float32's own rounding) in a walk whose last state is asked
// for, in its spans' states too.
#pragma once

#include <cfloat>

#include "mixer_internal.h"
#include "xt.h"

namespace ssd {

template <typename T> struct LaCfg;
template <> struct LaCfg<bf16> {
    static constexpr int Q = 64;    // tokens per chunk
    static constexpr int TPK = 2;   // 16-wide tiles per k operand
    static constexpr int PARTS = 2; // terms of a score or an entering state as an operand
};
template <> struct LaCfg<float> {
    static constexpr int Q = 32;
    static constexpr int TPK = 1;
    static constexpr int PARTS = 1;
};

// The spans of all sequences, numbered so that no scan over the lengths is needed: row s
// owns the numbers s per_row ..; packed sequence s owns lo_s / span + s .. (as many as it has
// spans, and at least one), of which the ones behind its last span are idle.
struct LaPlan {
    int span;       // tokens per span, a multiple of the chunk
    int per_row;    // spans of a row (no cu_seqlens)
    int64_t slots;  // numbers handed out
    bool split;     // some sequence may have more than one span
};
__device__ __forceinline__ int64_t la_first_slot(const LaWalk& w, const LaPlan& p, int s) {
    return w.cu ? seq_range(w, s).lo / p.span + s : (int64_t)s * p.per_row;
}
// Where the state that enters span j >= 1 of sequence s (first token lo) is kept; span j - 1
// leaves there what it adds.  Packed sequences share the places of whole spans' tokens: a
// sequence of n spans from token lo takes n - 1 of them from lo / span on, and the next one
// begins at least (n - 1) span + 1 tokens later, so that no number of sequences needs more
// than tokens / span.
__device__ __forceinline__ int64_t la_place(const LaWalk& w, const LaPlan& p, int s, int64_t lo,
                                            int64_t j) {
    return (w.cu ? lo / p.span : (int64_t)s * (p.per_row - 1)) + j - 1;
}
inline int64_t la_places(const LaWalk& w, const LaPlan& p) {
    return w.cu ? w.tokens / p.span : (int64_t)w.nseq * (p.per_row - 1);
}

struct LaSpan {
    int s, j;         // sequence, span of it; s < 0: idle
    int64_t lo, hi;   // tokens of the sequence
    int i0, n;        // first visited place, tokens of the span
    bool last;
};

__device__ __forceinline__ LaSpan la_span(const LaWalk& w, const LaPlan& p, int64_t slot) {
    int a = 0, b = w.nseq - 1;  // the last sequence whose numbers start at or below slot
    if (!w.cu) a = b = (int)(slot / p.per_row);
    while (a < b) {
        const int m = (a + b + 1) / 2;
        if (la_first_slot(w, p, m) <= slot) a = m;
        else b = m - 1;
    }
    const SeqRange r = seq_range(w, a);
    const int64_t j = slot - la_first_slot(w, p, a), len = r.hi - r.lo;
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

// Whether one of a vector's values is not finite.
__device__ __forceinline__ unsigned la_ones(unsigned u) {
    // a half's exponent of ones carries into its top bit
    return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
typedef unsigned la_u4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bool la_wild(bf16x8 v) {
    const la_u4 u = __builtin_bit_cast(la_u4, v);
    return (la_ones(u[0]) | la_ones(u[1]) | la_ones(u[2]) | la_ones(u[3])) != 0;
}
__device__ __forceinline__ bool la_wild(f32x4 v) {
    bool m = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = m || !(fabsf(v[i]) < INFINITY);
    return m;
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
    // whether a value is not finite
    __device__ __forceinline__ bool wild() const {
        bool m = false;
#pragma unroll
        for (int i = 0; i < NP; ++i) m = m || la_wild(v[i]);
        return m;
    }
};

// Channel of row 4 lg of tile t of M^T.
template <typename T>
__device__ __forceinline__ int la_channel(int t, int lg) {
    return sizeof(T) == 4 ? 16 * t + 4 * lg : 32 * (t / 2) + 8 * lg + 4 * (t % 2);
}

// b^T as the row operand of tile t of M^T, k the tokens from jb.
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

// A k operand from TPK stacked accumulator tiles, as a sum of PARTS terms: of bf16 the value cut
// off after 8 bits and the rest of it, rounded (2^-16 of the value is left out; rounding the
// first one as well would leave 2^-17 and makes the walks 2 % slower).
template <typename T>
__device__ __forceinline__ void la_frag(const f32x4* tiles,
                                        typename Mma<T>::Frag (&f)[LaCfg<T>::PARTS]) {
    if constexpr (sizeof(T) == 4) {
        f[0] = tiles[0];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = tiles[e / 4][e % 4];
            const unsigned hi = __float_as_uint(x) & 0xffff0000u;
            f[0][e] = __builtin_bit_cast(bf16, (unsigned short)(hi >> 16));
            f[1][e] = (bf16)(x - __uint_as_float(hi));
        }
    }
}

// Decays above 1: a chunk weighs its places without a token as well, whose zeros times an
// infinite power would be NaN.  Powers and weights are held to float32's largest value instead.
__device__ __forceinline__ float la_held(float w) {  // 0 or above, or NaN, which it leaves
    return w > FLT_MAX ? FLT_MAX : w;
}
__device__ __forceinline__ float la_within(float w) {
    return __builtin_amdgcn_fmed3f(w, -FLT_MAX, FLT_MAX);
}
// l^e, the exponent's product taken in float64 so that only exp2's own ulp is left.
__device__ __forceinline__ float la_pow(double l2, int e) {
    return e == 0 ? 1.f : la_held(__builtin_amdgcn_exp2f((float)(l2 * (double)e)));
}

enum LaOut { LA_STATE = 0, LA_ACT = 1, LA_F32 = 2 };  // what a walk leaves behind

template <typename T, int BD, int CD, int OUT>
constexpr int la_lds_bytes() {
    constexpr int Q = LaCfg<T>::Q, V = 16 / (int)sizeof(T), NT = Q / 16;
    return Q * (BD + V) * (int)sizeof(T) * (OUT ? 2 : 1) + Q * (CD + V) * (int)sizeof(T) +
           (OUT ? NT * (NT / LaCfg<T>::TPK) * LaCfg<T>::PARTS * 1024 + 16 + CD * 4 : 0);
}

// Two accumulator tiles, rounded, as one 16-byte run: a lane has channels 4 lg .. of both, and
// after exchanging with the lane group beside it channels 8 (lg / 2) .. of the one (even
// groups) or the other.
__device__ __forceinline__ bf16x8 la_pair(f32x4 a, f32x4 b) {
    typedef unsigned u2 __attribute__((ext_vector_type(2)));
    typedef unsigned u4 __attribute__((ext_vector_type(4)));
    const u2 x = __builtin_bit_cast(u2, bf16x4{(bf16)a[0], (bf16)a[1], (bf16)a[2], (bf16)a[3]});
    const u2 y = __builtin_bit_cast(u2, bf16x4{(bf16)b[0], (bf16)b[1], (bf16)b[2], (bf16)b[3]});
    const auto p = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
    const auto q = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
    return __builtin_bit_cast(bf16x8, u4{p[0], q[0], p[1], q[1]});
}

// One span of one head, by a workgroup of four waves.  SPLITS: bf16 terms per weighted c (1
// for float32).  `ws`: the states that enter spans, [place][H][wave][tile][lane] f32x4.
//
// A c_j that is not finite times a masked score's 0 would be NaN in the outputs before j.  A
// chunk that has one puts 0 in its place, and NaN into the state and, from j on, the
// outputs of its channel.  Both happen where few registers are live.
template <typename T, int BD, int CD, bool REV, int OUT, int SPLITS>
__device__ __forceinline__ void la_walk(const LaWalk& w, const LaPlan& plan,
                                        f32x4* __restrict__ ws, unsigned char* lds, int64_t slot,
                                        int h) {
    typedef Mma<T> M;
    typedef typename M::Frag Frag;
    constexpr int Q = LaCfg<T>::Q, TPK = LaCfg<T>::TPK, NT = Q / 16, NK = NT / TPK;
    constexpr int PARTS = LaCfg<T>::PARTS;
    constexpr int SL = M::SL, KS = M::KS, KB = BD / KS;
    constexpr int BT = BD / 16, CW = CD / 4, CT = CW / 16;  // tiles of M^T of one wave
    constexpr int AP = LaRows<T, BD, REV>::PITCH, CP = LaRows<T, CD, REV>::PITCH;
    T* sb = (T*)lds;
    T* sc = sb + Q * AP;
    T* sa = sc + Q * CP;
    Frag* sp = (Frag*)(sa + Q * AP);  // scores, [row tile][k block][part][lane]
    int* wild = (int*)(sp + NT * NK * PARTS * 64);  // a c of the chunk is not finite
    int* wild_row = wild + 4;               // the first such row of each channel, or Q
    if (OUT && threadIdx.x == 0) *wild = 0;

    const LaSpan sp_ = la_span(w, plan, slot);
    if (sp_.s < 0 || (!OUT && sp_.last)) return;
    const int wave = wave_id(), lane = threadIdx.x % 64, lr = lane % 16, lg = lane / 16;
    const T* pa = (const T*)w.a + (int64_t)(h / w.a_div) * BD;
    const T* pb = (const T*)w.b + (int64_t)(h / w.b_div) * BD;
    const T* pc = (const T*)w.c + (int64_t)(h / w.c_div) * CD;
    const int ats = (int)w.a_ts, bts = (int)w.b_ts, cts = (int)w.c_ts;
    const int nch = (sp_.n + Q - 1) / Q;

    // tokens of chunk k in memory order: [t0, t0 + n)
    auto first_token = [&](int k, int n) {
        const int64_t i = sp_.i0 + (int64_t)k * Q;
        return REV ? sp_.hi - i - n : sp_.lo + i;
    };
    auto tokens_of = [&](int k) { return sp_.n - k * Q < Q ? sp_.n - k * Q : Q; };
    LaRows<T, BD, REV> ra, rb;
    LaRows<T, CD, REV> rc;
    auto load = [&](auto& rows, const T* p, int ts, int k) {
        const int n = tokens_of(k);
        rows.load(p, ts, first_token(k, n), n);
        __builtin_amdgcn_sched_barrier(15);  // memory accesses stay on their side
    };
    if (nch > 0) {
        load(rb, pb, bts, 0);
        load(rc, pc, cts, 0);
        if constexpr (OUT) load(ra, pa, ats, 0);
    }

    // the state that enters the span; this lane's elements of tile (t, u) are the four
    // channels of b from la_channel and channel 16 u + `col` of c
    f32x4 St[BT][CT];
    const int col = wave * CW + lr;
    const bool given = sp_.j == 0;
    // read by a span that has one before it, written (OUT = LA_STATE) for the span behind
    f32x4* mine = ws + ((la_place(w, plan, sp_.s, sp_.lo, sp_.j + (OUT ? 0 : 1)) * w.H + h) * 4 +
                        wave) * (BT * CT * 64) + lane;
    const int64_t state_at = ((int64_t)sp_.s * w.H + h) * (BD * CD);
    auto at = [&](int t, int u) { return (col + 16 * u) * BD + la_channel<T>(t, lg); };
    auto at_trans = [&](int t, int u, int r) {
        return (la_channel<T>(t, lg) + r) * CD + col + 16 * u;
    };
    if (OUT && !given) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) St[t][u] = mine[(t * CT + u) * 64];
    } else if (given && w.init && !w.trans) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) St[t][u] = *(const f32x4*)(w.init + state_at + at(t, u));
    } else if (given && w.init) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u)
#pragma unroll
                for (int r = 0; r < 4; ++r) St[t][u][r] = w.init[state_at + at_trans(t, u, r)];
    } else {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) St[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
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
            dg[r] = la_within(w.intra * la_pow(l2, d > 0 ? d : 0));
            lw[r] = la_within(w.intra * la_pow(l2, 16 + d));
        }
    }
    // s l^(Q-1-j) of the lane's k slots, j = KS k + 16 (s / 4) + 4 lg + s % 4: a factor of
    // the lane's and one that all lanes share, held as a scalar
    const float wl = la_pow(l2, 12 - 4 * lg);
    float wk[NK][SL];
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int s = 0; s < SL; ++s)
            wk[k][s] = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(
                la_within(w.state_scale * la_pow(l2, Q - 13 - (KS * k + 16 * (s / 4) + s % 4))))));
    // The given state of a REV walk is not decayed before its first use.
    const bool late = REV && given;
    // l^n, compounded from chunk to chunk: the exact power, rounded once
    auto power = [&](int e) { return e == 0 ? 1.f : la_held((float)exp((double)e * (double)ld)); };
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
        rb.store(sb);
        rc.store(sc);
        if constexpr (OUT) {
            ra.store(sa);
            if (rc.wild()) *wild = 1;
        }
        __syncthreads();
        bool tame = false;
        // The next chunk's rows are fetched in three goes, between which the misses of the last
        // one drain: in one go, after M a_i, the waves stand still until the CU has accepted
        // them (the backward's walks of 2 x 8192 tokens, 32 heads of 128 x 64, one bf16 a score:
        // 266 us instead of 280).  The last chunk's fetches repeat its rows (no branch, so no full waits at a join).
        const int next = k + 1 < nch ? k + 1 : k;
        load(rb, pb, bts, next);
        if constexpr (!OUT) load(rc, pc, cts, next);
        const float keep = k + 1 == nch ? llast : (k == 0 ? lfirst : lq);
        if (OUT && n != Q) {  // the last chunk's tokens begin at row Q - n
            int i0 = lr - (Q - n) + (late && k == 0 ? 0 : 1);
            asm volatile("" : "+v"(i0));  // computed here, not held from before the loop
#pragma unroll
            for (int t = 0; t < NT; ++t)
                row[t] = w.inter * la_pow(l2, 16 * t + i0 > 0 ? 16 * t + i0 : 0);
        }

        f32x4 o[NT][CT];
        if constexpr (OUT) {
            // The scores' k blocks up to the diagonal, (row tile, k block), dealt out evenly: of
            // bf16's ten tiles three, three, two and two.
            const int first = NT == 4 ? (wave < 2 ? 2 * wave : 3) : (wave > 0);
            const int units = NT == 4 ? (wave < 2 ? 2 : 1) : (wave < 3);
#pragma unroll 1
            for (int x = 0; x < units; ++x) {
                const int it = first + (NT == 4 && wave == 0 ? x : 0);
                const int kb = NT == 4 ? (wave == 0 ? 0 : (wave == 1 ? x : wave - 2)) : wave == 2;
                // both tiles' operands are read at once; a tile above the diagonal is dropped
                Frag af[KB], bf[TPK][KB];
#pragma unroll
                for (int q = 0; q < KB; ++q) {
                    af[q] = M::load(sa + (16 * it + lr) * AP + KS * q + SL * lg);
#pragma unroll
                    for (int e = 0; e < TPK; ++e)
                        bf[e][q] = M::load(sb + (16 * (kb * TPK + e) + lr) * AP + KS * q + SL * lg);
                }
                f32x4 tl[TPK];
#pragma unroll
                for (int e = 0; e < TPK; ++e) tl[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < KB; ++q)
#pragma unroll
                    for (int e = 0; e < TPK; ++e) tl[e] = M::mma(bf[e][q], af[q], tl[e]);
#pragma unroll
                for (int e = 0; e < TPK; ++e) {
                    const int d = it - (kb * TPK + e);
                    const float f = d <= 1 ? 1.f : (d == 2 ? l16 : l32);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        tl[e][r] = d < 0 || (d == 0 && 4 * lg + r > lr)
                                       ? 0.f
                                       : tl[e][r] * (d == 0 ? dg[r] : lw[r]) * f;
                }
                Frag pf[PARTS];
                la_frag<T>(tl, pf);
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    sp[((it * NK + kb) * PARTS + p) * 64 + lane] = pf[p];
            }
            if (*wild) {  // for the whole workgroup
                tame = true;
                if (threadIdx.x < CD) {
                    int first = Q;
#pragma unroll 1
                    for (int j = Q - 1; j >= 0; --j)
                        if (!(fabsf((float)sc[j * CP + threadIdx.x]) < INFINITY)) {
                            sc[j * CP + threadIdx.x] = (T)0.f;
                            first = j;
                        }
                    wild_row[threadIdx.x] = first;
                }
                __syncthreads();  // before bar 2 every wave has read the flag
                if (threadIdx.x == 0) *wild = 0;
            }
            load(ra, pa, ats, next);
            // l^(i+1) M a_i
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < CT; ++u) o[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                Frag sf[CT][PARTS];
#pragma unroll
                for (int u = 0; u < CT; ++u) {
                    f32x4 tl[TPK];
#pragma unroll
                    for (int e = 0; e < TPK; ++e) tl[e] = St[q * TPK + e][u];
                    la_frag<T>(tl, sf[u]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const Frag a = M::load(sa + (16 * t + lr) * AP + KS * q + SL * lg);
#pragma unroll
                    for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
                        for (int u = 0; u < CT; ++u) o[t][u] = M::mma(sf[u][p], a, o[t][u]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < CT; ++u) o[t][u] *= row[t];
            load(rc, pc, cts, next);
            __syncthreads();  // the scores are there
        }

        Frag cf[NK][CT];
#pragma unroll
        for (int kb = 0; kb < NK; ++kb)
#pragma unroll
            for (int u = 0; u < CT; ++u)
                cf[kb][u] = XT<T>::load(sc, CP, KS * kb, wave * CW + 16 * u, lane);
        if constexpr (OUT) {
#pragma unroll
            for (int part = PARTS - 1; part >= 0; --part) {
                Frag p[NT][NK];
#pragma unroll
                for (int kb = 0; kb < NK; ++kb)
#pragma unroll
                    for (int t = kb * TPK; t < NT; ++t)
                        p[t][kb] = sp[((t * NK + kb) * PARTS + part) * 64 + lane];
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int kb = 0; kb < NK; ++kb)
#pragma unroll
                    for (int t = kb * TPK; t < NT; ++t)
#pragma unroll
                        for (int u = 0; u < CT; ++u) o[t][u] = M::mma(cf[kb][u], p[t][kb], o[t][u]);
            }
        }
        if constexpr (OUT) {
            // a lane holds channels 4 lg .. of row lr of every tile; rows without a token are
            // beyond the buffer's bound
            if (tame)
#pragma unroll
                for (int u = 0; u < CT; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int first = wild_row[wave * CW + 16 * u + 4 * lg + r];
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            if (16 * t + lr >= first) o[t][u][r] = NAN;
                    }
            typedef typename std::conditional<OUT == LA_F32, float, T>::type OT;
            const __amdgpu_buffer_rsrc_t r = buf_rsrc(
                (OT*)w.out + first_token(k, n) * w.out_ts + (int64_t)h * CD, n * out_bytes);
            auto row_at = [&](int i) { return (REV ? Q - 1 - i : i - (Q - n)) * out_bytes; };
            if constexpr (sizeof(OT) == 2) {
                const int half = lg & 1, c8 = wave * CW + 8 * (lg >> 1);
                if constexpr (CT == 2) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        buf_store(la_pair(o[t][0], o[t][1]), r,
                                  row_at(16 * t + lr) + (c8 + 16 * half) * 2);
                } else {
#pragma unroll
                    for (int t = 0; t < NT; t += 2)
                        buf_store(la_pair(o[t][0], o[t + 1][0]), r,
                                  row_at(16 * (t + half) + lr) + c8 * 2);
                }
            } else {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int u = 0; u < CT; ++u)
                        buf_store(o[t][u], r, row_at(16 * t + lr) + (wave * CW + 16 * u + 4 * lg) * 4);
            }
        }

        // M <- l^n M + b^T (w c)
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
                    float x = (float)cf[kb][u][s] * wl * wk[kb][s];
#pragma unroll
                    for (int p = 0; p < SPLITS; ++p) {
                        wc[p][u][s] = (T)x;
                        x -= (float)wc[p][u][s];
                    }
                }
            // Two tiles of b are read while the products of the last two run: left to itself the
            // compiler reads one and waits for it (span pass of 2 x 8192 tokens, 32 heads of
            // 128 x 64: 47 us instead of 52).
            Frag bt[2] = {la_bt<T>(sb, AP, KS * kb, 0, lane), la_bt<T>(sb, AP, KS * kb, 1, lane)};
#pragma unroll
            for (int t = 0; t < BT; t += 2) {
                const int nx = t + 2 < BT ? t + 2 : t;
                const Frag n0 = la_bt<T>(sb, AP, KS * kb, nx, lane),
                           n1 = la_bt<T>(sb, AP, KS * kb, nx + 1, lane);
                __builtin_amdgcn_sched_barrier(6);  // only ALU work moves across
#pragma unroll
                for (int p = SPLITS - 1; p >= 0; --p)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int u = 0; u < CT; ++u)
                            St[t + e][u] = M::mma(bt[e], wc[p][u], St[t + e][u]);
                bt[0] = n0;
                bt[1] = n1;
            }
        }

        if (late && k == 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) row[t] *= l1;
        }
        if (OUT && tame)
#pragma unroll
            for (int u = 0; u < CT; ++u)
                if (wild_row[col + 16 * u] < Q)
#pragma unroll
                    for (int t = 0; t < BT; ++t) St[t][u] = f32x4{NAN, NAN, NAN, NAN};
    }

    if constexpr (!OUT) {
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) mine[(t * CT + u) * 64] = St[t][u];
    } else if (w.fin && sp_.last) {
        const float keep = REV && sp_.n > 0 ? power(1) : 1.f;
#pragma unroll
        for (int t = 0; t < BT; ++t)
#pragma unroll
            for (int u = 0; u < CT; ++u) {
                const f32x4 v = St[t][u] * keep;
                float* p = w.fin + state_at;
                if (w.trans) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[at_trans(t, u, r)] = v[r];
                } else {
                    *(f32x4*)(p + at(t, u)) = v;
                }
            }
    }
}

// What a workgroup of a launch works on.  The hardware deals workgroups out over the 8 XCDs
// in turn.  Those that read the same rows (the walks of a backward, the heads that share
// keys and values: `members` of them) go to one XCD, whose L2 then holds the rows; such
// units, and with them the idle numbers, are spread over all.  (In contiguous ranges to an
// XCD, idle ones leave some XCDs with more spans than they have room for at once: 119 us
// instead of 88 us for the walk of 2 x 8192 tokens, 32 heads of 128 x 64.)
struct LaItem {
    int64_t slot;
    int h, member;  // member / share: the walk
};
__device__ __forceinline__ LaItem la_item(const LaWalk& w, int members) {
    const int64_t unit = (int64_t)(blockIdx.x / 8 / members) * 8 + blockIdx.x % 8;
    const int groups = w.H / w.share;
    LaItem i;
    i.slot = unit / groups;
    i.member = (int)(blockIdx.x / 8 % members);
    i.h = (int)(unit % groups) * w.share + i.member % w.share;
    return i;
}
inline dim3 la_grid(const LaWalk& w, const LaPlan& p, int members) {
    const int64_t units = p.slots * (w.H / w.share);
    return dim3((unsigned)((units + 7) / 8 * 8 * members));
}

// Waves per SIMD that the registers allow.
template <int BD, int CD, int OUT>
constexpr int la_waves() {
    return BD + CD <= 128 || (OUT == LA_STATE && BD + CD <= 192) ? 3 : 2;
}

template <typename T, int BD, int CD, int OUT, int SPLITS>
__global__ void __launch_bounds__(256, (la_waves<BD, CD, OUT>()))
k_la_fwd(LaWalk w, LaPlan plan, f32x4* __restrict__ ws) {
    __shared__ __align__(16) unsigned char lds[la_lds_bytes<T, BD, CD, OUT>()];
    const LaItem i = la_item(w, w.share);
    if (i.slot < plan.slots) la_walk<T, BD, CD, false, OUT, SPLITS>(w, plan, ws, lds, i.slot, i.h);
}

// The three walks of the backward, DQ from the first token on, DV and DK from the last one
// back, in one launch: dv and dk then read q and do at the same time, from one L2.
enum { LA_DQ = 0, LA_DV = 1, LA_DK = 2 };
struct LaBwd {
    LaWalk w[3];
    f32x4* ws[3];
};
template <typename T, int DK, int DV, int OUT, int SPLITS, int SPLITS_DV>
__global__ void __launch_bounds__(256, (la_waves<DK, DV, OUT>()))
k_la_bwd(LaBwd b, LaPlan plan) {
    constexpr int LA = la_lds_bytes<T, DV, DK, OUT>(), LB = la_lds_bytes<T, DK, DV, OUT>();
    __shared__ __align__(16) unsigned char lds[LA > LB ? LA : LB];
    const LaItem i = la_item(b.w[0], 3 * b.w[0].share);
    if (i.slot >= plan.slots) return;
    const int walk = i.member / b.w[0].share;
    constexpr int ODQ = OUT == LA_STATE ? LA_STATE : LA_ACT;
    if (walk == LA_DQ)
        la_walk<T, DV, DK, false, ODQ, SPLITS>(b.w[LA_DQ], plan, b.ws[LA_DQ], lds, i.slot, i.h);
    else if (walk == LA_DV)
        la_walk<T, DK, DV, true, OUT, SPLITS_DV>(b.w[LA_DV], plan, b.ws[LA_DV], lds, i.slot, i.h);
    else
        la_walk<T, DV, DK, true, OUT, SPLITS>(b.w[LA_DK], plan, b.ws[LA_DK], lds, i.slot, i.h);
}

}  // namespace ssd
