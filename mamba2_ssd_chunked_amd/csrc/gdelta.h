// The gated delta rule over chunks of 64 tokens (bf16 and float32 MFMA): what its kernels share.
//
// With c_i the sum of the log decays of a chunk's tokens up to i, C its last, M_ij = e^(c_i - c_j)
// for j <= i, S the state that enters the chunk and B = diag(beta):
//   u_i = beta_i (v_i - e^(c_i) S k_i - sum_{j<i} M_ij (k_i . k_j) u_j)
// is a triangular system, (I + A) U = B (V - diag(e^c) K S^T) with A_ij = beta_i M_ij (k_i . k_j).  Its
// inverse T = (I + A)^-1 does not depend on the state, so that
//   k_gd_prep   T and P_ij = scale M_ij (q_i . k_j) of every chunk, all at once
//   k_gd_walk   from chunk to chunk  U = T B (V - e^c K S^T),  O = scale e^c Q S^T + P U,
//               S <- e^C S + sum_j e^(C - c_j) u_j k_j^T
// leave only the walk to go one chunk after the other.
//
// Backward, with G the gradient of the state behind the chunk and do that of its outputs:
//   k_gd_walk   again, keeping the entering states and U
//   k_gd_back   from the last chunk to the first
//                 Z = T^T (P^T do + e^(C - c) K G^T),  G <- e^C G + scale (e^c do)^T Q - (e^c B Z)^T K
//               keeping the G behind every chunk and Z
//   k_gd_chunk  all chunks at once, with E = scale M (do U^T) on and below the diagonal and N =
//               B M (Z U^T) below it
//                 dq = scale e^c do S + E K,  dv = B Z,  dbeta = Z . U / beta
//                 dk = E^T Q + e^(C - c) U G - e^c B Z S - (N + N^T) K
//               and dg: e^(c_i) multiplies q_i, divides v_i and nothing else if states are counted in
//               units of e^c, so the gradient of c_i is q_i . dq_i - v_i . dv_i, that of C has <G,
//               S behind the chunk> besides, and dg_t is the sum of them from t to the chunk's end.
//
// A wave owns 16 or 32 value channels for a whole sequence: columns of S^T, X = K S^T, U.  Operand
// layouts are those of la_walk.h, and every result in the chain is the next product's operand
// as it lies in registers, so that waves share nothing but the staged rows:
//   X [j][cd]   = K S^T    : rows of K; S^T's tiles, k its channels (la_channel)
//   U [i][cd]   = T R      : rows of T, kept in the order of its k slots; R made of X's tiles
//   S^T [bd][cd] += K^T U  : K read transposed (la_bt); U's tiles
//   O^T [cd][i] = S Q^T + U^T P^T : the same tiles as the other operand, so that a lane has four
//                 neighbouring channels of a token
#pragma once

#include "la_walk.h"
#include "layer_internal.h"

namespace ssd {

constexpr int GD_Q = GD_CHUNK, GD_NT = GD_Q / 16;

// Parts of a float32 value as an operand: bf16 cut off after 8 bits each, the last one rounded.
// Two leave out 2^-16 of it, three 2^-24.
template <typename T, int P>
__device__ __forceinline__ void gd_split(const f32x4* tiles, typename Mma<T>::Frag (&f)[P]) {
    if constexpr (sizeof(T) == 4) {
        f[0] = tiles[0];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float x = tiles[e / 4][e % 4];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (p == P - 1) {
                    f[p][e] = (bf16)x;
                } else {
                    const unsigned hi = __float_as_uint(x) & 0xffff0000u;
                    f[p][e] = __builtin_bit_cast(bf16, (unsigned short)(hi >> 16));
                    x -= __uint_as_float(hi);
                }
            }
        }
    }
}

// Rows of D elements of a chunk on their way into LDS, by NTHR threads; rows without a token are
// zeros (bounded loads).
template <typename T, int D, int NTHR = 256>
struct GdRows {
    static constexpr int VEC = 16 / (int)sizeof(T), VPR = D / VEC, NP = GD_Q * VPR / NTHR;
    static constexpr int PITCH = D + VEC;
    static_assert(GD_Q * VPR % NTHR == 0, "the threads tile the rows");
    typedef T vt __attribute__((ext_vector_type(VEC)));
    vt v[NP];

    __device__ __forceinline__ void load(const T* base, int64_t ts, int64_t t0, int n) {
        const int bytes = (int)ts * (int)sizeof(T);
        const __amdgpu_buffer_rsrc_t r = buf_rsrc(base + t0 * ts, n * bytes);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int x = i * NTHR + threadIdx.x;
            v[i] = buf_load<vt>(r, x / VPR * bytes + x % VPR * 16);
        }
    }
    __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int x = i * NTHR + threadIdx.x;
            *(vt*)(lds + x / VPR * PITCH + x % VPR * VEC) = v[i];
        }
    }
    // the first row of this thread with a value that is not finite, or GD_Q
    __device__ __forceinline__ int wild_row() const {
        int first = GD_Q;
#pragma unroll
        for (int i = NP - 1; i >= 0; --i)
            if (la_wild(v[i])) first = (i * NTHR + (int)threadIdx.x) / VPR;
        return first;
    }
};

// A row of T or P: for each part 64 columns, in the order of an operand's k slots: column 32 b + 16 e
// + 4 g + r stands at 32 b + 8 g + 4 e + r (float32: as it is).
template <typename T, int PARTS>
struct GdMat {
    static constexpr int D = GD_Q * PARTS, PITCH = GdRows<T, D>::PITCH;
    // row operand of tile t, columns of k block b
    __device__ static __forceinline__ typename Mma<T>::Frag row(const T* m, int t, int b, int part, int lane) {
        return Mma<T>::load(m + (16 * t + lane % 16) * PITCH + part * GD_Q + Mma<T>::KS * b +
                            Mma<T>::SL * (lane / 16));
    }
    // the transposed matrix's: rows are columns of tile t, k the rows of block b
    __device__ static __forceinline__ typename Mma<T>::Frag col(const T* m, int t, int b, int part, int lane) {
        return la_bt<T>(m + part * GD_Q, PITCH, Mma<T>::KS * b, t, lane);
    }
    // where the four columns 16 t + 4 lg .. stand
    __device__ static __forceinline__ int at(int t, int lg) { return la_channel<T>(t, lg); }
};

// c += a b for operands in parts, terms below the smallest part left out, small ones first.
// Transposed: c^T += b^T a^T (the same operands the other way round).
template <typename T, int PA, int PB>
__device__ __forceinline__ f32x4 gd_mma(const typename Mma<T>::Frag* a, const typename Mma<T>::Frag* b,
                                        f32x4 c) {
    constexpr int N = PA > PB ? PA : PB;
#pragma unroll
    for (int s = N - 1; s >= 0; --s)
#pragma unroll
        for (int x = 0; x <= s; ++x)
            if (x < PA && s - x < PB) c = Mma<T>::mma(a[x], b[s - x], c);
    return c;
}

// What a workgroup of a walk works on: one sequence, one head, one block of value channels.  Those
// that read the same keys go to one XCD (workgroup i runs on XCD i % 8).
struct GdItem {
    int s, h, cb;
};
__device__ __forceinline__ GdItem gd_item(const GdArgs& a, int nblk) {
    const int members = a.share * nblk, groups = a.H / a.share;
    const int64_t unit = (int64_t)(blockIdx.x / 8 / members) * 8 + blockIdx.x % 8;
    const int member = blockIdx.x / 8 % members;
    GdItem i;
    i.s = unit / groups < a.nseq ? (int)(unit / groups) : -1;
    i.h = (int)(unit % groups) * a.share + member / nblk;
    i.cb = member % nblk;
    return i;
}
inline dim3 gd_grid(const GdArgs& a, int nblk) {
    const int64_t units = (int64_t)a.nseq * (a.H / a.share);
    return dim3((unsigned)((units + 7) / 8 * 8 * a.share * nblk));
}

// Spans of one chunk each: numbers of chunks and places of the states that enter them.
inline LaPlan gd_plan(const GdArgs& a) {
    LaPlan p;
    p.span = GD_Q;
    p.per_row = (int)((a.seqlen + GD_Q - 1) / GD_Q);
    p.slots = a.cu ? a.tokens / GD_Q + a.nseq : (int64_t)a.nseq * p.per_row;
    p.split = false;
    return p;
}

// Per-token factors of a chunk in LDS.
struct GdScalars {
    float in[GD_Q], out[GD_Q], beta[GD_Q];  // e^c, e^(C - c), beta
    int bad;                                // first row with a value that is not finite, or GD_Q
};
__device__ __forceinline__ void gd_scalars_store(GdScalars* s, f32x4 v) {  // by the first wave
    s->in[threadIdx.x] = v[0];
    s->out[threadIdx.x] = v[1];
    s->beta[threadIdx.x] = v[2];
    const unsigned long long bad = __ballot(v[3] != 0.f);
    if (threadIdx.x == 0) s->bad = bad ? __ffsll(bad) - 1 : GD_Q;
}

}  // namespace ssd
