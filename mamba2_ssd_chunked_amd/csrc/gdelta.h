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
//
// What bounds them.  A chunk of 64 tokens depends on the one before it, so that a walk is as long as its
// longest sequence: 128 chunks of 128 x 64 take a team 2.3 us each, three barriers and the reads of what the other
// waves left in LDS.  With more heads and sequences than CUs a chunk of 128 x 128 takes a
// wave of two tiles 12000 cycles, 5800 of them matrix instructions.  prep is bound by its solves in float32 and
// their LDS reads (110 us for 8192 chunk-heads of 128, of 55 us of bytes), chunk by waiting for 256 KB a head,
// which nothing overlaps, with 54 registers spilled (915 us for 8192 of 128 x 128, 470 at the copy's rate).
#pragma once

#include "la_walk.h"
#include "layer_internal.h"

namespace ssd {

constexpr int GD_Q = GD_CHUNK, GD_NT = GD_Q / 16;

// The smallest beta that the backward's walks count with, since dbeta is divided by it; what it adds to states is
// far below float32's precision of what they stand for.  The chunks' gradients take the given one.
constexpr float GD_BETA_MIN = 9.094947017729282e-13f;  // 2^-40

// Parts of a float32 value as an operand: bf16 rounded, and so the remainders, which are exact.  Two
// leave out 2^-18 of it, three nothing.  The remainder of a value of a pair is one dot product, of the pair's
// bf16 and (-1, 0) or (0, -1), where taking the part apart and subtracting it would be two
// instructions.  (The constants come from registers: as immediates the compiler encodes (-1, 0) as what the
// hardware reads as (0, -1).)
template <typename T, int P>
__device__ __forceinline__ void gd_split(const f32x4* tiles, typename Mma<T>::Frag (&f)[P]) {
    if constexpr (sizeof(T) == 4) {
        f[0] = tiles[0];
    } else {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        unsigned first = 0x0000bf80u, second = 0xbf800000u;
        asm("" : "+s"(first), "+s"(second));
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float x = tiles[e / 4][e % 4], y = tiles[e / 4][e % 4 + 1];
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const b2 h = {(bf16)x, (bf16)y};
                f[p][e] = h[0];
                f[p][e + 1] = h[1];
                if (p < P - 1) {
                    x = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(b2, first), x, false);
                    y = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(b2, second), y, false);
                }
            }
        }
    }
}

// f(0), f(1), .. f(N - 1) with constants.
template <int... I, typename F>
__device__ __forceinline__ void gd_each(std::integer_sequence<int, I...>, F&& f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void gd_for(F&& f) {
    gd_each(std::make_integer_sequence<int, N>{}, f);
}

// gd_split of eight values in 4 P steps of a few instructions each, to be dealt out between matrix
// instructions; a pair's next step comes four steps later (a remainder takes a few cycles to arrive).
template <int P>
struct GdSplit {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    static constexpr int STEPS = 4 * P;
    bf16x8 f[P];
    float x[8];
    __device__ __forceinline__ void set(f32x4 a, f32x4 b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a[e], x[4 + e] = b[e];
    }
    template <int I>
    __device__ __forceinline__ void step(unsigned first, unsigned second) {
        constexpr int e = I % 4 * 2, p = I / 4;
        const b2 h = {(bf16)x[e], (bf16)x[e + 1]};
        f[p][e] = h[0];
        f[p][e + 1] = h[1];
        if constexpr (p < P - 1) {
            x[e] = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(b2, first), x[e], false);
            x[e + 1] = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(b2, second), x[e + 1], false);
        }
    }
};
// The combinations of PA and PB parts whose weight counts, small ones first: part I of the list.
template <int PT>
struct GdPairs {
    static constexpr int N = PT * (PT + 1) / 2;
    static constexpr int sum(int i) { return i < PT ? PT - 1 : (i < 2 * PT - 1 ? PT - 2 : 0); }
    static constexpr int a(int i) { return i < PT ? i : (i < 2 * PT - 1 ? i - PT : 0); }
    static constexpr int b(int i) { return sum(i) - a(i); }
};

// NM matrix instructions m(i) with NW pieces of other work w(i) dealt out evenly behind them, from the
// LEAD-th on; the compiler keeps the order.  A wave that has its SIMD for itself would else do one after the
// other.
template <int NM, int NW, int LEAD, typename FM, typename FW>
__device__ __forceinline__ void gd_weave(FM&& m, FW&& w) {
    constexpr int over = NM - LEAD > 0 ? NM - LEAD : 1;
    gd_for<NM>([&](auto I) {
        constexpr int i = decltype(I)::value - LEAD;
        m(I);
        constexpr int from = i < 0 ? 0 : i * NW / over, to = i < 0 ? 0 : (i + 1) * NW / over;
        gd_for<to - from>([&](auto J) { w(std::integral_constant<int, from + decltype(J)::value>{}); });
        __builtin_amdgcn_sched_barrier(0);
    });
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

// ---- staging -----------------------------------------------------------------------------------
// A chunk's operands go from memory to LDS without passing through registers (buffer_load ... lds: lane l of
// a wave writes 16 bytes at the wave's address + 16 l; beyond the bound it writes zeros), while the chunk
// before is computed: two buffers, one barrier per chunk.  The compiler does not know of these loads:
// gd_wait is what waits for them.
typedef int gd_i4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ gd_i4 gd_rsrc(const void* p, int bytes) {
    const uint64_t a = (uint64_t)p;
    return gd_i4{__builtin_amdgcn_readfirstlane((int)a), __builtin_amdgcn_readfirstlane((int)(a >> 32) & 0xffff),
                 __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}
__device__ __forceinline__ unsigned gd_lds(const void* p) {
    return __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(__attribute__((address_space(3))) const char*)p);
}
// The compiler does not look into the assembly: a descriptor that a vector instruction wrote (v_readfirstlane, or
// v_readlane of a spilled one) may be read by a vector memory instruction five wait states later only, so that each
// load brings its own five, the move to m0 and s_nop 3.
__device__ __forceinline__ void gd_dma16(gd_i4 r, unsigned lds, int off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r)
                 : "memory", "m0");
}
__device__ __forceinline__ void gd_dma4(gd_i4 r, unsigned lds, int off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(off), "s"(r)
                 : "memory", "m0");
}
// Until at most N of this wave's memory accesses are on their way: all but the last N are done.
template <int N>
__device__ __forceinline__ void gd_wait() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// 64 rows of D elements in LDS, without padding: the 16-byte pieces of a row are exchanged by its number,
// so that neither 16 rows' pieces nor the transposed reads of 4-row groups meet in a bank (of the
// latter half of each piece is read at once: twice is the least).
template <typename T, int D>
struct GdTile {
    static constexpr int RB = D * (int)sizeof(T), PPR = RB / 16, BYTES = GD_Q * RB;
    __device__ static __forceinline__ int flip(int row) {
        constexpr int m = PPR - 1;
        if constexpr (sizeof(T) == 4) return ((4 * ((row >> 2) & 3)) ^ (row & 3)) & m;
        else if constexpr (D == 128) return (4 * (row & 3)) ^ (2 * ((row >> 2) & 1));
        else return ((4 * ((row >> 1) & 1)) ^ (2 * ((row >> 2) & 1))) & m;
    }
    __device__ static __forceinline__ int at(int row, int piece) { return row * RB + ((piece ^ flip(row)) << 4); }
    static constexpr int FETCHES = BYTES / 1024;
    // the i-th fetch of rows `bytes` apart
    __device__ static __forceinline__ void fetch(gd_i4 r, int bytes, unsigned lds, int i, int lane) {
        const int x = i * 64 + lane, row = x / PPR, piece = (x % PPR) ^ flip(row);
        gd_dma16(r, lds + i * 1024, row * bytes + piece * 16);
    }
    // row operand: rows of tile t, k block q
    __device__ static __forceinline__ typename Mma<T>::Frag row(const char* m, int t, int q, int lane) {
        const int lr = lane % 16, lg = lane / 16;
        return *(const typename Mma<T>::Frag*)(m + 16 * t * RB + at(lr, 4 * q + lg));
    }
    // transposed, k the tokens from jb: columns of tile t in the order of la_channel ...
    __device__ static __forceinline__ typename Mma<T>::Frag bt(const char* m, int jb, int t, int lane) {
        if constexpr (sizeof(T) == 4) return xt(m, jb, 16 * t, lane);
        else return tr(m, jb, lane, 4 * (t / 2) + lane % 4, 8 * (t % 2));
    }
    // ... or the 16 from p0 on
    __device__ static __forceinline__ typename Mma<T>::Frag xt(const char* m, int jb, int p0, int lane) {
        if constexpr (sizeof(T) == 4) {
            const int i = lane % 16, g = lane / 16;
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = *(const float*)(m + jb * RB + at(4 * g + e, p0 / 4 + i / 4) + 4 * (i % 4));
            return v;
        } else {
            return tr(m, jb, lane, p0 / 8 + (lane % 4) / 2, 8 * (lane % 2));
        }
    }
    __device__ static __forceinline__ bf16x8 tr(const char* m, int jb, int lane, int piece, int byte) {
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s4 lds_s4;
        const char* a = m + jb * RB + at(4 * (lane / 16) + lane % 16 / 4, piece) + byte;
        const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)a));
        const bf16x4 hi = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(a + 16 * RB)));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// T or P.  In memory a row per token: for each part 64 columns, in the order of an operand's k slots (column
// 32 b + 16 e + 4 g + r stands at 32 b + 8 g + 4 e + r; float32: as it is).  In LDS the operands
// one after the other, those on and below the diagonal: 16 rows of 64 bytes, whose pieces are exchanged
// by the row's number against bank conflicts.
template <typename T, int PARTS>
struct GdMat {
    typedef typename Mma<T>::Frag Frag;
    static constexpr int TPK = LaCfg<T>::TPK, NK = GD_Q / Mma<T>::KS;
    static constexpr int D = GD_Q * PARTS, NTB = NK * (NK + 1) / 2 * TPK, BYTES = NTB * PARTS * 1024;
    __device__ static __forceinline__ int tb(int t, int b) {  // of (row tile, k block)
        return TPK == 2 ? (t < 2 ? t : 2 * t - 2 + b) : t * (t + 1) / 2 + b;
    }
    __device__ static __forceinline__ int slot(int lg, int lr) { return 4 * lr + (lg ^ (lr / 4)); }
    static constexpr int FETCHES = NTB * PARTS;
    static constexpr int ROW = D * (int)sizeof(T);  // bytes of a row in memory
    __device__ static __forceinline__ void fetch(gd_i4 r, unsigned lds, int i, int lane) {
        const int x = i / PARTS, p = i % PARTS;
        int t, b;
        if constexpr (TPK == 2) {
            t = x < 2 ? x : x / 2 + 1;
            b = x < 2 ? 0 : x % 2;
        } else {
            t = x < 1 ? 0 : (x < 3 ? 1 : (x < 6 ? 2 : 3));
            b = x - t * (t + 1) / 2;
        }
        // four lanes to 64 bytes of a row (sixteen rows' first pieces, then their second ones, .. take four times as long)
        const int lr = lane / 4, lg = lane % 4 ^ (lr / 4), row = 16 * t + lr;
        gd_dma16(r, lds + i * 1024, row * ROW + 16 * lg + p * (GD_Q * (int)sizeof(T)) + 64 * b);
    }
    // row operand of tile t, columns of k block b
    __device__ static __forceinline__ Frag row(const char* m, int t, int b, int part, int lane) {
        return *(const Frag*)(m + (tb(t, b) * PARTS + part) * 1024 + slot(lane / 16, lane % 16) * 16);
    }
    // the transposed matrix's: rows are columns of tile t, k the rows of block b
    __device__ static __forceinline__ Frag col(const char* m, int t, int b, int part, int lane) {
        if constexpr (sizeof(T) == 4) {
            const int i = lane % 16, g = lane / 16;
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = *(const float*)(m + tb(b, t) * 1024 + slot(i / 4, 4 * g + e) * 16 + 4 * (i % 4));
            return v;
        } else {
            typedef short s4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4 lds_s4;
            const char* a = m + part * 1024 + slot(lane % 4, 4 * (lane / 16) + lane % 16 / 4) * 16 + 8 * (t % 2);
            const bf16x4 lo = __builtin_bit_cast(
                bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(a + tb(2 * b, t / 2) * (PARTS * 1024))));
            const bf16x4 hi = __builtin_bit_cast(
                bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(a + tb(2 * b + 1, t / 2) * (PARTS * 1024))));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

// A matrix of a chunk by rows in LDS: for each part 64 columns, in the order of an operand's k slots: column 32 b + 16 e
// + 4 g + r stands at 32 b + 8 g + 4 e + r (float32: as it is).
template <typename T, int PARTS>
struct GdRowsMat {
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

// Waves of a walk's workgroup and column tiles of each; one wave: a team (gdelta_team.h).  A wave is bound by the
// instructions that it can issue and its workgroup by the operands that it reads from LDS, so that the fewest waves
// to a CU are the quickest where there are CUs left, and two tiles to a wave, which share operands, where
// there are none.  Sequences count alike whatever their lengths (a long one among many short ones is not walked
// as quickly as it could be).  Microseconds of a forward of rows of 2048 tokens (teams, two waves, four, four of two tiles):
//   bf16, 128 x 128  256 tiles 85 116 - 195, 320 146 120 - 197, 512 166 130 135 207, 768 240 243 160 227,
//                    1024 321 267 190 250; of 1024 tokens 1536 248 199 161 145, 2048 332 272 190 176
//   float32          256 152 344 - 585, 512 284 390 385 635, 768 438 758 432 681, 1024 581 798 468 719;
//                    of 1024 tokens 1536 446 603 434 401
// Operands of 64 channels move none of the bounds.
struct GdShape {
    int waves, tiles;
};
inline int64_t gd_tiles(const GdArgs& a) { return (int64_t)a.nseq * a.H * (a.valdim / 16); }
inline GdShape gd_shape(const GdArgs& a, bool f32) {
    const int64_t tiles = gd_tiles(a);
    if (tiles <= (f32 ? 512 : 256)) return {1, 1};
    if (tiles <= 512) return {2, 1};
    return {4, tiles <= 1024 ? 1 : a.valdim / 64};
}
// The same of the backward's walk, whose waves of two tiles hold too much: two waves or four (128 x 128 in bf16, all
// of a backward: 256 tiles of single waves 342, 335 of two; 512 tiles 548 and 559, 768 864 and 720; 2048 tiles of 1024
// tokens 888, of two tiles to a wave 923).
inline int gd_back_waves(const GdArgs& a) { return gd_tiles(a) <= 512 ? 2 : 4; }

// Spans of one chunk each: numbers of chunks and places of the states that enter them.
inline LaPlan gd_plan(const GdArgs& a) {
    LaPlan p;
    p.span = GD_Q;
    p.per_row = (int)((a.seqlen + GD_Q - 1) / GD_Q);
    p.slots = a.cu ? a.tokens / GD_Q + a.nseq : (int64_t)a.nseq * p.per_row;
    p.split = false;
    return p;
}

// Per-token factors of a chunk in LDS: e^c, e^(C - c) (-1 behind a value that is not finite), beta; zeros
// where there is no token.
struct GdScalars {
    float in[GD_Q], out[GD_Q], beta[GD_Q];
};
__device__ __forceinline__ void gd_scalars_fetch(const GdArgs& a, int64_t row0, int n, unsigned lds, int i, int lane) {
    const float* p = i == 0 ? a.in : (i == 1 ? a.out : a.beta_of);
    gd_dma4(gd_rsrc(p + row0, n * 4), lds + i * GD_Q * 4, lane * 4);
}
// The number of the J-th fetch of a wave of NW, of N in all (the last ones may be fetched twice).
template <int N, int NW>
__device__ __forceinline__ int gd_mine(int j, int wave) {
    const int i = j * NW + wave;
    return N % NW == 0 || i < N ? i : N - 1;
}
constexpr int gd_share(int n, int waves) { return (n + waves - 1) / waves; }

}  // namespace ssd
