// Shared pieces of the gated delta rule kernels (gfx950).
//
// Per sequence and value head, with a state S [dk][dv], a_t = exp(g_t):
//   S <- a_t S;  S <- S + beta_t k_t (v_t - S^T k_t)^T;  o_t = scale S^T q_t.
// Tokens are taken in chunks of 64. With G the running sum of g in a chunk,
// D_ij = exp(G_i - G_j) for j <= i and S0 the state before the chunk:
//   A_ij = beta_i D_ij (k_i . k_j) for j < i,         T = (I + A)^-1,
//   u = T diag(beta) (V - diag(exp G) K S0),           (what each token writes)
//   O = scale (diag(exp G) Q S0 + P u),                P_ij = D_ij (q_i . k_j), j <= i,
//   S1 = exp(G_last) S0 + K^T diag(exp(G_last - G)) u.
//
// Every product runs on the bf16 matrix cores (v_mfma_f32_16x16x32_bf16) with fp32
// accumulation. An fp32 value enters as a sum of bf16 parts (x = h1 + h2 + ..., each
// the rounding of what the ones before it leave): two parts hold 16 bits, three 24.
// bf16 plans give their inputs exactly in one part and carry the state and T in two; the
// residuals and what a chunk adds to the state have three (relative error of the fp32
// state measured 3e-7 to 7e-7; with two 3e-6, 8% faster; with one 2e-3). So have, in the backward,
// P, dU, r and exp(G) dO, which lead to dS (the fp32 gradient of the state 3e-6 off with two).
// Two also serve the states between the pieces of cut sequences, and P: with one the
// outputs are 2.2e-3 off, with two 1.7e-3, which is what their own rounding leaves (12
// products a chunk more, off the chain). fp32 plans use three parts throughout (1e-7), at 6
// products for each single one, still 2.7 times the rate of the fp32 matrix instruction.
//
// Fragment layouts of v_mfma_f32_16x16x32_bf16, lane l, g = l / 16:
//   A [16][32]: lane holds row l % 16, columns 8g .. 8g+7
//   B [32][16]: lane holds column l % 16, rows 8g .. 8g+7
//   D [16][16]: lane holds column l % 16, rows 4g .. 4g+3
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/hyena.h"

namespace hy {
namespace delta {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kC = 64;           // tokens per chunk
constexpr int kThreads = 256;    // four waves; wave w owns tokens 16w .. 16w+15 of a chunk
constexpr int kFragBytes = 1024; // one fragment part: 64 lanes of 8 bf16
constexpr int kTri = 6;          // fragments of a block-triangular 64 x 64 operand

// Decays below exp(-200) are 0 in fp32 even against the largest values, so the
// logarithm is held there: a gate of -inf (a reset) then stays finite in G_i - G_j.
constexpr double kMinLog = -200.0;

template <bool BF>
struct Io;
template <>
struct Io<true> {
    using T = __bf16;
    static constexpr int NI = 1;  // parts of an input operand (exact)
    static constexpr int NS = 2;  // parts of the state, T and the written values
    static constexpr int NE = 3;  // parts of the residuals and of what a chunk adds to the state; their gradients'
    static constexpr int NO = 2;  // parts of the state and of u against Q and P
    static constexpr int NP = 2;  // parts of P
    static constexpr int NK = 2;  // parts of what the backward's scans keep, in its products
};
template <>
struct Io<false> {
    using T = float;
    static constexpr int NI = 3;
    static constexpr int NS = 3;
    static constexpr int NE = 3;
    static constexpr int NO = 3;
    static constexpr int NP = 3;
    static constexpr int NK = 1;  // as fp32
};

// Fragment f of a lower triangular operand: its row tile and its half of the columns
__device__ __forceinline__ constexpr int tri_row(int f) { return f < 2 ? f : 2 + ((f - 2) >> 1); }
__device__ __forceinline__ constexpr int tri_half(int f) { return f < 2 ? 0 : (f - 2) & 1; }
// Row r of row tile t as the scans number them: the pair of tiles 2s, 2s + 1 covers
// rows 32 s .. 32 s + 31 such that the result rows that one lane holds in both (4 g + i
// of each) are rows 32 s + 8 g .. + 7 in order, which is what the same lane must hold
// of a right-hand operand. Results become operands without leaving their lane.
__device__ __forceinline__ constexpr int tile_row(int t, int r) {
    return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3);
}
template <int N>
struct Frag {
    bf16x8 p[N];
};

// two values rounded to bf16 in one instruction; and back
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x, y}), bf16x2));
}
template <int N>
__device__ __forceinline__ Frag<N> split8(const float (&x)[8]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    Frag<N> f;
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = pack2(r[2 * i], r[2 * i + 1]);
            if (n + 1 < N) {
                r[2 * i] -= __uint_as_float(w[i] << 16);
                r[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        f.p[n] = __builtin_bit_cast(bf16x8, w);
    }
    return f;
}

// products of parts (i, j) with i + j below the larger part count: the rest lies
// below the last part's rounding
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Frag<NA>& a, const Frag<NB>& b, f32x4 c) {
    constexpr int M = NA > NB ? NA : NB;
#pragma unroll
    for (int s = M - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < NB) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], c, 0, 0, 0);
        }
    return c;
}

// the same for J row tiles, products of one part pair next to each other so that
// consecutive instructions do not wait for each other's sums
template <int NA, int NB, int J>
__device__ __forceinline__ void mma_tiles(const Frag<NA> (&a)[J], const Frag<NB>& b, f32x4* c) {
    constexpr int M = NA > NB ? NA : NB;
#pragma unroll
    for (int s = M - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int k = s - i;
            if (k >= 0 && k < NB)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    c[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j].p[i], b.p[k], c[j], 0, 0, 0);
        }
}
// eight consecutive elements as fp32 / as an operand; zeros where !ok
__device__ __forceinline__ void load8(const __bf16* p, bool ok, float (&x)[8]) {
    bf16x8 v = {};
    if (ok) v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}
__device__ __forceinline__ void load8(const float* p, bool ok, float (&x)[8]) {
    f32x4 lo = {}, hi = {};
    if (ok) {
        lo = *reinterpret_cast<const f32x4*>(p);
        hi = *reinterpret_cast<const f32x4*>(p + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = lo[i];
        x[4 + i] = hi[i];
    }
}
// raw registers of eight elements: loads are issued ahead and split when used
struct Raw16 {
    bf16x8 v;
};
struct Raw32 {
    f32x4 lo, hi;
};
__device__ __forceinline__ Frag<1> to_frag(const Raw16& r) { return Frag<1>{{r.v}}; }
__device__ __forceinline__ Frag<3> to_frag(const Raw32& r) {
    const float x[8] = {r.lo[0], r.lo[1], r.lo[2], r.lo[3], r.hi[0], r.hi[1], r.hi[2], r.hi[3]};
    return split8<3>(x);
}
template <bool BF>
struct RawOf {
    using type = Raw16;
};
template <>
struct RawOf<false> {
    using type = Raw32;
};
template <bool BF>
using Raw = typename RawOf<BF>::type;

// Rows of a chunk as a buffer resource: `rows` (0 or less: none) rows of `width` bytes,
// `ld` bytes apart. Loads outside give zeros and stores outside are dropped by the
// hardware's range check, so ragged chunks and padded columns need no branches (whose
// merges would make every wait a full one). Offset kNoElem is outside any of them.
constexpr uint32_t kNoElem = 0x80000000u;
typedef __amdgpu_buffer_rsrc_t RowBuf;
__device__ __forceinline__ RowBuf row_buf(const void* base, int64_t rows, uint32_t ld, uint32_t width) {
    const int n = rows > kC ? kC : (int)rows;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, n > 0 ? (int)((n - 1) * ld + width) : 0,
                                             0x00020000);
}
__device__ __forceinline__ RowBuf plain_buf(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void buf_raw(RowBuf b, uint32_t off, Raw16& r) {
    r.v = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
}
__device__ __forceinline__ void buf_raw(RowBuf b, uint32_t off, Raw32& r) {
    r.lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
    r.hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off + 16, 0, 0));
}
__device__ __forceinline__ f32x4 buf_f4(RowBuf b, uint32_t off, int soff) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, soff, 0));
}
// 64 rows of DK elements in LDS as bf16 parts, read as operands along the rows (K S, Q S)
// or across them (K^T u, by the transposing LDS read). Rows are 64 bytes longer than
// their data, and eight rows shift by 16 bytes, so that consecutive rows start on other banks.
// Bank conflicts still take 31% of the scans' LDS cycles (42% of the ends'), by counter.
template <int NI, int DK>
struct Tile {
    static constexpr int pitch = 2 * DK + 64;
    alignas(16) unsigned char b[NI][kC * pitch];
    __device__ static constexpr int at(int row, int k) { return row * pitch + ((row >> 3) & 3) * 16 + 2 * k; }
    // row tile t, elements 32 s ..: lane (row tile_row(t, col), elements 32 s + 8 g ..)
    __device__ __forceinline__ Frag<NI> rows(int lane, int t, int s) const {
        const int col = lane & 15, g = lane >> 4;
        Frag<NI> f;
#pragma unroll
        for (int n = 0; n < NI; ++n)
            f.p[n] = *reinterpret_cast<const bf16x8*>(b[n] + at(tile_row(0, col), 8 * g) +
                                                      (4 * (t & 1) + 32 * (t >> 1)) * pitch + 64 * s);
        return f;
    }
    // column tile m, rows 32 s ..: lane (element tile_row(m, col), rows 32 s + 8 g ..). The
    // transposing read gives lane i of 16 element i % 4 of the four 8-byte pieces that
    // lanes i/4, i/4 + 4, i/4 + 8 and i/4 + 12 address: one column, four rows.
    __device__ __forceinline__ Frag<NI> cols(int lane, int m, int s) const {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* Lds4;
        const int r = lane & 15, g = lane >> 4;
        Frag<NI> f;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const unsigned char* p = b[n] + at(8 * g + (r >> 2), 8 * (r & 3)) + 32 * s * pitch + 64 * (m >> 1) + 8 * (m & 1);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(p + 4 * pitch));
            typedef short s16x8 __attribute__((ext_vector_type(8)));
            f.p[n] = __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        return f;
    }
};

// 64 rows of CB columns of v in LDS (bf16), read as results lie: lane (column, four rows)
template <int CB>
struct ColTile {
    static constexpr int pitch = 2 * CB + 16;
    alignas(16) unsigned char b[kC * pitch];
    // rows 32 (t / 2) + 8 g + 4 (t % 2) .. + 3 of column c0 + lane % 16, by the transposing read
    __device__ __forceinline__ u32x2 rows4(int lane, int t, int c0) const {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* Lds4;
        const int r = lane & 15, g = lane >> 4;
        const unsigned char* p = b + (8 * g + (r >> 2)) * pitch + 8 * (r & 3) + (32 * (t >> 1) + 4 * (t & 1)) * pitch + 2 * c0;
        return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)p));
    }
};

// A wave moves the tiles (or W waves a share each, rows 64 / W of them): 16 bytes a
// lane, 1 KiB an instruction, whole rows.
template <bool BF, int DK, int W = 1>
struct Stage {
    static constexpr int EPL = BF ? 8 : 4, LR = DK / EPL, RI = 64 / LR, N = LR / W;
    static_assert(W <= 4, "shares of 16 rows or more: their 16-byte shifts add up");
    u32x4 r[N];
    __device__ __forceinline__ void load(RowBuf b, uint32_t ld, int dk, int lane, int w = 0) {
        const uint32_t k = (lane % LR) * EPL, E = BF ? 2 : 4;
        const uint32_t off = (int)k < dk ? (lane / LR + w * (kC / W)) * ld + k * E : kNoElem;
#pragma unroll
        for (int i = 0; i < N; ++i)
            r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)(off + i * RI * ld), 0, 0));
    }
    __device__ __forceinline__ void store(Tile<BF ? 1 : 3, DK>& t, int lane, int w = 0) const {
        using TL = Tile<BF ? 1 : 3, DK>;
        const int at = (lane / LR) * TL::pitch + 2 * (lane % LR) * EPL + TL::at(w * (kC / W), 0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int o = at + i * RI * TL::pitch + ((i * RI >> 3) & 3) * 16;
            if constexpr (BF) {
                *reinterpret_cast<u32x4*>(t.b[0] + o) = r[i];
            } else {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(r[i][j]);
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    u32x2 w;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        w[j] = pack2(x[2 * j], x[2 * j + 1]);
                        x[2 * j] -= __uint_as_float(w[j] << 16);
                        x[2 * j + 1] -= __uint_as_float(w[j] & 0xffff0000u);
                    }
                    *reinterpret_cast<u32x2*>(t.b[n] + o) = w;
                }
            }
        }
    }
};

// part n of fragment f at byte `at` of a record
template <int N>
__device__ __forceinline__ Frag<N> buf_frag(RowBuf b, int at, int f, int lane) {
    Frag<N> r;
#pragma unroll
    for (int n = 0; n < N; ++n)
        r.p[n] = __builtin_bit_cast(bf16x8, buf_f4(b, lane * 16, at + (f * N + n) * kFragBytes));
    return r;
}

template <bool BF>
__device__ __forceinline__ void buf_store(RowBuf b, uint32_t off, float x) {
    if constexpr (BF)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)x), b, (int)off, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), b, (int)off, 0, 0);
}
template <bool BF>
__device__ __forceinline__ float buf_elem(RowBuf b, uint32_t off) {
    if constexpr (BF)
        return __uint_as_float((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, (int)off, 0, 0) << 16);
    else
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (int)off, 0, 0));
}
__device__ __forceinline__ int64_t uniform64(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)x);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

template <int N>
__device__ __forceinline__ Frag<N> get_frag(const __bf16* frag, int part_stride, int lane) {
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) f.p[n] = *reinterpret_cast<const bf16x8*>(frag + n * part_stride + lane * 8);
    return f;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// What is not finite must not reach tokens in front of it, but zeros of T and of P (and of the
// remainders' operand) multiply it there. Where a chunk's outputs show that they met such a
// value, they are made again: rows of x (four tiles, numbered as tile_row has them) from a
// column's first that is not finite on are cleared, and `poison` marks these rows of the result.
// One comparison and a branch a chunk, off the chain, where all is finite (in the state waves,
// whose schedule a branch cuts in two, they took 3% of the scan).
__device__ __forceinline__ int clear_from_first(f32x4 (&x)[4], int lane) {
    const int g = lane >> 4;
    int first = 64;
#pragma unroll
    for (int t = 3; t >= 0; --t)
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const int row = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + i;
            if (!finite(x[t][i]) && row < first) first = row;
        }
#pragma unroll
    for (int d = 16; d < 64; d <<= 1) {
        const int other = __shfl_xor(first, d);
        first = other < first ? other : first;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (32 * (t >> 1) + 8 * g + 4 * (t & 1) + i >= first) x[t][i] = 0.f;
    return first;
}
__device__ __forceinline__ void poison(f32x4 (&x)[4], int first, int lane) {
    const int g = lane >> 4;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (32 * (t >> 1) + 8 * g + 4 * (t & 1) + i >= first) x[t][i] = __builtin_nanf("");
}

// Instruction order of the region before it: N times one matrix instruction followed by
// V vector instructions and by M loads (a lone wave overlaps them only if they alternate).
template <int N, int V, int M>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (V) __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
        if (M) __builtin_amdgcn_sched_group_barrier(0x020, M, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// LDS traffic of the workgroup is complete and every wave is here; loads from
// global memory stay in flight (a __syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// ---------------------------------------------------------------- sequences
struct Seqs {
    const int64_t* start;  // [N + 1] token offsets, or null: N sequences of T tokens
    int64_t N, tokens, T, cpt;
};
struct Range {
    int64_t first, len, slot0;  // tokens first .. first+len-1; chunk c is workspace slot slot0 + c
};
// Offsets come from the device and cannot be checked on the host: they are held to
// 0 <= start[n] <= start[n+1] <= tokens here, so that no access leaves the arrays.
// Sequence n's chunks start at slot start[n]/64 + n: consecutive sequences never
// overlap and tokens/64 + N slots hold them all.
__device__ __forceinline__ Range seq_range(const Seqs& s, int64_t n) {
    Range r;
    if (!s.start) {
        r.first = n * s.T;
        r.len = s.T;
        r.slot0 = n * s.cpt;
    } else {
        int64_t b = s.start[n], e = s.start[n + 1];
        b = b < 0 ? 0 : (b > s.tokens ? s.tokens : b);
        e = e < b ? b : (e > s.tokens ? s.tokens : e);
        r.first = b;
        r.len = e - b;
        r.slot0 = b / kC + n;
    }
    return r;
}
// the sequence and chunk of a slot; false where the slot holds none
__device__ __forceinline__ bool find_chunk(const Seqs& s, int64_t slot, Range& r, int64_t& c, int64_t& n) {
    if (!s.start) {
        n = slot / s.cpt;
    } else {
        int64_t lo = 0, hi = s.N - 1;  // the last n whose first slot is not behind `slot`
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            int64_t b = s.start[mid];
            b = b < 0 ? 0 : (b > s.tokens ? s.tokens : b);
            if (b / kC + mid <= slot)
                lo = mid;
            else
                hi = mid - 1;
        }
        n = lo;
    }
    r = seq_range(s, n);
    c = slot - r.slot0;
    return c >= 0 && c * kC < r.len;
}

// Where few sequences would leave most of the card idle, long ones are cut into pieces of
// `len` chunks that are scanned side by side: a first scan takes every piece but the last
// from a zero state (its end B) and from the identity (its end M: the state behind a piece
// is M S + B), and each piece's own scan begins by carrying the state through the pieces
// before it. That is twice the scan's work and a third of its time from three pieces on,
// so a sequence of up to three pieces' length stays whole.
struct Pieces {
    int64_t len;    // chunks a piece; 0: every sequence whole
    int64_t per;    // piece slots a sequence, where all are of one length
    int64_t slots;  // of the call; sequence n's start at start[n] / (64 len) + n, as chunks do
    float* b;       // [slot][value head][16-column block][tile][lane][4] the ends B
    unsigned char* m;   // [slot][value head] the ends M, as left operands of state tiles in parts
    unsigned char* mt;  // their transposes (backward), or null
};
struct Piece {
    Range r;        // its tokens; chunk c of it is workspace slot r.slot0 + c
    int64_t n;      // sequence
    int64_t first;  // piece slot of the sequence's first piece
    int s, count;   // number in the sequence, pieces of the sequence
};
__device__ __forceinline__ bool find_piece(const Seqs& q, const Pieces& ps, int64_t slot, Piece& p) {
    if (!ps.len) {
        p.n = p.first = slot;
        p.r = seq_range(q, slot);
        p.s = 0;
        p.count = 1;
        return true;
    }
    if (!q.start) {
        p.n = slot / ps.per;
        p.first = p.n * ps.per;
    } else {
        const int64_t unit = kC * ps.len;
        auto start = [&](int64_t n) {
            const int64_t b = q.start[n];
            return b < 0 ? 0 : (b > q.tokens ? q.tokens : b);
        };
        int64_t lo = 0, hi = q.N - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (start(mid) / unit + mid <= slot)
                lo = mid;
            else
                hi = mid - 1;
        }
        p.n = lo;
        p.first = start(lo) / unit + lo;
    }
    p.r = seq_range(q, p.n);
    p.s = (int)(slot - p.first);
    const int64_t chunks = (p.r.len + kC - 1) / kC;
    p.count = chunks > 3 * ps.len ? (int)((chunks + ps.len - 1) / ps.len) : 1;
    if (p.s < 0 || p.s >= p.count) return false;
    if (p.count > 1) {
        const int64_t c0 = p.s * ps.len, left = p.r.len - c0 * kC;
        p.r.first += c0 * kC;
        p.r.slot0 += c0;
        p.r.len = left < ps.len * kC ? left : ps.len * kC;
    }
    return true;
}

// The running sum of the log decays over a chunk's 64 lanes, in 64 bits and to base 2:
// differences of it stay exact to fp32 however strong single decays are, and a decay is one
// hardware exp2 of such a difference (accurate to its last bit or two, as an expf would be).
__device__ __forceinline__ double chunk_decay(float g, int lane) {
    double G = ((double)g < kMinLog ? kMinLog : (double)g) * 1.4426950408889634074;  // a NaN stays one
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(G, d);
        if (lane >= d) G += up;
    }
    return G;
}

// The backward takes dbeta = r . (u / beta), so a write strength of zero is held at 2^-90
// in what it solves for u: the residual u / beta is then there for it, with room for its
// parts above the smallest fp32, and what is written beside it is 1e-27 of a residual.
constexpr float kMinBeta = 0x1p-90f;
__device__ __forceinline__ float held_beta(float b) { return fabsf(b) < kMinBeta ? kMinBeta : b; }

__device__ __forceinline__ float decay(double d) { return __builtin_amdgcn_exp2f((float)d); }

struct Shape {
    int hk, hv, group, dk, dv;
    int64_t ldq, ldk, ldv;
    float scale;
};

// What the preparation leaves for every (slot, value head), one record of `rec` bytes:
// fragments of T diag(beta) (and, for the forward, P; for the backward's second scan, T^T
// and P^T in records of their own), then exp(G) [64], exp(G_last - G) [64], beta [64].
template <bool BF>
struct Rec {
    static constexpr int t = 0;                                        // lower, NS parts
    static constexpr int p = kTri * Io<BF>::NS * kFragBytes;           // lower, NP parts
    static constexpr int sc = p + kTri * Io<BF>::NP * kFragBytes;
    static constexpr int bytes = sc + 1024;
    static constexpr int pt = kTri * Io<BF>::NS * kFragBytes;          // backward: T^T at 0, P^T here
    static constexpr int back = kTri * (Io<BF>::NS + Io<BF>::NE) * kFragBytes;
};
struct Prep {
    unsigned char* rec;   // [slot][value head]
    unsigned char* back;  // [slot][value head] T^T and P^T, upper fragments (backward)
};

// What the backward's scans leave for the chunk-parallel part: per (slot, value head) and
// block of 16 columns, the state (its gradient) as KS, a 64-token array as two operand
// fragments: lane l has column l % 16 of the block, elements 8 (l / 16) .. + 7 of 32. One
// contiguous store of 1 KiB in place of sixteen of 32-byte pieces. bf16 calls keep 24 bits of
// an fp32 value, the upper 16 of a lane's eight in 16 bytes and the rest in 8 behind them: with
// bf16 alone, dk and dg were up to 3e-3 off and dbeta 3.4e-3 (rounding by itself leaves 1.7e-3);
// with a second bf16 part the scans and the gradients of 8 sequences of 8192 tokens, which are
// bound by these bytes, take 1209 us in place of 1100.
template <bool BF, int KS>
struct Kept {
    static constexpr int frag = 512 * (BF ? 3 : 4);  // bytes of a fragment
    static constexpr int state = KS * frag, rows = 2 * frag;
};
// Fragment s of those at p (n of them; nothing is kept where !ok). bf16 calls store without a
// branch: the reverse scan's packing then shares a schedule with the products around it (402 us
// in place of 450). Its fp32 calls, whose registers are all taken, and the forward's keeping
// scan (297 us in place of 310) fare better with one.
template <bool BF>
__device__ __forceinline__ void keep_frag(unsigned char* p, bool ok, int n, int s, int lane, const f32x4& a, const f32x4& b) {
    if constexpr (BF) {
        uint32_t t[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = __float_as_uint(a[i]) + 0x80u;
            t[4 + i] = __float_as_uint(b[i]) + 0x80u;
        }
        u32x4 hi;
        u32x2 lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) hi[i] = __builtin_amdgcn_perm(t[2 * i + 1], t[2 * i], 0x07060302);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            lo[i] = __builtin_amdgcn_perm(t[4 * i + 1], t[4 * i], 0x0c0c0501) | __builtin_amdgcn_perm(t[4 * i + 3], t[4 * i + 2], 0x05010c0c);
        const RowBuf to = plain_buf(p, ok ? n * 1536 : 0);
        __builtin_amdgcn_raw_buffer_store_b128(hi, to, lane * 16, s * 1536, 0);
        __builtin_amdgcn_raw_buffer_store_b64(lo, to, lane * 8, s * 1536 + 1024, 0);
    } else if (ok) {
        *reinterpret_cast<f32x4*>(p + s * 2048 + lane * 32) = a;
        *reinterpret_cast<f32x4*>(p + s * 2048 + lane * 32 + 16) = b;
    }
}
// a lane's part of a kept fragment, on its way and as eight values
template <bool BF>
struct KeptRaw {
    u32x4 a;
    typename std::conditional<BF, u32x2, u32x4>::type b;
    __device__ __forceinline__ void load(RowBuf from, uint32_t frag, int lane) {
        a = __builtin_bit_cast(u32x4, buf_f4(from, frag + lane * (BF ? 16 : 32), 0));
        if constexpr (BF)
            b = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(from, (int)(frag + 1024 + lane * 8), 0, 0));
        else
            b = __builtin_bit_cast(u32x4, buf_f4(from, frag + lane * 32 + 16, 0));
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (BF)
                x[i] = __uint_as_float(__builtin_amdgcn_perm(a[i >> 1], b[i >> 2], (i & 1 ? 0x0706000c : 0x0504000c) | ((i & 3) << 8)));
            else
                x[i] = __uint_as_float(i < 4 ? a[i & 3] : b[i & 3]);
        }
    }
};

constexpr int64_t kMaxTokens = int64_t(1) << 31;
constexpr int64_t kMaxSeqs = int64_t(1) << 24;
constexpr int64_t kMaxLd = int64_t(1) << 22;  // elements: 64 rows stay below 2^31 bytes

// A launch takes fewer than 2^32 threads along an axis.
constexpr bool fits_launch(int64_t blocks, int64_t threads) { return blocks < ((int64_t(1) << 32) + threads - 1) / threads; }
// workgroups a (sequence, value head) of the scans, and their threads
constexpr int scan_columns(bool bf) { return bf ? 32 : 16; }
constexpr int scan_threads(bool bf) { return bf ? 256 : 192; }

constexpr int kCus = 256;
// Shorter pieces gain nothing: the ends' launch and the carries (5 us a piece) cost what the
// shorter scans save. One bf16 sequence, 6 heads of 128, cut and whole: 1600 tokens 58 and
// 62 us, 2048 65 and 76, 4096 95 and 139, 16384 178 and 507; backward 138 and 141, 143 and
// 167, 205 and 294, 504 and 1121.
constexpr int64_t kMinPiece = 8;

struct PrepArgs;
struct ScanArgs;

}  // namespace delta

struct DeltaCall {
    hyena_delta_params_t p;
    hyena_delta_inputs_t in;
    delta::Seqs seqs;
    delta::Shape shape;
    int64_t slots;
    bool bf;
    int dkp;  // dim_k rounded up to 64 or 128
};

// shape alone; and with the sequences and (unless null) the inputs: fills c; and whether the
// launches over whole sequences take that many
hyena_status_t delta_check_shape(const hyena_delta_params_t* p, DeltaCall& c);
hyena_status_t delta_check(const hyena_delta_params_t* p, int64_t N, int64_t tokens, const int64_t* seq_start,
                           const hyena_delta_inputs_t* in, DeltaCall& c);
hyena_status_t delta_check_launches(const DeltaCall& c);
// bytes of the preparation's workspace; pointers from base
size_t delta_prep_layout(const DeltaCall& c, bool bwd, unsigned char* base, delta::Prep& o);
hipError_t delta_prep(const DeltaCall& c, bool bwd, const delta::Prep& o, hipStream_t st);
// how (and whether) the call's long sequences are cut; bytes of the pieces' workspace
delta::Pieces delta_pieces(const DeltaCall& c);
size_t delta_pieces_layout(const DeltaCall& c, bool bwd, unsigned char* base, delta::Pieces& o);
// the state scan: outputs, or (keep) states and written values for the backward; the
// pieces' ends first where sequences are cut
hipError_t delta_scan(const DeltaCall& c, bool keep, const delta::ScanArgs& a, hipStream_t st);

}  // namespace hy
