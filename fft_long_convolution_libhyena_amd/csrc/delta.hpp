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
// bf16 plans give their inputs exactly in one part and carry the state, T and the
// written values in two (relative error of the fp32 state measured 3e-6; one part
// would leave 2e-3); fp32 plans use three parts throughout (1e-7), at 6 products for
// each single one, still 2.7 times the rate of the fp32 matrix instruction.
//
// Fragment layouts of v_mfma_f32_16x16x32_bf16, lane l, g = l / 16:
//   A [16][32]: lane holds row l % 16, columns 8g .. 8g+7
//   B [32][16]: lane holds column l % 16, rows 8g .. 8g+7
//   D [16][16]: lane holds column l % 16, rows 4g .. 4g+3
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

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
    static constexpr int NO = 2;  // parts of the state and of u against Q and P
    static constexpr int NP = 1;  // parts of P
};
template <>
struct Io<false> {
    using T = float;
    static constexpr int NI = 3;
    static constexpr int NS = 3;
    static constexpr int NO = 3;
    static constexpr int NP = 3;
};

template <int N>
struct Frag {
    bf16x8 p[N];
};

template <int N>
__device__ __forceinline__ Frag<N> split8(const float (&x)[8]) {
    Frag<N> f;
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __bf16 h = (__bf16)r[i];
            f.p[n][i] = h;
            if (n + 1 < N) r[i] -= (float)h;
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

// the same for J right-hand operands, products of one part pair next to each other so
// that consecutive instructions do not wait for each other's sums
template <int NA, int NB, int J>
__device__ __forceinline__ void mma_each(const Frag<NA>& a, const Frag<NB> (&b)[J], f32x4 (&c)[J]) {
    constexpr int M = NA > NB ? NA : NB;
#pragma unroll
    for (int s = M - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int k = s - i;
            if (k >= 0 && k < NB)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    c[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b[j].p[k], c[j], 0, 0, 0);
        }
}
template <int N, int M>
__device__ __forceinline__ Frag<N> first_parts(const Frag<M>& f) {
    Frag<N> r;
#pragma unroll
    for (int n = 0; n < N; ++n) r.p[n] = f.p[n];
    return r;
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
__device__ __forceinline__ Raw16 load_raw(const __bf16* p, bool ok) {
    Raw16 r = {};
    if (ok) r.v = *reinterpret_cast<const bf16x8*>(p);
    return r;
}
__device__ __forceinline__ Raw32 load_raw(const float* p, bool ok) {
    Raw32 r = {};
    if (ok) {
        r.lo = *reinterpret_cast<const f32x4*>(p);
        r.hi = *reinterpret_cast<const f32x4*>(p + 4);
    }
    return r;
}
__device__ __forceinline__ Frag<1> to_frag(const Raw16& r) { return Frag<1>{{r.v}}; }
__device__ __forceinline__ Frag<3> to_frag(const Raw32& r) {
    const float x[8] = {r.lo[0], r.lo[1], r.lo[2], r.lo[3], r.hi[0], r.hi[1], r.hi[2], r.hi[3]};
    return split8<3>(x);
}
template <bool BF>
using Raw = decltype(load_raw((const typename Io<BF>::T*)nullptr, true));

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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void buf_raw(RowBuf b, uint32_t off, Raw16& r) {
    r.v = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
}
__device__ __forceinline__ void buf_raw(RowBuf b, uint32_t off, Raw32& r) {
    r.lo = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
    r.hi = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off + 16, 0, 0));
}
// N (1 or 2) consecutive elements: raw registers, their values, and back
template <bool BF, int N>
struct Cols {
    uint32_t w[BF ? 1 : N];
};
template <bool BF, int N>
__device__ __forceinline__ void buf_cols(RowBuf b, uint32_t off, Cols<BF, N>& c) {
    if constexpr (BF && N == 1)
        c.w[0] = __builtin_amdgcn_raw_buffer_load_b16(b, (int)off, 0, 0);
    else if constexpr (!BF && N == 2) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(b, (int)off, 0, 0));
        c.w[0] = v[0];
        c.w[1] = v[1];
    } else
        c.w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, (int)off, 0, 0);
}
template <bool BF, int N>
__device__ __forceinline__ float col_value(const Cols<BF, N>& c, int j) {
    if constexpr (BF) return __uint_as_float(j == 0 ? c.w[0] << 16 : c.w[0] & 0xffff0000u);
    return __uint_as_float(c.w[BF ? 0 : j]);
}
template <bool BF, int N>
__device__ __forceinline__ void buf_store(RowBuf b, uint32_t off, const float (&x)[N]) {
    if constexpr (BF) {
        typedef __bf16 bf16xn __attribute__((ext_vector_type(N)));
        bf16xn v;
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = (__bf16)x[j];
        if constexpr (N == 2)
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), b, (int)off, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, v), b, (int)off, 0, 0);
    } else if constexpr (N == 2) {
        const u32x2 v = {__float_as_uint(x[0]), __float_as_uint(x[1])};
        __builtin_amdgcn_raw_buffer_store_b64(v, b, (int)off, 0, 0);
    } else {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[0]), b, (int)off, 0, 0);
    }
}
__device__ __forceinline__ int64_t uniform64(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)x);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)x >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// N (1 or 2) consecutive elements
template <int N>
__device__ __forceinline__ void load_cols(const __bf16* p, bool ok, float (&x)[N]) {
    if constexpr (N == 2) {
        uint32_t v = 0;
        if (ok) v = *reinterpret_cast<const uint32_t*>(p);
        x[0] = __uint_as_float(v << 16);
        x[1] = __uint_as_float(v & 0xffff0000u);
    } else {
        x[0] = ok ? (float)p[0] : 0.f;
    }
}
template <int N>
__device__ __forceinline__ void load_cols(const float* p, bool ok, float (&x)[N]) {
    if constexpr (N == 2) {
        float2 v = make_float2(0.f, 0.f);
        if (ok) v = *reinterpret_cast<const float2*>(p);
        x[0] = v.x;
        x[1] = v.y;
    } else {
        x[0] = ok ? p[0] : 0.f;
    }
}
template <int N>
__device__ __forceinline__ void store_cols(__bf16* p, const float (&x)[N]) {
    if constexpr (N == 2) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        bf16x2 v = {(__bf16)x[0], (__bf16)x[1]};
        *reinterpret_cast<bf16x2*>(p) = v;
    } else {
        p[0] = (__bf16)x[0];
    }
}
template <int N>
__device__ __forceinline__ void store_cols(float* p, const float (&x)[N]) {
    if constexpr (N == 2)
        *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
    else
        p[0] = x[0];
}

// Four values of a D tile (rows 4g..4g+3 of 16-row tile `half` of a 32-row block)
// into part n of the block's B fragment.
template <int N>
__device__ __forceinline__ void put_rows(__bf16* frag, int part_stride, int half, int lane, const float (&x)[4]) {
    const int g = lane >> 4, col = lane & 15;
    __bf16* p = frag + ((2 * half + (g >> 1)) * 16 + col) * 8 + (g & 1) * 4;
    float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int n = 0; n < N; ++n) {
        bf16x4 h;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = (__bf16)r[i];
            if (n + 1 < N) r[i] -= (float)h[i];
        }
        *reinterpret_cast<bf16x4*>(p + n * part_stride) = h;
    }
}
template <int N>
__device__ __forceinline__ Frag<N> get_frag(const __bf16* frag, int part_stride, int lane) {
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) f.p[n] = *reinterpret_cast<const bf16x8*>(frag + n * part_stride + lane * 8);
    return f;
}

// LDS traffic of the workgroup is complete and every wave is here; loads from
// global memory stay in flight (a __syncthreads would wait for them).
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// fragment number of block (row tile i, 32-column step s) of a lower / upper
// block-triangular operand
__device__ __forceinline__ constexpr int lower_frag(int i, int s) { return i < 2 ? i : 2 + (i - 2) * 2 + s; }
__device__ __forceinline__ constexpr int upper_frag(int i, int s) { return i < 2 ? 2 * i + s : 2 + i; }

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

struct Shape {
    int hk, hv, group, dk, dv;
    int64_t ldq, ldk, ldv;
    float scale;
};

// Workspace of the chunk-parallel part, per (slot, value head) unless noted.
struct Prep {
    __bf16* t;    // T, lower fragments, NS parts
    __bf16* p;    // P, lower fragments (forward)
    __bf16* tt;   // T^T and P^T, upper fragments, NS parts (backward)
    __bf16* pt;
    void* kt;     // K^T fragments per (slot, key head): dk/16 row tiles x 2 steps
    void* qt;     // Q^T likewise (backward)
    float* sc;    // exp(G) [64], exp(G_last - G) [64], beta [64]
};

constexpr int64_t kMaxTokens = int64_t(1) << 31;
constexpr int64_t kMaxSeqs = int64_t(1) << 24;
constexpr int64_t kMaxLd = int64_t(1) << 22;  // elements: 64 rows stay below 2^31 bytes

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

// shape alone; and with the sequences and (unless null) the inputs: fills c
hyena_status_t delta_check_shape(const hyena_delta_params_t* p, DeltaCall& c);
hyena_status_t delta_check(const hyena_delta_params_t* p, int64_t N, int64_t tokens, const int64_t* seq_start,
                           const hyena_delta_inputs_t* in, DeltaCall& c);
// bytes of the preparation's workspace; pointers from base
size_t delta_prep_layout(const DeltaCall& c, bool bwd, unsigned char* base, delta::Prep& o);
hipError_t delta_prep(const DeltaCall& c, bool bwd, const delta::Prep& o, hipStream_t st);
// the state scan: outputs, or (keep) states and written values for the backward
hipError_t delta_scan(const DeltaCall& c, bool keep, const delta::ScanArgs& a, hipStream_t st);

}  // namespace hy
