// Gated linear recurrence: what its forward, backward and step share.
//
// Per sequence and channel, with the pre-activations r and i and the channel's rate c > 0:
//   log a = -c sig(r),   h <- a h + m sig(i) x,   m = sqrt(1 - a^2),   y = h.
// A run of tokens acts on the state as h -> A h + H (A the product of its a, H what it
// gives from zero), and runs join: (A2, H2) after (A1, H1) is (A2 A1, A2 H1 + H2). So the
// tokens, all sequences behind each other, are cut into chunks, whose (A, H) need
// only their own tokens; the states in front of the chunks follow from these. A token that
// begins a sequence takes its initial state in and lets nothing of what lies in front through
// (not as a factor 0: an infinity there must not become NaN here).
//
// A workgroup has one chunk and 128 channels: a wave 16 (backward: 8) tokens, a lane two channels. All
// tokens of a lane are loaded at once and stay in registers from the first pass (which gives
// the wave's A and H) to the second (which gives the outputs).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hyena.h"
#include "plan.hpp"

namespace hy {
namespace rec {

constexpr int kWaves = 8;                // of a workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kVec = 2;                  // channels a lane
constexpr int kCols = 64 * kVec;         // channels a workgroup
// Tokens a wave, forward and backward (which holds twice as much of each)
constexpr int kForwardSpan = 16, kBackwardSpan = 8;
constexpr int kForwardChunk = kWaves * kForwardSpan, kBackwardChunk = kWaves * kBackwardSpan;
static_assert(kBackwardChunk == HYENA_RECURRENCE_CARRY && kForwardChunk % kBackwardChunk == 0, "states kept for the backward");
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - kForwardChunk;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ sequences

// Sequences in the packed tokens: starts from memory, or every T tokens.
struct Seqs {
    const int64_t* start;  // [N + 1] or null
    int32_t N, tokens, T;

    __device__ __forceinline__ int at(int n) const {  // clamped to the tokens
        if (!start) return n * T;                     // n <= N: at most tokens
        const int64_t s = start[n];
        return s < 0 ? 0 : s > tokens ? tokens : (int)s;
    }
    // the last sequence that starts at or in front of t (-1: none)
    __device__ __forceinline__ int of(int t) const {
        if (!start) return (int)((uint32_t)t / (uint32_t)T);
        int lo = 0, hi = N;  // the answer + 1 lies in [lo, hi]
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (at(mid) <= t)
                lo = mid + 1;
            else
                hi = mid;
        }
        return lo - 1;
    }
    __device__ __forceinline__ int begin() const { return start ? at(0) : 0; }
    __device__ __forceinline__ int end() const { return start ? at(N) : tokens; }
};

// What a wave's S tokens t0 .. are: those of some sequence are [lo, hi); bit s of `first`:
// token t0 + s begins a sequence, of `last`: ends one.
template <int S>
struct Span {
    int t0, lo, hi;
    uint32_t first, last;

    __device__ __forceinline__ Span(const Seqs& q, int t) : t0(t), first(0), last(0) {
        const int b = q.begin(), e = q.end();
        lo = b > t0 ? b : t0;
        hi = e < t0 + S ? e : t0 + S;
        if (lo >= hi) {
            lo = hi = t0;
            return;
        }
        uint32_t starts = 0;  // of tokens t0 .. t0 + S
        for (int n = q.of(lo); n <= q.N; ++n) {
            const int s = q.at(n < 0 ? 0 : n);
            if (s > t0 + S) break;
            if (s >= t0) starts |= 1u << (s - t0);
        }
        first = starts & ((1u << S) - 1);
        last = starts >> 1;
        if (hi == e) last |= 1u << (hi - 1 - t0);
        // offsets that decrease may name tokens outside [lo, hi)
        const uint32_t mine = ((1u << (hi - t0)) - 1) & ~((1u << (lo - t0)) - 1);
        first &= mine;
        last &= mine;
    }
    __device__ __forceinline__ bool has(int k) const { return t0 + k >= lo && t0 + k < hi; }
    __device__ __forceinline__ int row(int k) const {  // a row that may be read
        const int t = t0 + k;
        return t < lo ? lo : t >= hi ? hi - 1 : t;
    }
};

// ------------------------------------------------------------------ values

template <bool BF>
struct Io;
template <>
struct Io<true> {
    using Raw = uint32_t;  // two bf16
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ void get(Raw w, float (&x)[kVec]) {
        x[0] = __uint_as_float(w << 16);
        x[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw put(const float (&x)[kVec]) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x[0], x[1]}), bf16x2));
    }
};
template <>
struct Io<false> {
    typedef float Raw __attribute__((ext_vector_type(2)));
    static constexpr int kBytes = 4;
    static __device__ __forceinline__ void get(Raw w, float (&x)[kVec]) {
        x[0] = w[0];
        x[1] = w[1];
    }
    static __device__ __forceinline__ Raw put(const float (&x)[kVec]) { return Raw{x[0], x[1]}; }
};

template <bool BF>
__device__ __forceinline__ typename Io<BF>::Raw load_row(const void* base, int64_t ld, int row, int col) {
    const char* p = (const char*)base + (int64_t)row * ld * Io<BF>::kBytes;
    return *reinterpret_cast<const typename Io<BF>::Raw*>(p + (uint32_t)(col * Io<BF>::kBytes));
}
template <bool BF>
__device__ __forceinline__ void store_row(void* base, int64_t ld, int row, int col, const float (&x)[kVec]) {
    char* p = (char*)base + (int64_t)row * ld * Io<BF>::kBytes;
    *reinterpret_cast<typename Io<BF>::Raw*>(p + (uint32_t)(col * Io<BF>::kBytes)) = Io<BF>::put(x);
}

__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}
// a = exp(-w) and q = 1 - a^2 for w = -log a >= 0. Near a = 1 the error of a counts once for every
// token that a state outlives, and 1 - a^2 cancels: below w = 1/2 a comes from e = 1 - exp(-w) as
// w times a polynomial (a fit of degree 5 at Chebyshev points, 5e-9 off) with half a step of error and no
// bias, and q = e (1 + a) keeps e's digits. (With the exponential instruction, a step off to one
// side, states of 2000 tokens with a around 0.999 were 2.7e-6 off in place of 5e-7.)
__device__ __forceinline__ void decay(float w, float& a, float& q) {
    float p = fmaf(w, -0.0011237150756642222f, 0.008190003223717213f);
    p = fmaf(w, p, -0.04163024201989174f);
    p = fmaf(w, p, 0.16666245460510254f);
    p = fmaf(w, p, -0.4999998211860657f);
    p = fmaf(w, p, 1.f);
    const float far = __builtin_amdgcn_exp2f(-kLog2e * w);
    const bool near = w < 0.5f;
    const float e = near ? w * p : 1.f - far;
    a = near ? 1.f - e : far;
    q = fmaf(e, a, e);
}
__device__ __forceinline__ void gate(float x, float r, float i, float rate, float& a, float& b) {
    float q;
    decay(rate * sigmoid(r), a, q);
    b = __builtin_amdgcn_sqrtf(q) * sigmoid(i) * x;
}

// ------------------------------------------------------------------ states between chunks

// Chunks pass their states on inside one launch. Workgroups take chunks in the order of a
// ticket; each publishes its (A, H) as soon as it has its own tokens, and only then waits for
// those in front of it. What it waits for belongs to lower tickets, which have been drawn by workgroups that
// run, so every wait ends; a bound on the polls ends it whatever a caller does to the workspace
// (states are NaN then). A word of 64 bits holds both values of a channel and that they are
// there, so no fences are needed: 0 until then, with bit 63 set (A >= 0), and A = 2 for a
// chunk in which a sequence begins (its H is a state). The last of every 32 chunks publishes, as such
// a word, the state behind it; so a chunk folds at most 32 words, always in the same order, and states run
// through long sequences at a hop for 32 chunks. A wave polls four words at once.
constexpr int kGroup = 32;
constexpr int kPolls = 1 << 20;  // about a second
constexpr float kReset = 2.f;
static_assert(kGroup == 4 * kWaves, "four words a wave");

using Word = unsigned long long;
__device__ __forceinline__ Word make_word(float A, float H) {
    A = A == A ? A : 0.f;  // H is NaN where A is
    return (Word)(__float_as_uint(A) | 0x80000000u) << 32 | __float_as_uint(H);
}
__device__ __forceinline__ void join_word(float A, float H, float& h) { h = A == kReset ? H : fmaf(A, h, H); }

__device__ __forceinline__ void publish(Word* words, int order, int dim, int col, const float (&A)[kVec], const float (&H)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        __hip_atomic_store(words + (int64_t)order * dim + col + j, make_word(A[j], H[j]), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
}

// (A, H) of this wave's words: 4 wave .. of those in front of chunk `order` in its group, the first of
// which is the last of the group before
__device__ __forceinline__ void look_back(const Word* words, int order, int dim, int col, int wave, float (&A)[kVec],
                                          float (&H)[kVec]) {
    const int base = (order & ~(kGroup - 1)) - 1;
    Word v[4][kVec];
    for (int polls = 0;; ++polls) {
        Word there = ~(Word)0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int at = base + 4 * wave + k;
            const bool need = at >= 0 && at < order;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                v[k][j] = (Word)0xbf800000u << 32;  // (1, 0): nothing happens
                if (need) v[k][j] = __hip_atomic_load(words + (int64_t)at * dim + col + j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                there &= v[k][j];
            }
        }
        if (__all((int)(there >> 63))) break;
        if (polls >= kPolls) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[3][j] = make_word(kReset, __uint_as_float(0x7fc00000u));
            break;
        }
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        A[j] = 1.f;
        H[j] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float a = __uint_as_float((uint32_t)(v[k][j] >> 32) & 0x7fffffffu), h = __uint_as_float((uint32_t)v[k][j]);
            join_word(a, h, H[j]);
            A[j] = a == kReset || A[j] == kReset ? kReset : A[j] * a;
        }
    }
}

// ------------------------------------------------------------------ host side

struct Call {
    hyena_recurrence_params_t p;
    hyena_recurrence_inputs_t in;
    Seqs seqs;
    bool bf;
    int64_t chunks, back_chunks, blocks;  // chunks of tokens (forward, backward), blocks of channels
};

hyena_status_t check(const hyena_recurrence_params_t* p, int64_t N, int64_t tokens, const int64_t* seq_start,
                     const hyena_recurrence_inputs_t* in, Call& c);
// 64-bit values at the head of a workspace that start() clears: the tickets of up to two launches, then the words
constexpr int kHead = 2;
inline int64_t word_count(const Call& c, int64_t chunks) { return chunks > 1 ? chunks * c.p.dim : 0; }
// Clears `n` values of 64 bits and passes the states of sequences without tokens on; no launch without either.
hipError_t start(const Call& c, void* clear, int64_t n, const float* from, float* to, hipStream_t st);
// y, state_out and carry may each be null
hipError_t forward(const Call& c, const float* state_in, void* y, float* state_out, float* carry, uint32_t* ticket,
                   Word* words, hipStream_t st);

}  // namespace rec
}  // namespace hy
