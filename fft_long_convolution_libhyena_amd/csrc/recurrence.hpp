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
// A workgroup has one chunk and 128 channels: a wave 20 (backward: 10, short forward: 8) tokens, a lane two channels. All
// tokens of a lane are loaded at once and stay in registers from the first pass (which gives
// the wave's A and H) to the second (which gives the outputs).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hyena.h"
#include "plan.hpp"

namespace hy {
namespace rec {

constexpr int kVec = 2;                  // channels a lane
constexpr int kCols = 64 * kVec;         // channels a workgroup
// Tokens of a wave and of a chunk: in bf16 as many as 128 registers hold, which leaves two workgroups a CU (the
// backward holds twice as much of each, exp(-i) in LDS). In fp32 the same spans take 138 and 158 registers, one workgroup a
// CU; twice the bytes are in flight for it (1 x 65536 x 768: 178 us forward, 334 backward, 91% and 85% of a copy's rate by
// inputs and outputs; other spans were measured in bf16 only). Forward of 1 x 65536 x 768 with 8, 12, 16, 18, 20 and 22
// tokens a wave: 134, 112, 107, 104, 102 and 103 us; with 32 in waves at two or three a SIMD 114 and 125. Training step
// of 8 x 8192 with 6, 8 and 10 in the backward: 334, 297 and 285 us (8 without LDS the same, 10 without it spills: 375).
constexpr int kForwardSpan = 20, kBackwardSpan = 10;
// Tokens of a wave in a forward whose chunks then take no more workgroups than there are CUs: less to load and
// to work through before the states pass on, while there are few chunks to pass through. 64, 512 and 2048 tokens
// of 768 channels with 8 and 20: 5.4 and 7.2, 9.8 and 13.5, 12.8 and 14.7 us; 4096 tokens: 18.9 and 17.6.
constexpr int kShortSpan = 8;
constexpr int kShortGrid = 256;
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kBackwardChunk = kWaves * kBackwardSpan;
static_assert(kBackwardChunk == HYENA_RECURRENCE_CARRY, "states kept for the backward");
static_assert(kForwardSpan <= 32 && kForwardSpan <= kBackwardChunk, "bits of a span; one kept state at most in it");
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 256;
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
};

// What a wave's S tokens t0 .. are; lane s finds out about token t0 + s. Bit s of `have`: it is of some
// sequence, of `first`: begins one, of `last`: ends one. Offsets that decrease give other bits, but
// sequences and rows stay in range. Tokens of no sequence lie in front of the first and behind the last
// one, so what they do to states reaches no other token: they take part with the values of some row.
template <int S>
struct Span {
    int t0, mine;  // mine: the sequence of this lane's token
    uint32_t have, first, last;

    __device__ __forceinline__ Span(const Seqs& q, int t0_) : t0(t0_) {
        const int t = t0 + (threadIdx.x & 63);
        const bool in = (threadIdx.x & 63) < S && t < q.tokens;
        mine = in ? q.of(t) : -1;
        const bool some = mine >= 0 && mine < q.N;
        mine = some ? mine : 0;
        const int end = some ? q.at(mine + 1) : 0;
        have = (uint32_t)__ballot(some && t < end);
        first = (uint32_t)__ballot(some && t < end && q.at(mine) == t);
        last = (uint32_t)__ballot(some && t + 1 == end);
    }
    __device__ __forceinline__ bool has(int s) const { return have >> s & 1; }
    __device__ __forceinline__ bool begins(int s) const { return first >> s & 1; }
    __device__ __forceinline__ bool ends(int s) const { return last >> s & 1; }
    __device__ __forceinline__ int sequence(int s) const { return __builtin_amdgcn_readlane(mine, s); }
    // a row of some sequence, from t0 on: token s's, where it has one (not without any)
    __device__ __forceinline__ int row(int s) const { return has(s) ? s : __builtin_ctz(have); }
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

// Rows t0 .. of an array, read and written by buffer instructions: the row is a scalar offset and the
// lane's channels a constant one, so an access costs no vector arithmetic; a lane behind the last channel
// has the offset kNone outside of the range, loads 0 and stores nothing. Stores are marked as not read again soon
// (1 x 65536 x 768: 102 to 98 us, training step of 8 x 8192: 292 to 281; loads so too: 98 and 279, but small calls 2 us longer).
// Unlike the norms' (stream.hpp) this goes for small calls and lines covered in part too: no width from 8 to 2048 channels lost more
// than 1%, and forward and residual norm of its output together take, marked and not, for 4936 tokens of 768 channels 26.4 and
// 26.3 us, 16384 64.6 and 63.8, 32768 101 and 106, 65536 165 and 172.
constexpr int kNone = (int)0x80000000u;
template <bool BF>
struct Rows {
    __amdgpu_buffer_rsrc_t buf;
    int pitch;  // bytes

    // rows: at most 64; 64 * 2^22 * 4 bytes stay below kNone
    __device__ __forceinline__ Rows(const void* base, int64_t ld, int t0, int rows, int dim) {
        pitch = (int)ld * Io<BF>::kBytes;
        buf = __builtin_amdgcn_make_buffer_rsrc((char*)const_cast<void*>(base) + (int64_t)t0 * ld * Io<BF>::kBytes, 0,
                                                rows > 0 ? (rows - 1) * pitch + dim * Io<BF>::kBytes : 0, 0x00020000);
    }
    __device__ __forceinline__ typename Io<BF>::Raw load(int row, int at) const {
        if constexpr (BF)
            return __builtin_amdgcn_raw_buffer_load_b32(buf, at, row * pitch, 0);
        else
            return __builtin_bit_cast(typename Io<BF>::Raw, __builtin_amdgcn_raw_buffer_load_b64(buf, at, row * pitch, 0));
    }
    __device__ __forceinline__ void store(int row, int at, const float (&x)[kVec]) const {
        if constexpr (BF) {
            __builtin_amdgcn_raw_buffer_store_b32(Io<BF>::put(x), buf, at, row * pitch, 2);
        } else {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, Io<BF>::put(x)), buf, at, row * pitch, 2);
        }
    }
};

__device__ __forceinline__ float exp_minus(float x) { return __builtin_amdgcn_exp2f(-kLog2e * x); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp_minus(x)); }
// 1 - sig(x) from e = exp(-x) and sig(x), without the difference, which would cancel where the gate is open;
// 1 where e is infinite and sig(x) 0
__device__ __forceinline__ float one_minus(float e, float sig) { return fminf(e * sig, 1.f); }
// a = exp(-w) and q = 1 - a^2 for w = -log a >= 0. Near a = 1 the error of a counts once for every
// token that a state outlives, and 1 - a^2 cancels: below w = 1/2 a comes from e = 1 - exp(-w) as
// w times a polynomial (a fit of degree 5 at Chebyshev points, 5e-9 off) with half a step of error and no
// bias, and q = e (1 + a) keeps e's digits. (With the exponential instruction, a step off to one
// side, states of 2000 tokens with a around 0.999 were 2.7e-6 off in place of 5e-7.)
// least: added to e, so that q is not 0. near (of the wave): all w are known to be below 1/2, as rates below
// 1/2 make them.
__device__ __forceinline__ void decay(const float (&w)[kVec], bool near, float (&a)[kVec], float (&q)[kVec], float least = 0.f) {
    float e[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        float p = fmaf(w[j], -0.0011237150756642222f, 0.008190003223717213f);
        p = fmaf(w[j], p, -0.04163024201989174f);
        p = fmaf(w[j], p, 0.16666245460510254f);
        p = fmaf(w[j], p, -0.4999998211860657f);
        p = fmaf(w[j], p, 1.f);
        e[j] = fmaf(w[j], p, least);
        a[j] = 1.f - e[j];
    }
    if (!near)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const float far = __builtin_amdgcn_exp2f(-kLog2e * w[j]);
            a[j] = w[j] < 0.5f ? a[j] : far;
            e[j] = w[j] < 0.5f ? e[j] : 1.f - far;
        }
#pragma unroll
    for (int j = 0; j < kVec; ++j) q[j] = fmaf(e[j], a[j], e[j]);
}
// A of a run of tokens, from the sum of their w. (Their product loses a little at every token, always to the same
// side: 1 - k 2^-24 times A = 1 - d is A - k 2^-24 + k d 2^-24, and the last term is rounded away while k d < 1/2. With it
// states and gradients of 20001 tokens at rates of 1e-4 were 3e-5 to 7e-5 off, of 9001 at 1e-5 .. 1e-2 up to 3e-5; now
// 3e-7 to 4e-7, for at most 1% of the time.)
__device__ __forceinline__ void run_decay(const float (&w)[kVec], float (&A)[kVec]) {
    float q[kVec];
    decay(w, false, A, q);
}
__device__ __forceinline__ bool near_rates(const float (&rate)[kVec]) { return __all(rate[0] < 0.5f && rate[1] < 0.5f); }

// ------------------------------------------------------------------ states between chunks

// Chunks pass their states on inside one launch. Workgroups take chunks in the order of a
// ticket; each publishes its (A, H) as soon as it has its own tokens, and only then waits for
// those in front of it. What it waits for belongs to lower tickets, which have been drawn by workgroups that
// run, so every wait ends; a bound on the polls ends it whatever a caller does to the workspace
// (states are NaN then). A word of 64 bits holds both values of a channel and that they are
// there, so no fences are needed: 0 until then, with bit 63 set (A >= 0), and A = 2 for a
// chunk in which a sequence begins (its H is a state). The last of every 16 chunks publishes, as such
// a word, the state behind it; so a chunk folds at most 16 words, always in the same order, and states run
// through long sequences at a hop for 16 chunks. A wave polls its share of them at once; the words of
// even and of odd channels lie apart, so that it reads whole lines.
constexpr int kGroup = 16;
constexpr int kPolls = 1 << 22;  // some seconds

using Word = unsigned long long;
constexpr uint32_t kResetWord = 0xc0000000u;  // the high half: A = -2

// (A, H) of a lane's two channels
typedef float Link __attribute__((ext_vector_type(4)));  // A, A, H, H
__device__ __forceinline__ void join_link(bool reset, const Link& v, float (&h)[kVec]) {
    h[0] = reset ? v[2] : fmaf(v[0], h[0], v[2]);
    h[1] = reset ? v[3] : fmaf(v[1], h[1], v[3]);
}
// bit k: flag k of the workgroup's waves is set
__device__ __forceinline__ uint32_t flag_bits(const int (&flags)[kWaves], int lane) {
    return (uint32_t)__ballot(lane < kWaves && flags[lane & (kWaves - 1)] != 0);
}
// h through the links of waves k, k + step, ... n of them; mostly no sequence begins in any
template <class F>
__device__ __forceinline__ void join_links(uint32_t resets, int k, int step, int n, F link, float (&h)[kVec]) {
    if (!resets) {
#pragma unroll 2
        for (; n > 0; --n, k += step) {
            const Link v = link(k);
            h[0] = fmaf(v[0], h[0], v[2]);
            h[1] = fmaf(v[1], h[1], v[3]);
        }
    } else {
#pragma unroll 1
        for (; n > 0; --n, k += step) join_link(resets >> k & 1, link(k), h);
    }
}

__device__ __forceinline__ void publish(Word* words, int order, int dim, int col, bool reset, const float (&A)[kVec],
                                        const float (&H)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const float a = A[j] == A[j] ? A[j] : 0.f;  // H is NaN where A is
        const uint32_t hi = reset ? kResetWord : __float_as_uint(a) | 0x80000000u;
        __hip_atomic_store(words + (int64_t)order * dim + (uint32_t)(j * (dim / 2) + col / 2),
                           (Word)hi << 32 | __float_as_uint(H[j]), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// This wave's words: kPolled of them from kPolled * wave on, of those in front of chunk `order` in its group, the first of which is the
// last of the group before. ask() sends for them, done() waits for all, gives (A, H) of the run and
// returns whether a sequence begins in it.
struct LookBack {
    static constexpr int kPolled = kGroup / kWaves;
    const Word* words;
    int base, order, dim, col;
    Word v[kPolled][kVec];

    __device__ __forceinline__ LookBack(const Word* words_, int order_, int dim_, int col_, int wave)
        : words(words_), base((order_ & ~(kGroup - 1)) - 1 + kPolled * wave), order(order_), dim(dim_), col(col_) {}
    __device__ __forceinline__ void ask() {
#pragma unroll
        for (int k = 0; k < kPolled; ++k) {
            const int at = base + k;
            if (at >= 0 && at < order) {
                const Word* p = words + (int64_t)at * dim;
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    v[k][j] = __hip_atomic_load(p + (uint32_t)(j * (dim / 2) + col / 2), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[k][j] = (Word)0xbf800000u << 32;  // (1, 0): nothing happens
            }
        }
    }
    __device__ __forceinline__ bool done(Link& link) {
        for (int polls = 0;; ++polls) {
            Word there = ~(Word)0;
#pragma unroll
            for (int k = 0; k < kPolled; ++k)
#pragma unroll
                for (int j = 0; j < kVec; ++j) there &= v[k][j];
            if (__all((int)(there >> 63))) break;
            if (polls >= kPolls) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[kPolled - 1][j] = (Word)kResetWord << 32 | 0x7fc00000u;
                break;
            }
            __builtin_amdgcn_s_sleep(1);
            ask();
        }
        bool any = false;
        link = Link{1.f, 1.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < kPolled; ++k) {
            // the same for all channels
            const bool reset = __builtin_amdgcn_readfirstlane((int)(v[k][0] >> 32)) == (int)kResetWord;
            any |= reset;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float a = fabsf(__uint_as_float((uint32_t)(v[k][j] >> 32))), h = __uint_as_float((uint32_t)v[k][j]);
                link[2 + j] = reset ? h : fmaf(a, link[2 + j], h);
                link[j] *= a;
            }
        }
        return any;
    }
};

// ------------------------------------------------------------------ host side

struct Call {
    hyena_recurrence_params_t p;
    hyena_recurrence_inputs_t in;
    Seqs seqs;
    bool bf;
    int span;                             // tokens of a wave in the forward
    int64_t chunks, back_chunks, blocks;  // chunks of tokens (forward, backward), blocks of channels
};

// whole: of whole sequences, whose strides and grids of chunks are bounded; the step's are its own
hyena_status_t check(const hyena_recurrence_params_t* p, int64_t N, int64_t tokens, const int64_t* seq_start,
                     const hyena_recurrence_inputs_t* in, Call& c, bool whole = true);
// 64-bit values at the head of a workspace that start() clears: the tickets of up to two launches, then the words
constexpr int kHead = 2;
inline int64_t word_count(const Call& c, int64_t chunks) { return chunks > 1 ? chunks * c.p.dim : 0; }
// Words of the forward that cover this call and every one of fewer tokens or channels: a short span's chunks are
// many, but take at most kShortGrid workgroups
inline int64_t covering_words(const Call& c) {
    const int64_t own = word_count(c, c.chunks), brief = word_count(c, (c.seqs.tokens + kWaves * kShortSpan - 1) / (kWaves * kShortSpan));
    const int64_t most = brief < kShortGrid * kCols ? brief : kShortGrid * kCols;
    return own > most ? own : most;
}
// Clears `n` values of 64 bits, passes the states of sequences without tokens on and clears the rows of no sequence
// in `outs` (each may be null); no launch where there is nothing of it to do.
struct Outs {
    void* p[3];
};
hipError_t start(const Call& c, void* clear, int64_t n, const float* from, float* to, Outs outs, hipStream_t st);
// y, state_out and carry may each be null
hipError_t forward(const Call& c, const float* state_in, void* y, float* state_out, float* carry, uint32_t* ticket,
                   Word* words, hipStream_t st);

}  // namespace rec
}  // namespace hy
