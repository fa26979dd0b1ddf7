// Gated linear recurrence over whole sequences, forward (see recurrence.hpp).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "recurrence.hpp"

namespace hy {
namespace rec {
namespace {

struct ForwardArgs {
    Seqs seqs;
    hyena_recurrence_inputs_t in;
    const float *rate, *state_in;
    void* y;
    float *state_out, *carry;  // or null
    uint32_t* ticket;
    Word* words;               // [chunks][dim]; null: one chunk
    int dim, chunks, blocks;
};

// One chunk and 128 channels, S tokens a wave. 1 x 65536 x 768 in bf16 take 98 us, the start among them: 425 MB with words
// and kept states, at 4.3 TB/s (in fp32 178 us, 828 MB, 4.7); vector work fills half of the cycles. Without the look-back bf16
// would take 78: words are read past the caches, and chunks wait for others that started at about the same time.
template <bool BF, int S>
__global__ __launch_bounds__(kThreads, BF ? 4 : 2) void k_rec_forward(ForwardArgs p) {
    using Raw = typename Io<BF>::Raw;
    constexpr int W = kWaves;
    __shared__ Link sOwn[W][64], sBack[W][64];
    __shared__ float2 sSum[W][64];  // of the waves' w
    __shared__ int sOwnReset[W], sBackReset[W];
    __shared__ uint32_t sTicket;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ticket = blockIdx.x;
    if (p.words) {
        if (threadIdx.x == 0) sTicket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        ticket = __builtin_amdgcn_readfirstlane(sTicket);
    }
    const int chunk = (uint32_t)ticket / (uint32_t)p.blocks;
    if ((uint32_t)chunk >= (uint32_t)p.chunks) return;  // only where a caller's workspace is not this call's alone
    const int own = (ticket - chunk * p.blocks) * kCols + kVec * lane;
    const bool ok = own < p.dim;
    const int col = ok ? own : p.dim - kVec, at = ok ? own * Io<BF>::kBytes : kNone;
    const Span<S> span(p.seqs, chunk * (W * S) + wave * S);
    const int rows = p.seqs.tokens - span.t0 < S ? p.seqs.tokens - span.t0 : S;
    float a[S][kVec], b[S][kVec];
    float w_sum[kVec] = {}, A[kVec] = {1.f, 1.f}, H[kVec] = {};
    if (span.have) {
        Raw x[S], r[S], i[S];
        const Rows<BF> xs(p.in.x, p.in.ldx, span.t0, rows, p.dim), rs(p.in.r, p.in.ldr, span.t0, rows, p.dim),
            is(p.in.i, p.in.ldi, span.t0, rows, p.dim);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int row = span.row(s);
            r[s] = rs.load(row, at);
            i[s] = is.load(row, at);
            x[s] = xs.load(row, at);
        }
        float rate[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) rate[j] = p.rate[col + j];
        const bool near = near_rates(rate);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float xv[kVec], rv[kVec], iv[kVec], w[kVec], q[kVec];
            Io<BF>::get(x[s], xv);
            Io<BF>::get(r[s], rv);
            Io<BF>::get(i[s], iv);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                w[j] = rate[j] * sigmoid(rv[j]);
                w_sum[j] += w[j];
            }
            asm volatile("" : "+v"(w_sum[0]), "+v"(w_sum[1]));  // added here, or all w are kept for later and 8 values spill
            decay(w, near, a[s], q);
#pragma unroll
            for (int j = 0; j < kVec; ++j) b[s][j] = __builtin_amdgcn_sqrtf(q[j]) * sigmoid(iv[j]) * xv[j];
            if (span.begins(s)) {  // from the sequence's initial state, and from nothing in front of it
                const int64_t n = span.sequence(s);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    if (p.state_in) b[s][j] = fmaf(a[s][j], p.state_in[n * p.dim + col + j], b[s][j]);
                    H[j] = 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) H[j] = fmaf(a[s][j], H[j], b[s][j]);
        }
        run_decay(w_sum, A);
    }
    sOwn[wave][lane] = Link{A[0], A[1], H[0], H[1]};
    sSum[wave][lane] = float2{w_sum[0], w_sum[1]};
    if (lane == 0) sOwnReset[wave] = span.first != 0;
    __syncthreads();
    const uint32_t resets = flag_bits(sOwnReset, lane);
    float h[kVec] = {};
    if (p.words) {
        const bool publishes = wave == 0 && chunk + 1 < p.chunks, ends = (chunk & (kGroup - 1)) == kGroup - 1;
        float cw[kVec] = {}, cA[kVec] = {1.f, 1.f}, cH[kVec] = {};
        bool reset = false;
        if (publishes) {
            reset = resets != 0;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const Link v = sOwn[k][lane];
                const float2 u = sSum[k][lane];
                join_link(resets >> k & 1, v, cH);
                cw[0] += u.x;
                cw[1] += u.y;
            }
            run_decay(cw, cA);
            if (!ends && ok) publish(p.words, chunk, p.dim, own, reset, cA, cH);
        }
        if (chunk) {
            Link back;
            LookBack look(p.words, chunk, p.dim, col, wave);
            look.ask();
            const bool rs = look.done(back);
            sBack[wave][lane] = back;
            if (lane == 0) sBackReset[wave] = rs;
            __syncthreads();
            join_links(flag_bits(sBackReset, lane), 0, 1, W, [&](int k) { return sBack[k][lane]; }, h);
        }
        if (publishes && ends) {
            float e[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) e[j] = reset ? cH[j] : fmaf(cA[j], h[j], cH[j]);
            if (ok) publish(p.words, chunk, p.dim, own, true, e, e);
        }
    }
    join_links(resets, 0, 1, wave, [&](int k) { return sOwn[k][lane]; }, h);
    if (!span.have) return;
    // the state in front of one of these tokens may be one that the backward asks for
    const int kept = p.carry ? (kBackwardChunk - span.t0 % kBackwardChunk) % kBackwardChunk : S;
    const Rows<BF> ys(p.y, p.dim, span.t0, rows, p.dim);
    const uint32_t wanted = p.y ? span.have : 0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (s == kept && s < rows && ok)
#pragma unroll
            for (int j = 0; j < kVec; ++j) p.carry[(int64_t)((span.t0 + s) / kBackwardChunk) * p.dim + own + j] = h[j];
        if (span.begins(s)) h[0] = h[1] = 0.f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[j] = fmaf(a[s][j], h[j], b[s][j]);
        if (wanted >> s & 1) ys.store(s, at, h);
        if (span.ends(s) && p.state_out && ok) {
            const int64_t n = span.sequence(s);
#pragma unroll
            for (int j = 0; j < kVec; ++j) p.state_out[n * p.dim + own + j] = h[j];
        }
    }
}

// Clears what the chunks' words and tickets lie in (n words, 16 bytes a thread and round), and rows of no sequence;
// a sequence without tokens passes its state on.
__global__ __launch_bounds__(256) void k_rec_start(Word* clear, int64_t n, Seqs q, const float* from, float* to, int dim, Outs outs,
                                                   int row_bytes) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t e = first; 2 * e < n; e += step) __builtin_nontemporal_store(u32x4{}, reinterpret_cast<u32x4*>(clear) + e);
    if (to)
        for (int s = blockIdx.x; s < q.N; s += gridDim.x) {
            if (q.at(s + 1) > q.at(s)) continue;
            for (int c = threadIdx.x; c < dim; c += 256) {
                const int64_t e = (int64_t)s * dim + c;
                to[e] = from ? from[e] : 0.f;
            }
        }
    if (row_bytes) {  // a multiple of 16
        const int64_t lo = q.at(0), end = q.at(q.N), hi = end > lo ? end : lo, per = row_bytes / 16;
        for (int k = 0; k < 3; ++k) {
            u32x4* const p = reinterpret_cast<u32x4*>(outs.p[k]);
            if (!p) continue;
            for (int64_t e = first; e < lo * per; e += step) p[e] = u32x4{};
            for (int64_t e = hi * per + first; e < q.tokens * per; e += step) p[e] = u32x4{};
        }
    }
}

}  // namespace

hipError_t start(const Call& c, void* clear, int64_t n, const float* from, float* to, Outs outs, hipStream_t st) {
    if (!(c.seqs.start || c.seqs.T == 0)) to = nullptr;  // every sequence has tokens
    const bool rows = c.p.clear && c.seqs.start && c.seqs.tokens > 0;
    if (!n && !to && !rows) return hipSuccess;
    int64_t wgs = (n + 511) / 512;  // n is even
    wgs = to && wgs < c.seqs.N ? c.seqs.N : wgs;
    wgs = rows && wgs < 256 ? 256 : wgs;
    hipLaunchKernelGGL(k_rec_start, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, st, (Word*)clear, n, c.seqs, from, to,
                       (int)c.p.dim, outs, rows ? (int)c.p.dim * (c.bf ? 2 : 4) : 0);
    return hipGetLastError();
}

hipError_t forward(const Call& c, const float* state_in, void* y, float* state_out, float* carry, uint32_t* ticket,
                   Word* words, hipStream_t st) {
    ForwardArgs a{c.seqs, c.in,   c.p.rate, state_in, y, state_out, carry, ticket, c.chunks > 1 ? words : nullptr,
                  (int)c.p.dim, (int)c.chunks, (int)c.blocks};
    const dim3 grid((unsigned)(c.chunks * c.blocks));
    auto* const kernel = c.span == kShortSpan ? (c.bf ? k_rec_forward<true, kShortSpan> : k_rec_forward<false, kShortSpan>)
                                              : (c.bf ? k_rec_forward<true, kForwardSpan> : k_rec_forward<false, kForwardSpan>);
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

hyena_status_t check(const hyena_recurrence_params_t* p, int64_t N, int64_t tokens, const int64_t* seq_start,
                     const hyena_recurrence_inputs_t* in, Call& c, bool whole) {
    if (!p || p->dim < 1 || (p->dtype != HYENA_F32 && p->dtype != HYENA_BF16) || N < 1 || tokens < 0)
        return HYENA_ERR_INVALID_ARG;
    if (!p->rate || ((uintptr_t)p->rate & 3u) || ((uintptr_t)seq_start & 7u)) return HYENA_ERR_INVALID_ARG;
    if (!seq_start && tokens % N) return HYENA_ERR_INVALID_ARG;
    if (p->dim % 8 || p->dim > (int64_t(1) << 20) || N > (int64_t(1) << 24) || tokens > kMaxTokens)
        return HYENA_ERR_UNSUPPORTED;
    c.p = *p;
    c.bf = p->dtype == HYENA_BF16;
    c.blocks = (p->dim + kCols - 1) / kCols;
    auto chunks = [&](int span) { return (tokens + kWaves * span - 1) / (kWaves * span); };
    c.span = chunks(kShortSpan) * c.blocks <= kShortGrid ? kShortSpan : kForwardSpan;
    c.chunks = chunks(c.span);
    c.back_chunks = (tokens + kBackwardChunk - 1) / kBackwardChunk;
    if (whole && c.back_chunks * c.blocks >= (int64_t(1) << 32) / kThreads) return HYENA_ERR_UNSUPPORTED;
    c.seqs = Seqs{seq_start, (int)N, (int)tokens, (int)(tokens / N)};
    if (!in) return HYENA_OK;
    c.in = *in;
    const void* rows[] = {in->x, in->r, in->i};
    const int64_t lds[] = {in->ldx, in->ldr, in->ldi};
    for (int k = 0; k < 3; ++k) {
        if ((tokens > 0 && !rows[k]) || !aligned16(rows[k])) return HYENA_ERR_INVALID_ARG;
        // whole sequences: see Rows; the step's offsets are of 64 bits
        if (lds[k] < p->dim || lds[k] % (c.bf ? 8 : 4) || lds[k] > int64_t(1) << (whole ? 22 : 31)) return HYENA_ERR_INVALID_ARG;
    }
    return HYENA_OK;
}

}  // namespace rec
}  // namespace hy

extern "C" {

static size_t words_bytes(int64_t n) { return n ? (size_t)(hy::rec::kHead + n) * sizeof(hy::rec::Word) : 0; }

size_t hyena_recurrence_workspace_bytes(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                        const int64_t* seq_start) {
    hy::rec::Call c;
    if (hy::rec::check(params, N, tokens, seq_start, nullptr, c) != HYENA_OK) return 0;
    return words_bytes(hy::rec::covering_words(c));
}

hyena_status_t hyena_recurrence_forward(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                        const int64_t* seq_start, const hyena_recurrence_inputs_t* in,
                                        const float* state_in, void* y, float* state_out, float* carries,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace hy;
    rec::Call c;
    if (!in) return HYENA_ERR_INVALID_ARG;
    const hyena_status_t st = rec::check(params, N, tokens, seq_start, in, c);
    if (st != HYENA_OK) return st;
    if ((tokens > 0 && !y) || !aligned16(y) || !aligned16(state_in) || !aligned16(state_out) || !aligned16(carries))
        return HYENA_ERR_INVALID_ARG;
    const size_t need = words_bytes(rec::word_count(c, c.chunks));
    if (need && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    if (need && !aligned16(workspace)) return HYENA_ERR_INVALID_ARG;
    rec::Word* head = (rec::Word*)workspace;
    hipError_t e = rec::start(c, head, (int64_t)(need / sizeof(rec::Word)), state_in, state_out, {{y}}, stream);
    if (e == hipSuccess && tokens > 0)
        e = rec::forward(c, state_in, y, state_out, carries, (uint32_t*)head, head + rec::kHead, stream);
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
