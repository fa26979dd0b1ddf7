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

// One chunk and 128 channels.
template <bool BF>
__global__ __launch_bounds__(kThreads) void k_rec_forward(ForwardArgs p) {
    using Raw = typename Io<BF>::Raw;
    __shared__ float sA[kWaves][kCols], sH[kWaves][kCols], sBackA[kWaves][kCols], sBackH[kWaves][kCols];
    __shared__ uint32_t sTicket;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ticket = blockIdx.x;
    if (p.words) {
        if (threadIdx.x == 0) sTicket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        ticket = __builtin_amdgcn_readfirstlane(sTicket);
    }
    const int chunk = ticket / p.blocks, at = kVec * lane;
    if (chunk >= p.chunks) return;  // only where a caller's workspace is not this call's alone
    const int own = (ticket - chunk * p.blocks) * kCols + at;
    const bool ok = own < p.dim;
    const int col = ok ? own : p.dim - kVec;  // lanes behind the last channel load along
    const Span<kForwardSpan> span(p.seqs, chunk * kForwardChunk + wave * kForwardSpan);
    float a[kForwardSpan][kVec], b[kForwardSpan][kVec];
    float A[kVec] = {1.f, 1.f}, H[kVec] = {};
    if (span.hi > span.lo) {
        Raw x[kForwardSpan], r[kForwardSpan], i[kForwardSpan];
#pragma unroll
        for (int s = 0; s < kForwardSpan; ++s) {
            const int row = span.row(s);
            x[s] = load_row<BF>(p.in.x, p.in.ldx, row, col);
            r[s] = load_row<BF>(p.in.r, p.in.ldr, row, col);
            i[s] = load_row<BF>(p.in.i, p.in.ldi, row, col);
        }
        float rate[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) rate[j] = p.rate[col + j];
#pragma unroll
        for (int s = 0; s < kForwardSpan; ++s) {
            float xv[kVec], rv[kVec], iv[kVec];
            Io<BF>::get(x[s], xv);
            Io<BF>::get(r[s], rv);
            Io<BF>::get(i[s], iv);
#pragma unroll
            for (int j = 0; j < kVec; ++j) gate(xv[j], rv[j], iv[j], rate[j], a[s][j], b[s][j]);
            if (!span.has(s))
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    a[s][j] = 1.f;
                    b[s][j] = 0.f;
                }
            if (span.first >> s & 1) {  // from the sequence's initial state, and from nothing in front of it
                int n = p.seqs.of(span.t0 + s);
                n = n < 0 ? 0 : n;
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    if (p.state_in) b[s][j] = fmaf(a[s][j], p.state_in[(int64_t)n * p.dim + col + j], b[s][j]);
                    H[j] = b[s][j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    H[j] = fmaf(a[s][j], H[j], b[s][j]);
                    A[j] *= a[s][j];
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        sA[wave][at + j] = span.first ? kReset : A[j];
        sH[wave][at + j] = H[j];
    }
    __syncthreads();
    float h[kVec] = {};
    if (p.words) {
        const bool publishes = wave == 0 && ok && chunk + 1 < p.chunks, ends = (chunk & (kGroup - 1)) == kGroup - 1;
        float cA[kVec], cH[kVec];
        if (publishes) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                cA[j] = 1.f;
                cH[j] = 0.f;
            }
            for (int k = 0; k < kWaves; ++k)
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const float wA = sA[k][at + j];
                    join_word(wA, sH[k][at + j], cH[j]);
                    cA[j] = wA == kReset || cA[j] == kReset ? kReset : cA[j] * wA;
                }
            if (!ends) publish(p.words, chunk, p.dim, own, cA, cH);
        }
        if (chunk) {
            float bA[kVec], bH[kVec];
            look_back(p.words, chunk, p.dim, col, wave, bA, bH);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                sBackA[wave][at + j] = bA[j];
                sBackH[wave][at + j] = bH[j];
            }
            __syncthreads();
            for (int k = 0; k < kWaves; ++k)
#pragma unroll
                for (int j = 0; j < kVec; ++j) join_word(sBackA[k][at + j], sBackH[k][at + j], h[j]);
        }
        if (publishes && ends) {
            float e[kVec], reset[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                e[j] = h[j];
                join_word(cA[j], cH[j], e[j]);
                reset[j] = kReset;
            }
            publish(p.words, chunk, p.dim, own, reset, e);
        }
    }
    for (int k = 0; k < wave; ++k)
#pragma unroll
        for (int j = 0; j < kVec; ++j) join_word(sA[k][at + j], sH[k][at + j], h[j]);
    if (p.carry && span.t0 % kBackwardChunk == 0 && span.t0 < p.seqs.tokens && ok)
#pragma unroll
        for (int j = 0; j < kVec; ++j) p.carry[(int64_t)(span.t0 / kBackwardChunk) * p.dim + own + j] = h[j];
    if (!p.y || span.hi <= span.lo) return;
#pragma unroll
    for (int s = 0; s < kForwardSpan; ++s) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[j] = span.first >> s & 1 ? b[s][j] : fmaf(a[s][j], h[j], b[s][j]);
        if (ok && span.has(s)) store_row<BF>(p.y, p.dim, span.t0 + s, own, h);
        if (p.state_out && (span.last >> s & 1) && ok) {
            int n = p.seqs.of(span.t0 + s);
            n = n < 0 ? 0 : n;
#pragma unroll
            for (int j = 0; j < kVec; ++j) p.state_out[(int64_t)n * p.dim + own + j] = h[j];
        }
    }
}

// Clears what the chunks' words and tickets lie in; a sequence without tokens passes its state on.
__global__ __launch_bounds__(256) void k_rec_start(Word* clear, int64_t n, Seqs q, const float* from, float* to, int dim) {
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) clear[e] = 0;
    if (to)
        for (int s = blockIdx.x; s < q.N; s += gridDim.x) {
            if (q.at(s + 1) > q.at(s)) continue;
            for (int c = threadIdx.x; c < dim; c += 256) {
                const int64_t e = (int64_t)s * dim + c;
                to[e] = from ? from[e] : 0.f;
            }
        }
}

}  // namespace

hipError_t start(const Call& c, void* clear, int64_t n, const float* from, float* to, hipStream_t st) {
    if (!(c.seqs.start || c.seqs.T == 0)) to = nullptr;  // every sequence has tokens
    if (!n && !to) return hipSuccess;
    int64_t wgs = (n + 1023) / 1024;
    wgs = to && wgs < c.seqs.N ? c.seqs.N : wgs;
    hipLaunchKernelGGL(k_rec_start, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, st, (Word*)clear, n, c.seqs, from, to,
                       (int)c.p.dim);
    return hipGetLastError();
}

hipError_t forward(const Call& c, const float* state_in, void* y, float* state_out, float* carry, uint32_t* ticket,
                   Word* words, hipStream_t st) {
    ForwardArgs a{c.seqs, c.in,   c.p.rate, state_in, y, state_out, carry, ticket, c.chunks > 1 ? words : nullptr,
                  (int)c.p.dim, (int)c.chunks, (int)c.blocks};
    const dim3 grid((unsigned)(c.chunks * c.blocks));
    if (c.bf)
        hipLaunchKernelGGL(k_rec_forward<true>, grid, dim3(kThreads), 0, st, a);
    else
        hipLaunchKernelGGL(k_rec_forward<false>, grid, dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

hyena_status_t check(const hyena_recurrence_params_t* p, int64_t N, int64_t tokens, const int64_t* seq_start,
                     const hyena_recurrence_inputs_t* in, Call& c) {
    if (!p || p->dim < 1 || (p->dtype != HYENA_F32 && p->dtype != HYENA_BF16) || N < 1 || tokens < 0)
        return HYENA_ERR_INVALID_ARG;
    if (!p->rate || ((uintptr_t)p->rate & 3u) || ((uintptr_t)seq_start & 7u)) return HYENA_ERR_INVALID_ARG;
    if (!seq_start && tokens % N) return HYENA_ERR_INVALID_ARG;
    if (p->dim % 8 || p->dim > (int64_t(1) << 20) || N > (int64_t(1) << 24) || tokens > kMaxTokens)
        return HYENA_ERR_UNSUPPORTED;
    c.p = *p;
    c.bf = p->dtype == HYENA_BF16;
    c.chunks = (tokens + kForwardChunk - 1) / kForwardChunk;
    c.back_chunks = (tokens + kBackwardChunk - 1) / kBackwardChunk;
    c.blocks = (p->dim + kCols - 1) / kCols;
    if (c.back_chunks * c.blocks >= (int64_t(1) << 32) / kThreads) return HYENA_ERR_UNSUPPORTED;
    c.seqs = Seqs{seq_start, (int)N, (int)tokens, (int)(tokens / N)};
    if (!in) return HYENA_OK;
    c.in = *in;
    const void* rows[] = {in->x, in->r, in->i};
    const int64_t lds[] = {in->ldx, in->ldr, in->ldi};
    for (int k = 0; k < 3; ++k) {
        if ((tokens > 0 && !rows[k]) || !aligned16(rows[k])) return HYENA_ERR_INVALID_ARG;
        if (lds[k] < p->dim || lds[k] % (c.bf ? 8 : 4) || lds[k] > (int64_t(1) << 22)) return HYENA_ERR_INVALID_ARG;
    }
    return HYENA_OK;
}

}  // namespace rec
}  // namespace hy

extern "C" {

size_t hyena_recurrence_workspace_bytes(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                        const int64_t* seq_start) {
    hy::rec::Call c;
    if (hy::rec::check(params, N, tokens, seq_start, nullptr, c) != HYENA_OK) return 0;
    const int64_t n = hy::rec::word_count(c, c.chunks);
    return n ? (size_t)(hy::rec::kHead + n) * sizeof(hy::rec::Word) : 0;
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
    const size_t need = hyena_recurrence_workspace_bytes(params, N, tokens, seq_start);
    if (need && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    if (need && !aligned16(workspace)) return HYENA_ERR_INVALID_ARG;
    rec::Word* head = (rec::Word*)workspace;
    hipError_t e = rec::start(c, head, (int64_t)(need / sizeof(rec::Word)), state_in, state_out, stream);
    if (e == hipSuccess && tokens > 0)
        e = rec::forward(c, state_in, y, state_out, carries, (uint32_t*)head, head + rec::kHead, stream);
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
