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
    float* state_out;
    float2* ends;        // [chunks][dim]: (A, H) of the chunks; A = -1: a sequence begins inside
    float* carry;        // [chunks][dim]: states in front of the chunks
    int dim;
};

// One chunk and 128 channels; ENDS: only (A, H) of the chunk, otherwise the outputs from
// the state in front of it.
template <bool BF, bool ENDS>
__global__ __launch_bounds__(kThreads) void k_rec_forward(ForwardArgs p) {
    using Raw = typename Io<BF>::Raw;
    __shared__ float sA[kWaves][kCols], sH[kWaves][kCols];
    __shared__ int sReset[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunk = blockIdx.x, at = kVec * lane;
    const int own = blockIdx.y * kCols + at;
    const bool ok = own < p.dim;
    const int col = ok ? own : p.dim - kVec;  // lanes behind the last channel load along
    const Span span(p.seqs, chunk * kChunk + wave * kSpan);
    float a[kSpan][kVec], b[kSpan][kVec];
    float A[kVec] = {1.f, 1.f}, H[kVec] = {};
    auto begin = [&](int s, float (&h)[kVec]) {  // the initial state of the sequence that token s begins
        int n = p.seqs.of(span.t0 + s);
        n = n < 0 ? 0 : n;
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[j] = p.state_in ? p.state_in[(int64_t)n * p.dim + col + j] : 0.f;
    };
    if (span.hi > span.lo) {
        Raw x[kSpan], r[kSpan], i[kSpan];
#pragma unroll
        for (int s = 0; s < kSpan; ++s) {
            const int row = span.row(s);
            x[s] = load_row<BF>(p.in.x, p.in.ldx, row, col);
            r[s] = load_row<BF>(p.in.r, p.in.ldr, row, col);
            i[s] = load_row<BF>(p.in.i, p.in.ldi, row, col);
        }
        float rate[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) rate[j] = p.rate[col + j];
#pragma unroll
        for (int s = 0; s < kSpan; ++s) {
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
            if (span.first >> s & 1) begin(s, H);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                H[j] = fmaf(a[s][j], H[j], b[s][j]);
                A[j] *= a[s][j];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        sA[wave][at + j] = A[j];
        sH[wave][at + j] = H[j];
    }
    if (lane == 0) sReset[wave] = span.first != 0;
    __syncthreads();
    if constexpr (ENDS) {
        if (wave == 0 && ok) {
            float cA[kVec] = {1.f, 1.f}, cH[kVec] = {};
            bool reset = false;
            for (int w = 0; w < kWaves; ++w) {
                const bool rs = sReset[w];
                reset |= rs;
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const float wA = sA[w][at + j], wH = sH[w][at + j];
                    cH[j] = rs ? wH : fmaf(wA, cH[j], wH);
                    cA[j] *= wA;
                }
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                p.ends[(int64_t)chunk * p.dim + own + j] = float2{reset ? -1.f : cA[j], cH[j]};
        }
        return;
    }
    if (span.hi <= span.lo) return;
    float h[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) h[j] = p.carry[(int64_t)chunk * p.dim + col + j];
    for (int w = 0; w < wave; ++w) {
        const bool rs = sReset[w];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const float wH = sH[w][at + j];
            h[j] = rs ? wH : fmaf(sA[w][at + j], h[j], wH);
        }
    }
#pragma unroll
    for (int s = 0; s < kSpan; ++s) {
        if (span.first >> s & 1) begin(s, h);
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[j] = fmaf(a[s][j], h[j], b[s][j]);
        if (ok && span.has(s)) store_row<BF>(p.y, p.dim, span.t0 + s, own, h);
        if (p.state_out && (span.last >> s & 1) && ok) {
            int n = p.seqs.of(span.t0 + s);
            n = n < 0 ? 0 : n;
#pragma unroll
            for (int j = 0; j < kVec; ++j) p.state_out[(int64_t)n * p.dim + own + j] = h[j];
        }
    }
}

// states between the chunks of one channel, in order (DIR 1) or from the last (DIR -1)
__global__ __launch_bounds__(64) void k_rec_carry(const float2* ends, float* carry, int chunks, int dim, int dir) {
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (col >= dim) return;
    float h = 0.f;
    for (int k = 0; k < chunks; ++k) {
        const int64_t e = (int64_t)(dir > 0 ? k : chunks - 1 - k) * dim + col;
        const float2 v = ends[e];
        carry[e] = h;
        h = v.x < 0.f ? v.y : fmaf(v.x, h, v.y);
    }
}

// A sequence without tokens passes its state on.
__global__ __launch_bounds__(256) void k_rec_empty(Seqs q, const float* from, float* to, int dim) {
    for (int n = blockIdx.x; n < q.N; n += gridDim.x) {
        if (q.at(n + 1) > q.at(n)) continue;
        for (int c = threadIdx.x; c < dim; c += 256) {
            const int64_t e = (int64_t)n * dim + c;
            to[e] = from ? from[e] : 0.f;
        }
    }
}

}  // namespace

hipError_t join_chunks(const Call& c, const float2* ends, float* carry, int dir, hipStream_t st) {
    hipLaunchKernelGGL(k_rec_carry, dim3((unsigned)((c.p.dim + 63) / 64)), dim3(64), 0, st, ends, carry, (int)c.chunks,
                       (int)c.p.dim, dir);
    return hipGetLastError();
}

hipError_t pass_empty(const Call& c, const float* from, float* to, hipStream_t st) {
    if (!to || !(c.seqs.start || c.seqs.T == 0)) return hipSuccess;
    hipLaunchKernelGGL(k_rec_empty, dim3((unsigned)(c.seqs.N < 4096 ? c.seqs.N : 4096)), dim3(256), 0, st, c.seqs, from,
                       to, (int)c.p.dim);
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
    c.chunks = (tokens + kChunk - 1) / kChunk;
    c.blocks = (p->dim + kCols - 1) / kCols;
    if (c.chunks * c.blocks >= (int64_t(1) << 32) / kThreads) return HYENA_ERR_UNSUPPORTED;
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

hipError_t forward_carries(const Call& c, const float* state_in, float2* ends, float* carry, hipStream_t st) {
    ForwardArgs a{c.seqs, c.in, c.p.rate, state_in, nullptr, nullptr, ends, carry, (int)c.p.dim};
    const dim3 grid((unsigned)c.chunks, (unsigned)c.blocks);
    if (c.bf)
        hipLaunchKernelGGL((k_rec_forward<true, true>), grid, dim3(kThreads), 0, st, a);
    else
        hipLaunchKernelGGL((k_rec_forward<false, true>), grid, dim3(kThreads), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return join_chunks(c, ends, carry, 1, st);
}

}  // namespace rec
}  // namespace hy

extern "C" {

size_t hyena_recurrence_workspace_bytes(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                        const int64_t* seq_start) {
    hy::rec::Call c;
    if (hy::rec::check(params, N, tokens, seq_start, nullptr, c) != HYENA_OK) return 0;
    return (size_t)(c.chunks * params->dim) * 12;
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
    hipError_t e = rec::pass_empty(c, state_in, state_out, stream);
    if (e == hipSuccess && tokens > 0) {
        float2* ends = (float2*)workspace;
        float* carry = carries ? carries : (float*)(ends + c.chunks * params->dim);
        e = rec::forward_carries(c, state_in, ends, carry, stream);
        if (e != hipSuccess) return HYENA_ERR_DEVICE;
        rec::ForwardArgs a{c.seqs, c.in, params->rate, state_in, y, state_out, ends, carry, (int)params->dim};
        const dim3 grid((unsigned)c.chunks, (unsigned)c.blocks);
        if (c.bf)
            hipLaunchKernelGGL((rec::k_rec_forward<true, false>), grid, dim3(rec::kThreads), 0, stream, a);
        else
            hipLaunchKernelGGL((rec::k_rec_forward<false, false>), grid, dim3(rec::kThreads), 0, stream, a);
        e = hipGetLastError();
    }
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
