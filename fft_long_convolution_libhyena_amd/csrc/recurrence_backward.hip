// Gated linear recurrence over whole sequences, backward (see recurrence.hpp). With
// g[t] = a[t] dh[t], what token t hands to the one in front of it, and
// dh[t] = dy[t] + g[t + 1] (behind a sequence's last token: the final state's gradient),
//   dx = dh m sig(i),   di = dh m x sig(i) (1 - sig(i)),
//   W  = dh (a log(a) h[t - 1] - a^2 (log(a) / m) sig(i) x),
//   dr = (1 - sig(r)) W,   drate = sum W / c.
// log(a) / m -> 0 as a -> 1, so nothing is divided by 0 where a gate is shut; 1 - sig comes from exp(-r) and
// exp(-i), which are kept, so that the gradients of gates wide open keep their digits (2% of the training
// step's time against the difference). g runs
// through the chunks from the last to the first as h does from the first: (A, G) of a chunk
// need only its own tokens. h is computed again from the states in front of the chunks.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "recurrence.hpp"

namespace hy {
namespace rec {
namespace {

struct BackwardArgs {
    Seqs seqs;
    hyena_recurrence_inputs_t in;
    const float *rate, *state_in;
    const void* dy;
    const float* dstate_out;
    void *dx, *dr, *di;
    float* dstate_in;
    const float* carry;  // [chunks][dim]: states in front of the chunks
    float* part;         // [chunks][dim]: sums of W
    uint32_t* ticket;
    Word* words;         // [chunks][dim], from the last chunk on; null: one chunk
    int dim, chunks, blocks;
};

// One chunk and 128 channels, the chunks from the last to the first. 8 x 8192 x 768 in bf16 take 172 to 177 us: 752 MB
// at 4.3 TB/s, vector work 65% of the cycles (without the last pass's polynomial, with 1 - a kept in place of a: 1 us less).
template <bool BF>
__global__ __launch_bounds__(kThreads, BF ? 4 : 2) void k_rec_backward(BackwardArgs p) {
    using Raw = typename Io<BF>::Raw;
    constexpr int S = kBackwardSpan, W = kWaves;
    __shared__ Link sG[W][64], sBehind[W][64];  // (A, G) of the waves and of the chunks behind
    __shared__ float2 sSum[W][64];               // of the waves' w
    __shared__ float2 sH[W][64], sEi[W][S][64];  // sEi: a lane's own exp(-i), kept for the last pass
    __shared__ int sFirst[W], sLast[W], sBehindReset[W];
    __shared__ uint32_t sTicket;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ticket = blockIdx.x;
    if (p.words) {
        if (threadIdx.x == 0) sTicket = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        ticket = __builtin_amdgcn_readfirstlane(sTicket);
    }
    const int order = (uint32_t)ticket / (uint32_t)p.blocks, chunk = p.chunks - 1 - order;
    if ((uint32_t)order >= (uint32_t)p.chunks) return;  // only where a caller's workspace is not this call's alone
    const int own = (ticket - order * p.blocks) * kCols + kVec * lane;
    const bool ok = own < p.dim;
    const int col = ok ? own : p.dim - kVec, at = ok ? own * Io<BF>::kBytes : kNone;
    const Span<S> span(p.seqs, chunk * kBackwardChunk + wave * S);
    const int rows = p.seqs.tokens - span.t0 < S ? p.seqs.tokens - span.t0 : S;
    auto state = [&](const float* from, int s, float (&h)[kVec]) {
        const int64_t n = span.sequence(s);
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[j] = from ? from[n * p.dim + col + j] : 0.f;
    };
    Raw x[S], dy[S], i[S];
    float er[S][kVec], a[S][kVec], b[S][kVec];  // exp(-r), a, m sig(i) x
    float rate[kVec], w_sum[kVec] = {}, A[kVec] = {1.f, 1.f}, H[kVec] = {}, G[kVec] = {};
#pragma unroll
    for (int j = 0; j < kVec; ++j) rate[j] = p.rate[col + j];
    const bool near = near_rates(rate);
    if (span.have) {
        Raw r[S];
        const Rows<BF> xs(p.in.x, p.in.ldx, span.t0, rows, p.dim), rs(p.in.r, p.in.ldr, span.t0, rows, p.dim),
            is(p.in.i, p.in.ldi, span.t0, rows, p.dim), ds(p.dy, p.dim, span.t0, rows, p.dim);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int row = span.row(s);
            r[s] = rs.load(row, at);
            dy[s] = ds.load(row, at);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int row = span.row(s);
            i[s] = is.load(row, at);
            x[s] = xs.load(row, at);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float rv[kVec], q[kVec], w[kVec];
            Io<BF>::get(r[s], rv);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                er[s][j] = exp_minus(rv[j]);
                w[j] = rate[j] * __builtin_amdgcn_rcpf(1.f + er[s][j]);
            }
            decay(w, near, a[s], q);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                b[s][j] = __builtin_amdgcn_sqrtf(q[j]);
                w_sum[j] += w[j];
            }
        }
        run_decay(w_sum, A);
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
            float d[kVec];
            Io<BF>::get(dy[s], d);
            if (span.ends(s)) state(p.dstate_out, s, G);
#pragma unroll
            for (int j = 0; j < kVec; ++j) G[j] = a[s][j] * (d[j] + G[j]);
        }
    }
    sG[wave][lane] = Link{A[0], A[1], G[0], G[1]};
    sSum[wave][lane] = float2{w_sum[0], w_sum[1]};
    if (lane == 0) {
        sFirst[wave] = span.first != 0;
        sLast[wave] = span.last != 0;
    }
    __syncthreads();
    // (A, G) goes out as soon as it is known; the words of the chunks behind travel while the waves
    // work on what only this chunk needs
    const bool publishes = p.words && wave == 0 && order + 1 < p.chunks, ends = (order & (kGroup - 1)) == kGroup - 1;
    const bool looks = p.words && order;
    float cw[kVec] = {}, cA[kVec] = {1.f, 1.f}, cG[kVec] = {};
    bool reset = false;
    const uint32_t first_bits = flag_bits(sFirst, lane), last_bits = flag_bits(sLast, lane);
    if (publishes) {
        reset = last_bits != 0;
#pragma unroll
        for (int k = W - 1; k >= 0; --k) {
            const Link v = sG[k][lane];
            const float2 u = sSum[k][lane];
            join_link(last_bits >> k & 1, v, cG);
            cw[0] += u.x;
            cw[1] += u.y;
        }
        run_decay(cw, cA);
        if (!ends && ok) publish(p.words, order, p.dim, own, reset, cA, cG);
    }
    LookBack look(p.words, order, p.dim, col, wave);
    if (looks) look.ask();
    if (span.have) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float xv[kVec], iv[kVec];
            Io<BF>::get(x[s], xv);
            Io<BF>::get(i[s], iv);
            if (span.begins(s)) state(p.state_in, s, H);
            float ei[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                ei[j] = exp_minus(iv[j]);
                b[s][j] *= __builtin_amdgcn_rcpf(1.f + ei[j]) * xv[j];
                H[j] = fmaf(a[s][j], H[j], b[s][j]);
            }
            sEi[wave][s][lane] = float2{ei[0], ei[1]};
        }
    }
    sH[wave][lane] = float2{H[0], H[1]};
    if (looks) {
        Link back;
        const bool rs = look.done(back);
        sBehind[wave][lane] = back;
        if (lane == 0) sBehindReset[wave] = rs;
    }
    __syncthreads();
    float g[kVec] = {}, h[kVec] = {};
    if (looks)
        join_links(flag_bits(sBehindReset, lane), 0, 1, W, [&](int k) { return sBehind[k][lane]; }, g);
    if (publishes && ends) {
        float e[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) e[j] = reset ? cG[j] : fmaf(cA[j], g[j], cG[j]);
        if (ok) publish(p.words, order, p.dim, own, true, e, e);
    }
    float sum[kVec] = {};
    if (span.have) {
        join_links(last_bits, W - 1, -1, W - 1 - wave, [&](int k) { return sG[k][lane]; }, g);
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[j] = p.carry[(int64_t)chunk * p.dim + col + j];
        join_links(
            first_bits, 0, 1, wave,
            [&](int k) {
                const Link v = sG[k][lane];
                const float2 u = sH[k][lane];
                return Link{v[0], v[1], u.x, u.y};
            },
            h);
#pragma unroll
        for (int s = 0; s < S; ++s) {  // b becomes the states in front of the tokens
            if (span.begins(s)) state(p.state_in, s, h);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float before = h[j];
                h[j] = fmaf(a[s][j], h[j], b[s][j]);
                b[s][j] = before;
            }
        }
        const Rows<BF> oxs(p.dx, p.dim, span.t0, rows, p.dim), ors(p.dr, p.dim, span.t0, rows, p.dim),
            ois(p.di, p.dim, span.t0, rows, p.dim);
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
            if (!span.has(s)) continue;
            float xv[kVec], d[kVec], ox[kVec], orr[kVec], oi[kVec], w[kVec], shut[kVec], again[kVec], q[kVec];
            Io<BF>::get(x[s], xv);
            Io<BF>::get(dy[s], d);
            if (span.ends(s)) state(p.dstate_out, s, g);
            const float2 kept = sEi[wave][s][lane];
            const float ei[kVec] = {kept.x, kept.y};
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float sr = __builtin_amdgcn_rcpf(1.f + er[s][j]);
                w[j] = rate[j] * sr;
                shut[j] = one_minus(er[s][j], sr);
            }
            decay(w, near, again, q, 1e-37f);  // w / m is 0 where both are
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float dh = d[j] + g[j];
                const float si = __builtin_amdgcn_rcpf(1.f + ei[j]);
                const float rs = __builtin_amdgcn_rsqf(q[j]), sx = si * xv[j], aw = a[s][j] * w[j];
                ox[j] = dh * (q[j] * rs) * si;
                oi[j] = ox[j] * xv[j] * one_minus(ei[j], si);
                const float share = dh * aw * fmaf(a[s][j] * rs, sx, -b[s][j]);
                orr[j] = shut[j] * share;
                sum[j] += share;
                g[j] = a[s][j] * dh;
            }
            oxs.store(s, at, ox);
            ors.store(s, at, orr);
            ois.store(s, at, oi);
            if (p.dstate_in && span.begins(s) && ok) {
                const int64_t n = span.sequence(s);
#pragma unroll
                for (int j = 0; j < kVec; ++j) p.dstate_in[n * p.dim + own + j] = g[j];
            }
        }
    }
    __syncthreads();
    sH[wave][lane] = float2{sum[0], sum[1]};
    __syncthreads();
    if (wave == 0 && ok) {
        float2 t{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float2 v = sH[k][lane];
            t.x += v.x;
            t.y += v.y;
        }
        *reinterpret_cast<float2*>(p.part + (int64_t)chunk * p.dim + own) = t;
    }
}

// drate: 32 channels x 32 rows of threads over the chunks' sums, 16 of each thread on their way
__global__ __launch_bounds__(1024) void k_rec_drate(const float* part, const float* rate, float* drate, int64_t chunks,
                                                    int dim) {
    constexpr int kAhead = 16;
    __shared__ double red[32][33];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5, e = blockIdx.x * 32 + c;
    double s = 0;
    if (e < dim)
        for (int64_t i = r; i < chunks; i += 32 * kAhead) {
            float x[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {  // rows behind the last are read again, without a branch
                const int64_t row = i + 32 * j;
                x[j] = part[(row < chunks ? row : chunks - 1) * dim + e];
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) s += i + 32 * j < chunks ? (double)x[j] : 0.;
        }
    red[r][c] = s;
    __syncthreads();
    for (int d = 16; d > 0; d >>= 1) {
        if (r < d) red[r][c] += red[r + d][c];
        __syncthreads();
    }
    if (r == 0 && e < dim) drate[e] = (float)(red[0][c] / (double)rate[e]);
}

// What start() clears (tickets, then the words of the backward and, without carries, the
// forward), then the partial sums and, without carries, the states in front of the chunks
struct Layout {
    Word* head;
    int64_t clear;  // words
    float *part, *carry;
    size_t bytes;
};
// forward_words: of the forward that makes the states again
Layout layout(const Call& c, bool carries, int64_t forward_words, void* base) {
    const int64_t n = word_count(c, c.back_chunks) + (carries ? 0 : forward_words), kept = c.back_chunks * c.p.dim;
    Layout l;
    l.head = (Word*)base;
    l.clear = n ? kHead + n : 0;
    l.part = (float*)(l.head + l.clear);
    l.carry = l.part + kept;
    l.bytes = (size_t)l.clear * sizeof(Word) + (size_t)kept * (carries ? 4 : 8);
    return l;
}

}  // namespace
}  // namespace rec
}  // namespace hy

extern "C" {

size_t hyena_recurrence_backward_workspace_bytes(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                                 const int64_t* seq_start, const float* carries) {
    hy::rec::Call c;
    if (hy::rec::check(params, N, tokens, seq_start, nullptr, c) != HYENA_OK) return 0;
    return hy::rec::layout(c, carries != nullptr, hy::rec::covering_words(c), nullptr).bytes;
}

hyena_status_t hyena_recurrence_backward(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                         const int64_t* seq_start, const hyena_recurrence_inputs_t* in,
                                         const float* state_in, const float* carries, const void* dy,
                                         const float* dstate_out, void* dx, void* dr, void* di, float* drate,
                                         float* dstate_in, void* workspace, size_t workspace_bytes,
                                         hipStream_t stream) {
    using namespace hy;
    rec::Call c;
    if (!in) return HYENA_ERR_INVALID_ARG;
    const hyena_status_t st = rec::check(params, N, tokens, seq_start, in, c);
    if (st != HYENA_OK) return st;
    const void* rows[] = {dy, dx, dr, di};
    for (const void* q : rows)
        if ((tokens > 0 && !q) || !aligned16(q)) return HYENA_ERR_INVALID_ARG;
    const void* states[] = {state_in, carries, dstate_out, dstate_in};
    for (const void* q : states)
        if (!aligned16(q)) return HYENA_ERR_INVALID_ARG;
    if (!drate || ((uintptr_t)drate & 3u)) return HYENA_ERR_INVALID_ARG;
    const rec::Layout l = rec::layout(c, carries != nullptr, rec::word_count(c, c.chunks), workspace);
    if (l.bytes && (!workspace || workspace_bytes < l.bytes)) return HYENA_ERR_WORKSPACE;
    if (l.bytes && !aligned16(workspace)) return HYENA_ERR_INVALID_ARG;
    const int dim = (int)params->dim;
    hipError_t e = rec::start(c, l.head, l.clear, dstate_out, dstate_in, {{dx, dr, di}}, stream);
    if (e == hipSuccess && tokens > 0) {
        rec::Word* const words = l.head + rec::kHead;
        uint32_t* const tickets = (uint32_t*)l.head;
        if (!carries)
            e = rec::forward(c, state_in, nullptr, nullptr, l.carry, tickets + 1, words + rec::word_count(c, c.back_chunks),
                             stream);
        if (e != hipSuccess) return HYENA_ERR_DEVICE;
        rec::BackwardArgs a{c.seqs, c.in,      params->rate, state_in, dy,      dstate_out,
                            dx,     dr,        di,           dstate_in, carries ? carries : l.carry,
                            l.part, tickets,   c.back_chunks > 1 ? words : nullptr, dim, (int)c.back_chunks, (int)c.blocks};
        const dim3 grid((unsigned)(c.back_chunks * c.blocks));
        if (c.bf)
            hipLaunchKernelGGL(rec::k_rec_backward<true>, grid, dim3(rec::kThreads), 0, stream, a);
        else
            hipLaunchKernelGGL(rec::k_rec_backward<false>, grid, dim3(rec::kThreads), 0, stream, a);
        e = hipGetLastError();
    }
    if (e == hipSuccess) {
        hipLaunchKernelGGL(rec::k_rec_drate, dim3((unsigned)((dim + 31) / 32)), dim3(1024), 0, stream, l.part,
                           params->rate, drate, c.back_chunks, dim);
        e = hipGetLastError();
    }
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
