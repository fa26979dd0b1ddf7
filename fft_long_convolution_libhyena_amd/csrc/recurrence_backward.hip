// Gated linear recurrence over whole sequences, backward (see recurrence.hpp). With
// g[t] = a[t] dh[t], what token t hands to the one in front of it, and
// dh[t] = dy[t] + g[t + 1] (behind a sequence's last token: the final state's gradient),
//   dx = dh m sig(i),   di = dh m x sig(i) (1 - sig(i)),
//   W  = dh (a log(a) h[t - 1] - a^2 (log(a) / m) sig(i) x),
//   dr = (1 - sig(r)) W,   drate = sum W / c.
// log(a) / m -> 0 as a -> 1, so nothing is divided by 0 where a gate is shut. g runs
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
    float2* ends;         // [chunks][dim]: (A, G); A = -1: a sequence ends inside
    const float* carry;   // [chunks][dim]: states in front of the chunks
    const float* behind;  // [chunks][dim]: g behind the chunks
    float* part;          // [chunks][dim]: sums of W
    int dim;
};

template <bool BF, bool ENDS>
__global__ __launch_bounds__(kThreads) void k_rec_backward(BackwardArgs p) {
    using Raw = typename Io<BF>::Raw;
    __shared__ float sA[kWaves][kCols], sH[kWaves][kCols], sG[kWaves][kCols];
    __shared__ int sFirst[kWaves], sLast[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunk = blockIdx.x, at = kVec * lane;
    const int own = blockIdx.y * kCols + at;
    const bool ok = own < p.dim;
    const int col = ok ? own : p.dim - kVec;
    const Span span(p.seqs, chunk * kChunk + wave * kSpan);
    auto state = [&](const float* from, int s, float (&h)[kVec]) {
        int n = p.seqs.of(span.t0 + s);
        n = n < 0 ? 0 : n;
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[j] = from ? from[(int64_t)n * p.dim + col + j] : 0.f;
    };
    Raw x[kSpan], dy[kSpan];
    float w[kSpan][kVec], a[kSpan][kVec], si[kSpan][kVec];  // w = -log a
    float A[kVec] = {1.f, 1.f}, H[kVec] = {}, G[kVec] = {}, rate[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) rate[j] = p.rate[col + j];
    const bool some = span.hi > span.lo;
    if (some) {
        Raw r[kSpan], i[kSpan];
#pragma unroll
        for (int s = 0; s < kSpan; ++s) {
            const int row = span.row(s);
            r[s] = load_row<BF>(p.in.r, p.in.ldr, row, col);
            dy[s] = load_row<BF>(p.dy, p.dim, row, col);
            if constexpr (!ENDS) {
                x[s] = load_row<BF>(p.in.x, p.in.ldx, row, col);
                i[s] = load_row<BF>(p.in.i, p.in.ldi, row, col);
            }
        }
#pragma unroll
        for (int s = 0; s < kSpan; ++s) {
            float rv[kVec], xv[kVec], iv[kVec];
            Io<BF>::get(r[s], rv);
            if constexpr (!ENDS) {
                Io<BF>::get(x[s], xv);
                Io<BF>::get(i[s], iv);
            }
            if (span.first >> s & 1) state(p.state_in, s, H);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                float q;
                w[s][j] = rate[j] * sigmoid(rv[j]);
                decay(w[s][j], a[s][j], q);
                if (!span.has(s)) a[s][j] = 1.f;
                A[j] *= a[s][j];
                if constexpr (!ENDS) {
                    si[s][j] = sigmoid(iv[j]);
                    if (span.has(s)) H[j] = fmaf(a[s][j], H[j], __builtin_amdgcn_sqrtf(q) * si[s][j] * xv[j]);
                }
            }
        }
#pragma unroll
        for (int s = kSpan - 1; s >= 0; --s) {
            float d[kVec];
            Io<BF>::get(dy[s], d);
            if (span.last >> s & 1) state(p.dstate_out, s, G);
            if (span.has(s))
#pragma unroll
                for (int j = 0; j < kVec; ++j) G[j] = a[s][j] * (d[j] + G[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        sA[wave][at + j] = A[j];
        sH[wave][at + j] = H[j];
        sG[wave][at + j] = G[j];
    }
    if (lane == 0) {
        sFirst[wave] = span.first != 0;
        sLast[wave] = span.last != 0;
    }
    __syncthreads();
    if constexpr (ENDS) {
        if (wave == 0 && ok) {
            float cA[kVec] = {1.f, 1.f}, cG[kVec] = {};
            bool reset = false;
            for (int w = kWaves - 1; w >= 0; --w) {
                const bool rs = sLast[w];
                reset |= rs;
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const float wA = sA[w][at + j], wG = sG[w][at + j];
                    cG[j] = rs ? wG : fmaf(wA, cG[j], wG);
                    cA[j] *= wA;
                }
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                p.ends[(int64_t)chunk * p.dim + own + j] = float2{reset ? -1.f : cA[j], cG[j]};
        }
        return;
    }
    float sum[kVec] = {};
    if (some) {
        float h[kVec], g[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            h[j] = p.carry[(int64_t)chunk * p.dim + col + j];
            g[j] = p.behind[(int64_t)chunk * p.dim + col + j];
        }
        for (int k = 0; k < wave; ++k) {
            const bool rs = sFirst[k];
#pragma unroll
            for (int j = 0; j < kVec; ++j) h[j] = rs ? sH[k][at + j] : fmaf(sA[k][at + j], h[j], sH[k][at + j]);
        }
        for (int k = kWaves - 1; k > wave; --k) {
            const bool rs = sLast[k];
#pragma unroll
            for (int j = 0; j < kVec; ++j) g[j] = rs ? sG[k][at + j] : fmaf(sA[k][at + j], g[j], sG[k][at + j]);
        }
        float before[kSpan][kVec];
#pragma unroll
        for (int s = 0; s < kSpan; ++s) {
            float xv[kVec];
            Io<BF>::get(x[s], xv);
            if (span.first >> s & 1) state(p.state_in, s, h);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                before[s][j] = h[j];
                float ar, q;
                decay(w[s][j], ar, q);
                if (span.has(s)) h[j] = fmaf(a[s][j], h[j], __builtin_amdgcn_sqrtf(q) * si[s][j] * xv[j]);
            }
        }
#pragma unroll
        for (int s = kSpan - 1; s >= 0; --s) {
            if (!span.has(s)) continue;
            float xv[kVec], d[kVec], ox[kVec], orr[kVec], oi[kVec];
            Io<BF>::get(x[s], xv);
            Io<BF>::get(dy[s], d);
            if (span.last >> s & 1) state(p.dstate_out, s, g);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float dh = d[j] + g[j];
                float ar, q;
                decay(w[s][j], ar, q);
                q += 1e-37f;  // w / m is 0 where both are
                const float rs = __builtin_amdgcn_rsqf(q), m = q * rs;
                ox[j] = dh * m * si[s][j];
                oi[j] = ox[j] * xv[j] * (1.f - si[s][j]);
                const float aw = a[s][j] * w[s][j];
                const float W = dh * (a[s][j] * aw * rs * si[s][j] * xv[j] - aw * before[s][j]);
                orr[j] = fmaf(-w[s][j], __builtin_amdgcn_rcpf(rate[j]), 1.f) * W;
                sum[j] += W;
                g[j] = a[s][j] * dh;
            }
            if (ok) {
                store_row<BF>(p.dx, p.dim, span.t0 + s, own, ox);
                store_row<BF>(p.dr, p.dim, span.t0 + s, own, orr);
                store_row<BF>(p.di, p.dim, span.t0 + s, own, oi);
                if (p.dstate_in && (span.first >> s & 1)) {
                    int n = p.seqs.of(span.t0 + s);
                    n = n < 0 ? 0 : n;
#pragma unroll
                    for (int j = 0; j < kVec; ++j) p.dstate_in[(int64_t)n * p.dim + own + j] = g[j];
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kVec; ++j) sH[wave][at + j] = sum[j];
    __syncthreads();
    if (wave == 0 && ok)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            float t = 0.f;
            for (int w = 0; w < kWaves; ++w) t += sH[w][at + j];
            p.part[(int64_t)chunk * p.dim + own + j] = t;
        }
}

// drate: 32 channels x 32 rows of threads over the chunks' sums
__global__ __launch_bounds__(1024) void k_rec_drate(const float* part, const float* rate, float* drate, int64_t chunks,
                                                    int dim) {
    __shared__ double red[32][33];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5, e = blockIdx.x * 32 + c;
    double s = 0;
    if (e < dim)
        for (int64_t i = r; i < chunks; i += 32) s += (double)part[i * dim + e];
    red[r][c] = s;
    __syncthreads();
    for (int d = 16; d > 0; d >>= 1) {
        if (r < d) red[r][c] += red[r + d][c];
        __syncthreads();
    }
    if (r == 0 && e < dim) drate[e] = (float)(red[0][c] / (double)rate[e]);
}

struct Layout {
    float2* ends;
    float *carry, *behind, *part;
    size_t bytes;
};
Layout layout(const Call& c, bool carries, void* base) {
    const size_t n = (size_t)(c.chunks * c.p.dim);
    Layout l;
    unsigned char* at = (unsigned char*)base;
    l.ends = (float2*)at;
    l.behind = (float*)(at + 8 * n);
    l.part = l.behind + n;
    l.carry = l.part + n;
    l.bytes = (carries ? 16 : 20) * n;
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
    return hy::rec::layout(c, carries != nullptr, nullptr).bytes;
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
    const rec::Layout l = rec::layout(c, carries != nullptr, workspace);
    if (l.bytes && (!workspace || workspace_bytes < l.bytes)) return HYENA_ERR_WORKSPACE;
    if (l.bytes && !aligned16(workspace)) return HYENA_ERR_INVALID_ARG;
    const int dim = (int)params->dim;
    hipError_t e = rec::pass_empty(c, dstate_out, dstate_in, stream);
    if (e == hipSuccess && tokens > 0) {
        if (!carries) e = rec::forward_carries(c, state_in, l.ends, l.carry, stream);
        if (e != hipSuccess) return HYENA_ERR_DEVICE;
        rec::BackwardArgs a{c.seqs,  c.in, params->rate, state_in, dy,       dstate_out,
                            dx,      dr,   di,           dstate_in, l.ends,  carries ? carries : l.carry,
                            l.behind, l.part, dim};
        const dim3 grid((unsigned)c.chunks, (unsigned)c.blocks), block(rec::kThreads);
        if (c.bf)
            hipLaunchKernelGGL((rec::k_rec_backward<true, true>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((rec::k_rec_backward<false, true>), grid, block, 0, stream, a);
        e = hipGetLastError();
        if (e == hipSuccess) e = rec::join_chunks(c, l.ends, l.behind, -1, stream);
        if (e != hipSuccess) return HYENA_ERR_DEVICE;
        if (c.bf)
            hipLaunchKernelGGL((rec::k_rec_backward<true, false>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((rec::k_rec_backward<false, false>), grid, block, 0, stream, a);
        e = hipGetLastError();
    }
    if (e == hipSuccess) {
        hipLaunchKernelGGL(rec::k_rec_drate, dim3((unsigned)((dim + 31) / 32)), dim3(1024), 0, stream, l.part,
                           params->rate, drate, c.chunks, dim);
        e = hipGetLastError();
    }
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
