// Gated delta rule, recurrent form: a few tokens of every sequence against states
// that stay in a pool in device memory (one read and one write of each state, whatever
// the number of tokens).
//
// With s = S^T k and z = S^T q over the old state, one pass over S gives both:
//   w = beta (v - a s);   S <- a S + k w^T;   o = scale (a z + (k . q) w),  a = exp(g),
// so a token costs one reduction over the state's rows. A wave holds 32 columns of a
// head's state in registers: lane l has columns 4 (l % 8) .. +3 of rows l/8, l/8 + 8,
// ...; a row's 32 columns are one 128-byte line, and the sums over rows end in three
// exchanges between lanes 8, 16 and 32 apart. Bound by the state's bytes: 96 rows of 16 heads
// of 128 x 128 (201 MB read and written) take 35 us, 5.8 TB/s; a single row of 6 heads 6.4 us in
// a graph: a launch and three trips to memory, each of which waits for the one before (the
// slot, the other rows' slots with the state under way, the token).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/hyena.h"
#include "delta.hpp"
#include "plan.hpp"

namespace hy {

using namespace delta;

hyena_status_t delta_check_shape(const hyena_delta_params_t* p, DeltaCall& c) {
    if (!p || p->heads_k < 1 || p->heads_v < 1 || p->dim_k < 1 || p->dim_v < 1) return HYENA_ERR_INVALID_ARG;
    if (p->dtype != HYENA_F32 && p->dtype != HYENA_BF16) return HYENA_ERR_INVALID_ARG;
    if (p->heads_v % p->heads_k) return HYENA_ERR_INVALID_ARG;
    if (p->heads_v > 65535 || p->dim_k % 8 || p->dim_v % 8 || p->dim_k > 128 || p->dim_v > 256)
        return HYENA_ERR_UNSUPPORTED;
    c.p = *p;
    c.bf = p->dtype == HYENA_BF16;
    c.dkp = p->dim_k <= 64 ? 64 : 128;
    c.shape = Shape{};
    c.shape.hk = (int)p->heads_k;
    c.shape.hv = (int)p->heads_v;
    c.shape.group = (int)(p->heads_v / p->heads_k);
    c.shape.dk = (int)p->dim_k;
    c.shape.dv = (int)p->dim_v;
    c.shape.scale = p->scale;
    return HYENA_OK;
}

namespace {

struct StepArgs {
    Shape sh;
    const void *q, *k, *v, *g, *beta;
    float* states;          // [num_states][hv][dk][dv]
    const int32_t* slots;   // [B] or null
    int64_t B, T, num_states;
    void* o;
    int nblk;               // 32-column blocks per head
};

constexpr int kMaxWaves = 4;

// One workgroup per (row, value head) and group of column blocks, one block a wave.
template <bool BF, int DK>
__global__ __launch_bounds__(64 * kMaxWaves) void k_delta_step(StepArgs a) {
    using T = typename Io<BF>::T;
    constexpr int R = DK / 8;  // rows per lane
    __shared__ float lk[DK], lq[DK];
    __shared__ int next_row, seen;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nthreads = blockDim.x;
    const int r0 = lane >> 3, c4 = 4 * (lane & 7);
    int64_t row = blockIdx.x / a.sh.hv;
    const int h = (int)(blockIdx.x % a.sh.hv), hk = h / a.sh.group;
    const int dk = a.sh.dk, dv = a.sh.dv;
    const int cb = (blockIdx.y * (nthreads >> 6) + wave) * 32 + c4;
    const bool cok = cb < dv;
    int64_t slot = row;
    if (a.slots) slot = a.slots[row];
    if (slot < 0 || slot >= a.num_states) {
        // a row without a state: zeros out
        if (cok && r0 == 0)
            for (int64_t t = 0; t < a.T; ++t) {
                T* op = (T*)a.o + ((row * a.T + t) * a.sh.hv + h) * (int64_t)dv + cb;
#pragma unroll
                for (int i = 0; i < 4; ++i) op[i] = (T)0.f;
            }
        return;
    }
    float* sp = a.states + (slot * a.sh.hv + h) * (int64_t)dk * dv + cb;
    f32x4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        S[i] = f32x4{};
        if (cok && r0 + 8 * i < dk) S[i] = *reinterpret_cast<const f32x4*>(sp + (int64_t)(r0 + 8 * i) * dv);
    }
    for (;;) {
        // Rows that name the same slot are successive tokens of it: the workgroup of the
        // first such row takes them in order, the others leave.
        int64_t following = a.B;
        if (a.slots) {
            if (tid == 0) {
                seen = 0;
                next_row = 0x7fffffff;
            }
            __syncthreads();
            int mine = 0x7fffffff, before = 0;
            const bool first = row == (int64_t)(blockIdx.x / a.sh.hv);
            for (int64_t i = (first ? 0 : row + 1) + tid; i < a.B; i += nthreads)
                if (a.slots[i] == (int32_t)slot) {
                    if (i < row) before = 1;
                    if (i > row && (int)i < mine) mine = (int)i;
                }
            if (before) atomicOr(&seen, 1);
            if (mine != 0x7fffffff) atomicMin(&next_row, mine);
            __syncthreads();
            if (seen) return;
            if (next_row != 0x7fffffff) following = next_row;
        }
        for (int64_t t = 0; t < a.T; ++t) {
            const int64_t tok = row * a.T + t;
            const T* qp = (const T*)a.q + tok * a.sh.ldq + (int64_t)hk * dk;
            const T* kp = (const T*)a.k + tok * a.sh.ldk + (int64_t)hk * dk;
            __syncthreads();
            for (int i = tid; i < DK; i += nthreads) {
                lq[i] = i < dk ? (float)qp[i] : 0.f;
                lk[i] = i < dk ? (float)kp[i] : 0.f;
            }
            float v[4] = {};
            if (cok) {
                const T* vp = (const T*)a.v + tok * a.sh.ldv + (int64_t)h * dv + cb;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (float)vp[i];
            }
            const float dec = expf((float)((const T*)a.g)[tok * a.sh.hv + h]);
            const float bet = (float)((const T*)a.beta)[tok * a.sh.hv + h];
            __syncthreads();
            float s[4] = {}, z[4] = {}, kq = 0.f;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float kk = lk[r0 + 8 * i], qq = lq[r0 + 8 * i];
                kq = fmaf(kk, qq, kq);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[j] = fmaf(kk, S[i][j], s[j]);
                    z[j] = fmaf(qq, S[i][j], z[j]);
                }
            }
#pragma unroll
            for (int d = 8; d < 64; d <<= 1) {
                kq += __shfl_xor(kq, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[j] += __shfl_xor(s[j], d);
                    z[j] += __shfl_xor(z[j], d);
                }
            }
            float w[4], o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = bet * (v[j] - dec * s[j]);
                o[j] = a.sh.scale * (dec * z[j] + kq * w[j]);
            }
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float kk = lk[r0 + 8 * i];
#pragma unroll
                for (int j = 0; j < 4; ++j) S[i][j] = fmaf(kk, w[j], dec * S[i][j]);
            }
            if (cok && r0 == 0) {
                T* op = (T*)a.o + (tok * a.sh.hv + h) * (int64_t)dv + cb;
#pragma unroll
                for (int i = 0; i < 4; ++i) op[i] = (T)o[i];
            }
        }
        if (following >= a.B) break;
        row = following;
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (cok && r0 + 8 * i < dk) *reinterpret_cast<f32x4*>(sp + (int64_t)(r0 + 8 * i) * dv) = S[i];
}

// a head's blocks together, so that q, k and the slots are read once for them (one wave a
// workgroup: 36.9 us in place of 34.2 at 96 rows of 16 heads of 128 x 128, the same at 1 to 32)
int step_waves(const StepArgs& a) { return a.nblk < kMaxWaves ? a.nblk : kMaxWaves; }

template <bool BF, int DK>
hipError_t launch_step_t(const StepArgs& a, hipStream_t st) {
    const int64_t rows = a.B * a.sh.hv;
    const int waves = step_waves(a);
    hipLaunchKernelGGL((k_delta_step<BF, DK>), dim3((unsigned)rows, (unsigned)((a.nblk + waves - 1) / waves)),
                       dim3(64 * waves), 0, st, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace hy

extern "C" {

hyena_status_t hyena_delta_step(const hyena_delta_params_t* params, int64_t B, int64_t T,
                                const hyena_delta_inputs_t* in, float* states, int64_t num_states,
                                const int32_t* slots, void* o, hipStream_t stream) {
    using hy::aligned16;
    hy::DeltaCall c;
    if (!in || !states || !o || B < 1 || T < 1 || num_states < 1) return HYENA_ERR_INVALID_ARG;
    if (B > (int64_t(1) << 24) || T > (int64_t(1) << 24) || num_states > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    const hyena_status_t st = hy::delta_check(params, B, B * T, nullptr, in, c);
    if (st != HYENA_OK) return st;
    if (!aligned16(states) || !aligned16(o) || ((uintptr_t)slots & 3u)) return HYENA_ERR_INVALID_ARG;
    if (!slots && num_states < B) return HYENA_ERR_INVALID_ARG;
    hy::StepArgs a{c.shape, in->q, in->k, in->v, in->g, in->beta, states, slots, B, T, num_states, o,
                   (c.shape.dv + 31) / 32};
    if (!hy::delta::fits_launch(B * c.shape.hv, 64 * hy::step_waves(a))) return HYENA_ERR_UNSUPPORTED;
    hipError_t e;
    if (c.bf)
        e = c.dkp == 64 ? hy::launch_step_t<true, 64>(a, stream) : hy::launch_step_t<true, 128>(a, stream);
    else
        e = c.dkp == 64 ? hy::launch_step_t<false, 64>(a, stream) : hy::launch_step_t<false, 128>(a, stream);
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
