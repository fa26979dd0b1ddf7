// Gated linear recurrence, recurrent form: a few tokens of every row against states that
// stay in a pool in device memory (see recurrence.hpp). A workgroup has one row and 512
// channels, two a lane; all of it is fp32. With slots every workgroup looks through all of them for rows that share its
// own: work that grows with the square of the rows. One token of 2048 channels, with slots and with the rows in order (captured):
// 256 rows 4.2 and 3.6 us, 1024 9.1 and 6.7, 4096 44 and 18, 16384 411 and 60.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "recurrence.hpp"

namespace hy {
namespace rec {
namespace {

constexpr int kStepThreads = 256;

struct StepArgs {
    hyena_recurrence_inputs_t in;
    const float* rate;
    float* states;
    const int32_t* slots;
    void* y;
    int64_t B, T, num_states;
    int dim;
};

template <bool BF>
__device__ __forceinline__ void take(const void* base, int64_t e, float (&x)[kVec]) {
    Io<BF>::get(*reinterpret_cast<const typename Io<BF>::Raw*>((const char*)base + e * Io<BF>::kBytes), x);
}
template <bool BF>
__device__ __forceinline__ void put(void* base, int64_t e, const float (&x)[kVec]) {
    *reinterpret_cast<typename Io<BF>::Raw*>((char*)base + e * Io<BF>::kBytes) = Io<BF>::put(x);
}

template <bool BF>
__global__ __launch_bounds__(kStepThreads) void k_rec_step(StepArgs p) {
    __shared__ int next_row, seen;
    const int tid = threadIdx.x;
    const int col = kVec * (blockIdx.y * kStepThreads + tid);
    const bool ok = col < p.dim;
    int64_t row = blockIdx.x;
    const int64_t slot = p.slots ? p.slots[row] : row;
    if (slot < 0 || slot >= p.num_states) {  // a row without a state: zeros out
        const float zero[kVec] = {};
        if (ok)
            for (int64_t t = 0; t < p.T; ++t) put<BF>(p.y, (row * p.T + t) * p.dim + col, zero);
        return;
    }
    float* const sp = p.states + slot * p.dim + col;
    float h[kVec] = {}, rate[kVec] = {};
    if (ok) {
        const float2 v = *reinterpret_cast<const float2*>(sp);
        h[0] = v.x;
        h[1] = v.y;
#pragma unroll
        for (int j = 0; j < kVec; ++j) rate[j] = p.rate[col + j];
    }
    for (;;) {
        // Rows that name the same slot are successive tokens of it: the workgroup of the
        // first such row takes them in order, the others leave.
        int64_t following = p.B;
        if (p.slots) {
            if (tid == 0) {
                seen = 0;
                next_row = 0x7fffffff;
            }
            __syncthreads();
            int mine = 0x7fffffff, before = 0;
            const bool first = row == (int64_t)blockIdx.x;
            for (int64_t i = (first ? 0 : row + 1) + tid; i < p.B; i += kStepThreads)
                if (p.slots[i] == (int32_t)slot) {
                    if (i < row) before = 1;
                    if (i > row && (int)i < mine) mine = (int)i;
                }
            if (before) atomicOr(&seen, 1);
            if (mine != 0x7fffffff) atomicMin(&next_row, mine);
            __syncthreads();
            const int stop = seen, next = next_row;
            __syncthreads();  // read by all before the next round clears them
            if (stop) return;
            if (next != 0x7fffffff) following = next;
        }
        if (ok)
            for (int64_t t = 0; t < p.T; ++t) {
                const int64_t tok = row * p.T + t;
                float x[kVec], r[kVec], i[kVec];
                take<BF>(p.in.x, tok * p.in.ldx + col, x);
                take<BF>(p.in.r, tok * p.in.ldr + col, r);
                take<BF>(p.in.i, tok * p.in.ldi + col, i);
                float w[kVec], a[kVec], q[kVec];
#pragma unroll
                for (int j = 0; j < kVec; ++j) w[j] = rate[j] * sigmoid(r[j]);
                decay(w, false, a, q);
#pragma unroll
                for (int j = 0; j < kVec; ++j) h[j] = fmaf(a[j], h[j], __builtin_amdgcn_sqrtf(q[j]) * sigmoid(i[j]) * x[j]);
                put<BF>(p.y, tok * p.dim + col, h);
            }
        if (following >= p.B) break;
        row = following;
    }
    if (ok) *reinterpret_cast<float2*>(sp) = float2{h[0], h[1]};
}

}  // namespace
}  // namespace rec
}  // namespace hy

extern "C" {

hyena_status_t hyena_recurrence_step(const hyena_recurrence_params_t* params, int64_t B, int64_t T,
                                     const hyena_recurrence_inputs_t* in, float* states, int64_t num_states,
                                     const int32_t* slots, void* y, hipStream_t stream) {
    using namespace hy;
    rec::Call c;
    if (!in || !states || !y || B < 1 || T < 1 || num_states < 1) return HYENA_ERR_INVALID_ARG;
    if (B > (int64_t(1) << 24) || T > (int64_t(1) << 24) || num_states > 0x7fffffff) return HYENA_ERR_UNSUPPORTED;
    const hyena_status_t st = rec::check(params, B, B * T, nullptr, in, c, false);
    if (st != HYENA_OK) return st;
    if (!aligned16(states) || !aligned16(y) || ((uintptr_t)slots & 3u)) return HYENA_ERR_INVALID_ARG;
    if (!slots && num_states < B) return HYENA_ERR_INVALID_ARG;
    const int64_t wide = rec::kVec * rec::kStepThreads, blocks = (params->dim + wide - 1) / wide;
    if (B * blocks >= (int64_t(1) << 32) / rec::kStepThreads) return HYENA_ERR_UNSUPPORTED;
    rec::StepArgs a{c.in, params->rate, states, slots, y, B, T, num_states, (int)params->dim};
    const dim3 grid((unsigned)B, (unsigned)blocks);
    if (c.bf)
        hipLaunchKernelGGL(rec::k_rec_step<true>, grid, dim3(rec::kStepThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(rec::k_rec_step<false>, grid, dim3(rec::kStepThreads), 0, stream, a);
    return hipGetLastError() == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
