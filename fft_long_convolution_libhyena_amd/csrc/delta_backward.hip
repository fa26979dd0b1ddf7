// Gated delta rule, backward over whole sequences: the preparation and the forward's
// state scan again (keeping the state before every chunk and the written values), the
// reverse scan, and the chunk-parallel gradients.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hyena.h"
#include "delta.hpp"
#include "delta_grad.hpp"
#include "delta_rev.hpp"
#include "plan.hpp"

namespace hy {

using namespace delta;

namespace {

struct BackLayout {
    Prep prep;
    Pieces pieces;
    void *s0, *ds1, *u, *r;
    size_t bytes;
};

BackLayout back_layout(const DeltaCall& c, unsigned char* base) {
    BackLayout b{};
    size_t at = delta_prep_layout(c, true, base, b.prep);
    auto take = [&](size_t bytes) {
        void* p = base ? base + at : nullptr;
        at += (bytes + 255) & ~(size_t)255;
        return p;
    };
    const size_t cols = (size_t)c.slots * c.shape.hv * ((c.shape.dv + 15) / 16 * 16) * (c.bf ? 3 : 4);  // as Kept
    const size_t states = cols * c.dkp, rows = cols * kC;
    b.s0 = take(states);
    b.ds1 = take(states);
    b.u = take(rows);
    b.r = take(rows);
    b.bytes = at + delta_pieces_layout(c, true, base ? base + at : nullptr, b.pieces);
    return b;
}

template <bool BF, int DK, bool ENDS>
hipError_t launch_rev_t(const DeltaCall& c, RevArgs a, hipStream_t st) {
    using Cfg = RevCfg<BF, DK>;
    constexpr int lds = (int)sizeof(typename Cfg::Lds);
    static_assert(lds <= 160 * 1024, "LDS of a CU");
    static_assert(16 * Cfg::NB == scan_columns(BF) && Cfg::threads <= scan_threads(BF), "what delta_check_launches takes it for");
    a.nblk = (c.shape.dv + 16 * Cfg::NB - 1) / (16 * Cfg::NB);
    a.nb16 = (c.shape.dv + 15) / 16;
    const int64_t pairs = (a.pieces.slots * c.shape.hv + 7) / 8 * 8;
    const hipError_t e =
        hipFuncSetAttribute((const void*)k_delta_rev<BF, DK, ENDS>, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_delta_rev<BF, DK, ENDS>), dim3((unsigned)(pairs * a.nblk)), dim3(Cfg::threads), lds, st, a);
    return hipGetLastError();
}

template <bool BF, int DK, bool SHARED>
hipError_t launch_grad_t(const DeltaCall& c, const GradArgs& a, hipStream_t st) {
    constexpr int lds = (int)sizeof(GradLds<BF, DK>);
    static_assert(lds <= (BF ? 80 : 160) * 1024, "two workgroups a CU in bf16");
    const hipError_t e =
        hipFuncSetAttribute((const void*)k_delta_grad<BF, DK, SHARED>, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_delta_grad<BF, DK, SHARED>), dim3((unsigned)c.slots, (unsigned)c.shape.hk), dim3(kThreads), lds, st,
                       a);
    return hipGetLastError();
}

template <bool BF, int DK>
hipError_t launch_back_t(const DeltaCall& c, const RevArgs& r, const GradArgs& g, hipStream_t st) {
    hipError_t e = hipSuccess;
    if (r.pieces.len) e = launch_rev_t<BF, DK, true>(c, r, st);
    if (e == hipSuccess) e = launch_rev_t<BF, DK, false>(c, r, st);
    if (e != hipSuccess || c.seqs.tokens < 1) return e;
    return c.shape.group > 1 ? launch_grad_t<BF, DK, true>(c, g, st) : launch_grad_t<BF, DK, false>(c, g, st);
}

}  // namespace
}  // namespace hy

extern "C" {

size_t hyena_delta_backward_workspace_bytes(const hyena_delta_params_t* params, int64_t N, int64_t tokens,
                                            const int64_t* seq_start) {
    hy::DeltaCall c;
    if (hy::delta_check(params, N, tokens, seq_start, nullptr, c) != HYENA_OK || hy::delta_check_launches(c) != HYENA_OK) return 0;
    return hy::back_layout(c, nullptr).bytes;
}

hyena_status_t hyena_delta_backward(const hyena_delta_params_t* params, int64_t N, int64_t tokens,
                                    const int64_t* seq_start, const hyena_delta_inputs_t* in, const float* state_in,
                                    const void* dout, const float* dstate_out, void* dq, void* dk, void* dv, void* dg,
                                    void* dbeta, float* dstate_in, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream) {
    using hy::aligned16;
    hy::DeltaCall c;
    if (!in) return HYENA_ERR_INVALID_ARG;
    hyena_status_t st = hy::delta_check(params, N, tokens, seq_start, in, c);
    if (st == HYENA_OK) st = hy::delta_check_launches(c);
    if (st != HYENA_OK) return st;
    const void* need_rows[] = {dout, dq, dk, dv, dg, dbeta};
    for (const void* p : need_rows)
        if ((tokens > 0 && !p) || !aligned16(p)) return HYENA_ERR_INVALID_ARG;
    if (!aligned16(state_in) || !aligned16(dstate_out) || !aligned16(dstate_in)) return HYENA_ERR_INVALID_ARG;
    const hy::BackLayout b = hy::back_layout(c, (unsigned char*)workspace);
    if (b.bytes && (!workspace || workspace_bytes < b.bytes)) return HYENA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return HYENA_ERR_INVALID_ARG;
    if (hy::delta_prep(c, true, b.prep, stream) != hipSuccess) return HYENA_ERR_DEVICE;
    if (c.slots > 0 && tokens > 0) {
        hy::delta::ScanArgs f{};
        f.seqs = c.seqs;
        f.sh = c.shape;
        f.k = in->k;
        f.v = in->v;
        f.prep = b.prep;
        f.s_in = state_in;
        f.s0 = b.s0;
        f.u = b.u;
        f.pieces = b.pieces;
        if (hy::delta_scan(c, true, f, stream) != hipSuccess) return HYENA_ERR_DEVICE;
    }
    hy::delta::RevArgs r{c.seqs, c.shape, in->q, in->k, b.prep, dout, dstate_out, dstate_in, b.ds1, b.r, b.pieces, 0, 0};
    hy::delta::GradArgs g{c.seqs, c.shape, in->q, in->k, in->g, in->beta, dout, b.s0, b.ds1, b.u, b.r, dq, dk, dv, dg, dbeta};
    hipError_t e;
    if (c.bf)
        e = c.dkp == 64 ? hy::launch_back_t<true, 64>(c, r, g, stream) : hy::launch_back_t<true, 128>(c, r, g, stream);
    else
        e = c.dkp == 64 ? hy::launch_back_t<false, 64>(c, r, g, stream) : hy::launch_back_t<false, 128>(c, r, g, stream);
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
