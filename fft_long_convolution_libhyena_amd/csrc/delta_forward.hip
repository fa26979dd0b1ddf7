// Gated delta rule, forward over whole sequences (chunked): argument checks,
// workspace layout and launches of the preparation and the state scan.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/hyena.h"
#include "delta.hpp"
#include "delta_prep.hpp"
#include "delta_scan.hpp"
#include "plan.hpp"

namespace hy {

using namespace delta;

hyena_status_t delta_check(const hyena_delta_params_t* p, int64_t N, int64_t tokens, const int64_t* seq_start,
                           const hyena_delta_inputs_t* in, DeltaCall& c) {
    const hyena_status_t st = delta_check_shape(p, c);
    if (st != HYENA_OK) return st;
    if (N < 1 || tokens < 0 || (!seq_start && tokens % N)) return HYENA_ERR_INVALID_ARG;
    if (!(p->scale >= -3.402823466e38f && p->scale <= 3.402823466e38f)) return HYENA_ERR_INVALID_ARG;
    if (((uintptr_t)seq_start & 7u) != 0) return HYENA_ERR_INVALID_ARG;
    if (p->heads_v * p->dim_v > kMaxLd || p->heads_k * p->dim_k > kMaxLd) return HYENA_ERR_UNSUPPORTED;
    if (in) {
        c.in = *in;
        const void* rows[] = {in->q, in->k, in->v};
        for (const void* x : rows)
            if (tokens > 0 && (!x || !aligned16(x))) return HYENA_ERR_INVALID_ARG;
        const void* gates[] = {in->g, in->beta};  // read one element at a time
        for (const void* x : gates)
            if (tokens > 0 && (!x || ((uintptr_t)x & (c.bf ? 1u : 3u)))) return HYENA_ERR_INVALID_ARG;
        const int64_t v = c.bf ? 8 : 4;  // elements per 16 bytes: operand rows start on 16 bytes
        const int64_t ld[] = {in->ldq, in->ldk, in->ldv};
        const int64_t width[] = {p->heads_k * p->dim_k, p->heads_k * p->dim_k, p->heads_v * p->dim_v};
        for (int i = 0; i < 3; ++i)
            if (ld[i] < width[i] || ld[i] % v || ld[i] > kMaxLd) return HYENA_ERR_INVALID_ARG;
        c.shape.ldq = in->ldq;
        c.shape.ldk = in->ldk;
        c.shape.ldv = in->ldv;
    }
    if (N > kMaxSeqs || tokens > kMaxTokens) return HYENA_ERR_UNSUPPORTED;
    c.seqs.start = seq_start;
    c.seqs.N = N;
    c.seqs.tokens = tokens;
    c.seqs.T = seq_start ? 0 : tokens / N;
    c.seqs.cpt = (c.seqs.T + kC - 1) / kC;
    c.slots = tokens < 1 ? 0 : seq_start ? tokens / kC + N : N * c.seqs.cpt;
    // one workgroup per (slot, value head) and per column block of a (sequence, value head)
    if (c.slots * p->heads_v > (int64_t(1) << 30) || N * p->heads_v > (int64_t(1) << 26)) return HYENA_ERR_UNSUPPORTED;
    return HYENA_OK;
}

hyena_status_t delta_check_launches(const DeltaCall& c) {
    const int w = scan_columns(c.bf);
    const int64_t pairs = (c.seqs.N * c.shape.hv + 7) / 8 * 8;
    return fits_launch(c.slots, kThreads) && fits_launch(pairs * ((c.shape.dv + w - 1) / w), scan_threads(c.bf))
               ? HYENA_OK
               : HYENA_ERR_UNSUPPORTED;
}

size_t delta_prep_layout(const DeltaCall& c, bool bwd, unsigned char* base, Prep& o) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char* p = base ? base + at : nullptr;
        at += (bytes + 255) & ~(size_t)255;
        return p;
    };
    const size_t pv = (size_t)c.slots * c.shape.hv;
    o = Prep{};
    o.rec = take(pv * (c.bf ? Rec<true>::bytes : Rec<false>::bytes));
    if (bwd) o.back = take(pv * (c.bf ? Rec<true>::back : Rec<false>::back));
    return at;
}

namespace {

constexpr int kClearMost = 8;
struct ClearArgs {
    const int64_t* start;
    int64_t N, tokens;
    unsigned char* p[kClearMost];
    int64_t bytes[kClearMost];
};
// One array a grid row, both ranges of it as 16-byte pieces where they are aligned to them.
// Without rows to clear it is a launch (2 us); a fill of every output would be up to 90 us
// beside a backward of 1200 (8 sequences of 8192 tokens).
__global__ __launch_bounds__(256) void k_clear_rows(ClearArgs a) {
    int64_t lo = a.start[0], hi = a.start[a.N];
    lo = lo < 0 ? 0 : lo < a.tokens ? lo : a.tokens;
    hi = hi < lo ? lo : hi < a.tokens ? hi : a.tokens;
    unsigned char* const p = a.p[blockIdx.y];
    const int64_t row = a.bytes[blockIdx.y], step = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool wide = !(((uintptr_t)p | (uintptr_t)row) & 15u);
    auto clear = [&](unsigned char* q, int64_t n) {
        if (wide)
            for (int64_t i = first; i < n / 16; i += step) *reinterpret_cast<u32x4*>(q + 16 * i) = u32x4{};
        else
            for (int64_t i = first; i < n / 2; i += step) *reinterpret_cast<uint16_t*>(q + 2 * i) = 0;
    };
    clear(p, lo * row);
    clear(p + hi * row, (a.tokens - hi) * row);
}

template <bool BF, int DK, bool BWD>
hipError_t launch_prep_t(const DeltaCall& c, const Prep& o, hipStream_t st) {
    using L = PrepLds<BF, DK>;
    PrepArgs a{c.seqs, c.shape, c.in.q, c.in.k, c.in.g, c.in.beta, o};
    if (sizeof(L) > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute((const void*)k_delta_prep<BF, DK, BWD>,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(L));
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_delta_prep<BF, DK, BWD>), dim3((unsigned)c.slots, (unsigned)c.shape.hv), dim3(kThreads),
                       sizeof(L), st, a);
    return hipGetLastError();
}

template <bool BF, int DK, int MODE>
hipError_t launch_scan_t(const DeltaCall& c, ScanArgs a, hipStream_t st) {
    using Cfg = ScanCfg<BF, DK, MODE>;
    constexpr int lds = (int)sizeof(typename Cfg::Lds);
    static_assert(Cfg::ENDS || (16 * Cfg::NB == scan_columns(BF) && Cfg::threads <= scan_threads(BF)),
                  "what delta_check_launches takes them for (the ends run on few workgroups)");
    const int w = 16 * Cfg::NB;
    a.nbv = (c.shape.dv + w - 1) / w;
    a.nblk = a.nbv + (Cfg::ENDS ? (DK + w - 1) / w : 0);
    a.nb16 = (c.shape.dv + 15) / 16;
    const int64_t pairs = (a.pieces.slots * c.shape.hv + 7) / 8 * 8;
    const hipError_t e = hipFuncSetAttribute((const void*)k_delta_scan<BF, DK, MODE>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_delta_scan<BF, DK, MODE>), dim3((unsigned)(pairs * a.nblk)), dim3(Cfg::threads), lds, st, a);
    return hipGetLastError();
}

template <bool BF, int DK>
hipError_t launch_scans_t(const DeltaCall& c, bool keep, const ScanArgs& a, hipStream_t st) {
    if (a.pieces.len) {
        const hipError_t e = launch_scan_t<BF, DK, kScanEnds>(c, a, st);
        if (e != hipSuccess) return e;
    }
    return keep ? launch_scan_t<BF, DK, kScanKeep>(c, a, st) : launch_scan_t<BF, DK, kScanOut>(c, a, st);
}

}  // namespace

Pieces delta_pieces(const DeltaCall& c) {
    Pieces p{};
    p.slots = c.seqs.N;
    // piece slots whose workgroups, of the scan or of the ends, all run at once (one a CU)
    const int64_t wn = c.bf ? 32 : 16, we = c.bf ? 64 : 48, dv = c.shape.dv;
    const int64_t scan = (dv + wn - 1) / wn, ends = (dv + we - 1) / we + (c.dkp + we - 1) / we;
    const int64_t room = kCus / (c.shape.hv * (scan > ends ? scan : ends)), N = c.seqs.N;
    if (room < 3 * N) return p;
    const int64_t chunks = c.seqs.start ? (c.seqs.tokens + kC - 1) / kC : c.seqs.cpt;  // of one sequence at most
    const int64_t fit = c.seqs.start ? room - N + (N == 1) : room / N;
    const int64_t len = (chunks + fit - 1) / fit;
    p.len = len < kMinPiece ? kMinPiece : len;
    if (chunks <= 3 * p.len) {
        p.len = 0;
        return p;
    }
    p.per = (chunks + p.len - 1) / p.len;
    p.slots = c.seqs.start ? c.seqs.tokens / (kC * p.len) + N : N * p.per;
    return p;
}

size_t delta_pieces_layout(const DeltaCall& c, bool bwd, unsigned char* base, Pieces& o) {
    o = delta_pieces(c);
    if (!o.len) return 0;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char* p = base ? base + at : nullptr;
        at += (bytes + 255) & ~(size_t)255;
        return p;
    };
    const size_t heads = (size_t)o.slots * c.shape.hv;
    const size_t m = heads * c.dkp * c.dkp * 2 * (c.bf ? Io<true>::NS : Io<false>::NS);
    o.b = (float*)take(heads * ((c.shape.dv + 15) / 16 * 16) * c.dkp * sizeof(float));
    o.m = take(m);
    if (bwd) o.mt = take(m);
    return at;
}

hipError_t delta_prep(const DeltaCall& c, bool bwd, const Prep& o, hipStream_t st) {
    if (c.slots < 1 || c.seqs.tokens < 1) return hipSuccess;
    if (c.bf) {
        if (c.dkp == 64) return bwd ? launch_prep_t<true, 64, true>(c, o, st) : launch_prep_t<true, 64, false>(c, o, st);
        return bwd ? launch_prep_t<true, 128, true>(c, o, st) : launch_prep_t<true, 128, false>(c, o, st);
    }
    if (c.dkp == 64) return bwd ? launch_prep_t<false, 64, true>(c, o, st) : launch_prep_t<false, 64, false>(c, o, st);
    return bwd ? launch_prep_t<false, 128, true>(c, o, st) : launch_prep_t<false, 128, false>(c, o, st);
}

hipError_t delta_scan(const DeltaCall& c, bool keep, const ScanArgs& a, hipStream_t st) {
    if (c.bf) return c.dkp == 64 ? launch_scans_t<true, 64>(c, keep, a, st) : launch_scans_t<true, 128>(c, keep, a, st);
    return c.dkp == 64 ? launch_scans_t<false, 64>(c, keep, a, st) : launch_scans_t<false, 128>(c, keep, a, st);
}

}  // namespace hy

extern "C" {

size_t hyena_delta_workspace_bytes(const hyena_delta_params_t* params, int64_t N, int64_t tokens,
                                   const int64_t* seq_start) {
    hy::DeltaCall c;
    if (hy::delta_check(params, N, tokens, seq_start, nullptr, c) != HYENA_OK || hy::delta_check_launches(c) != HYENA_OK) return 0;
    hy::delta::Prep o;
    hy::delta::Pieces p;
    return hy::delta_prep_layout(c, false, nullptr, o) + hy::delta_pieces_layout(c, false, nullptr, p);
}

hyena_status_t hyena_delta_clear_rows(int64_t N, int64_t tokens, const int64_t* seq_start, int count,
                                      void* const* arrays, const int64_t* row_bytes, hipStream_t stream) {
    if (N < 1 || tokens < 0 || tokens > hy::delta::kMaxTokens || !seq_start || ((uintptr_t)seq_start & 7u) || count < 1 ||
        count > hy::kClearMost || !arrays || !row_bytes)
        return HYENA_ERR_INVALID_ARG;
    hy::ClearArgs a{seq_start, N, tokens, {}, {}};
    for (int i = 0; i < count; ++i) {
        if ((tokens > 0 && !arrays[i]) || ((uintptr_t)arrays[i] & 1u) || row_bytes[i] < 2 || row_bytes[i] % 2 ||
            row_bytes[i] > (int64_t(1) << 31))
            return HYENA_ERR_INVALID_ARG;
        a.p[i] = (unsigned char*)arrays[i];
        a.bytes[i] = row_bytes[i];
    }
    if (tokens < 1) return HYENA_OK;
    hipLaunchKernelGGL(hy::k_clear_rows, dim3(256, (unsigned)count), dim3(256), 0, stream, a);
    return hipGetLastError() == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

hyena_status_t hyena_delta_forward(const hyena_delta_params_t* params, int64_t N, int64_t tokens,
                                   const int64_t* seq_start, const hyena_delta_inputs_t* in, const float* state_in,
                                   void* o, float* state_out, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    using hy::aligned16;
    hy::DeltaCall c;
    if (!in) return HYENA_ERR_INVALID_ARG;
    hyena_status_t st = hy::delta_check(params, N, tokens, seq_start, in, c);
    if (st == HYENA_OK) st = hy::delta_check_launches(c);
    if (st != HYENA_OK) return st;
    if ((tokens > 0 && !o) || !aligned16(o) || !aligned16(state_in) || !aligned16(state_out))
        return HYENA_ERR_INVALID_ARG;
    hy::delta::ScanArgs a{};
    const size_t prep = hy::delta_prep_layout(c, false, (unsigned char*)workspace, a.prep);
    const size_t need =
        prep + hy::delta_pieces_layout(c, false, workspace ? (unsigned char*)workspace + prep : nullptr, a.pieces);
    if (need && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return HYENA_ERR_INVALID_ARG;
    hipError_t e = hy::delta_prep(c, false, a.prep, stream);
    if (e != hipSuccess) return HYENA_ERR_DEVICE;
    a.seqs = c.seqs;
    a.sh = c.shape;
    a.q = in->q;
    a.k = in->k;
    a.v = in->v;
    a.s_in = state_in;
    a.s_out = state_out;
    a.o = o;
    e = hy::delta_scan(c, false, a, stream);
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
