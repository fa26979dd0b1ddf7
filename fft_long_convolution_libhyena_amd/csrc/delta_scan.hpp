// The state scan of the gated delta rule: one workgroup of four waves carries 16 NT
// columns of one (sequence, value head)'s state through its chunks.
//
// Wave w owns tokens 16w .. 16w+15 of a chunk (K S, Q S, T e, P u) and rows
// DK/4 w .. of the state, which stay in its registers in fp32. Every operand element
// on the left of a product is thus read by exactly one wave, straight from memory into
// registers; the right-hand operands (the state's parts, the residual e, the written
// values u) pass between the waves through LDS as fragments, with three barriers a
// chunk. The next chunk's left operands are loaded as soon as this chunk's are used;
// the barriers leave those loads in flight, and no load is conditional.
#pragma once
#include "delta.hpp"

namespace hy {
namespace delta {

struct ScanArgs {
    Seqs seqs;
    Shape sh;
    const void *q, *k, *v;
    Prep prep;
    const float* s_in;  // [N][hv][dk][dv] or null (zeros)
    float* s_out;       // likewise, or null
    void* o;            // [tokens][hv][dv] (outputs)
    void* s0;           // [slot][hv][dk][dv] state before every chunk (for the backward)
    void* u;            // [tokens][hv][dv] written values (for the backward)
    int nblk;           // column blocks per head
};

enum { kScanOut = 0, kScanKeep = 1 };

template <bool BF, int DK, int NT>
struct ScanLds {
    using IO = Io<BF>;
    alignas(16) __bf16 s[DK / 32][NT][IO::NS][512];
    alignas(16) __bf16 e[2][NT][IO::NS][512];
    alignas(16) __bf16 u[2][NT][IO::NO][512];
    alignas(16) __bf16 ku[2][NT][IO::NS][512];
};

template <bool BF, int DK, int NT, int MODE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 2))) void k_delta_scan(ScanArgs a) {
    using IO = Io<BF>;
    using T = typename IO::T;
    constexpr int KS = DK / 32, MT = DK / 64;
    constexpr int NS = IO::NS, NP = IO::NP, NO = IO::NO;
    constexpr uint32_t E = sizeof(T);
    extern __shared__ __align__(16) unsigned char lds_raw[];
    ScanLds<BF, DK, NT>& l = *reinterpret_cast<ScanLds<BF, DK, NT>*>(lds_raw);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, col = lane & 15;
    // column blocks of one head sit 8 workgroups apart, so that they land on one XCD
    // and share its L2 for the head's operands
    const int64_t bid = blockIdx.x;
    const int64_t pair = bid / (8 * a.nblk) * 8 + (bid & 7);
    const int blk = (int)(bid / 8 % a.nblk);
    const int hv = a.sh.hv;
    if (pair >= a.seqs.N * hv) return;
    const int64_t n = pair / hv;
    const int h = (int)(pair % hv), hk = h / a.sh.group;
    const Range rr = seq_range(a.seqs, n);
    const int64_t first = uniform64(rr.first), len = uniform64(rr.len), slot0 = uniform64(rr.slot0);
    const int64_t nch = (len + kC - 1) / kC;
    const int dk = a.sh.dk, dv = a.sh.dv;
    const int c0 = blk * 16 * NT + NT * col;  // this lane's first column
    const bool cok = c0 < dv;

    f32x4 S[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 16 * (wave * MT + m) + 4 * g + i;
            float x[NT];
            load_cols<NT>(a.s_in + ((n * hv + h) * dk + k) * dv + c0, a.s_in && k < dk && cok, x);
#pragma unroll
            for (int j = 0; j < NT; ++j) S[m][j][i] = x[j];
        }

    const int row = 16 * wave + col;     // token of this lane's operand rows
    const int drow = 16 * wave + 4 * g;  // first of this lane's four result rows
    const uint32_t ldk = (uint32_t)a.sh.ldk * E, ldq = (uint32_t)a.sh.ldq * E, ldv = (uint32_t)a.sh.ldv * E;
    const uint32_t ldo = (uint32_t)(hv * dv) * E;
    uint32_t koff[KS], qoff[KS], voff[4], ooff[4], soff[MT][4];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const uint32_t k = 32 * s + 8 * g;
        koff[s] = (int)k < dk ? row * ldk + k * E : kNoElem;
        qoff[s] = (int)k < dk ? row * ldq + k * E : kNoElem;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        voff[i] = cok ? (drow + i) * ldv + c0 * E : kNoElem;
        ooff[i] = cok ? (drow + i) * ldo + c0 * E : kNoElem;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = 16 * (wave * MT + m) + 4 * g + i;
            soff[m][i] = cok && k < dk ? (uint32_t)(k * dv + c0) * E : kNoElem;
        }
    const T* kbase = (const T*)a.k + first * a.sh.ldk + (int64_t)hk * dk;
    const T* qbase = (const T*)a.q + first * a.sh.ldq + (int64_t)hk * dk;
    const T* vbase = (const T*)a.v + first * a.sh.ldv + (int64_t)h * dv;
    T* obase = (T*)(MODE == kScanOut ? a.o : a.u) + (first * hv + h) * (int64_t)dv;

    Raw<BF> K[KS], Q[KS], KT[MT][2];
    Frag<NS> Tf[2];
    Frag<NP> Pf[2];
    Cols<BF, NT> V[4];
    f32x4 gam, kap, bet;
    float glast = 0.f;
    auto load_k = [&](int64_t c) {
        const RowBuf b = row_buf(kbase + c * kC * a.sh.ldk, len - c * kC, ldk, dk * E);
#pragma unroll
        for (int s = 0; s < KS; ++s) buf_raw(b, koff[s], K[s]);
    };
    auto load_q = [&](int64_t c) {
        const RowBuf b = row_buf(qbase + c * kC * a.sh.ldq, len - c * kC, ldq, dk * E);
#pragma unroll
        for (int s = 0; s < KS; ++s) buf_raw(b, qoff[s], Q[s]);
    };
    auto load_v = [&](int64_t c) {
        const RowBuf b = row_buf(vbase + c * kC * a.sh.ldv, len - c * kC, ldv, dv * E);
#pragma unroll
        for (int i = 0; i < 4; ++i) buf_cols<BF, NT>(b, voff[i], V[i]);
    };
    auto load_sc = [&](int64_t c) {
        const float* sc = a.prep.sc + ((slot0 + c) * hv + h) * 3 * kC;
        gam = *reinterpret_cast<const f32x4*>(sc + drow);
        kap = *reinterpret_cast<const f32x4*>(sc + kC + drow);
        bet = *reinterpret_cast<const f32x4*>(sc + 2 * kC + drow);
        glast = sc[kC - 1];
    };
    // every fragment of row tile `wave`: one step for tiles 0 and 1 (read twice, so
    // that no load is conditional), two below
    const int f0 = lower_frag(wave, 0), f1 = lower_frag(wave, wave >= 2 ? 1 : 0);
    auto load_t = [&](int64_t c) {
        const __bf16* p = a.prep.t + ((slot0 + c) * hv + h) * kTri * NS * 512;
        Tf[0] = get_frag<NS>(p + f0 * NS * 512, 512, lane);
        Tf[1] = get_frag<NS>(p + f1 * NS * 512, 512, lane);
    };
    auto load_p = [&](int64_t c) {
        const __bf16* p = a.prep.p + ((slot0 + c) * hv + h) * kTri * NP * 512;
        Pf[0] = get_frag<NP>(p + f0 * NP * 512, 512, lane);
        Pf[1] = get_frag<NP>(p + f1 * NP * 512, 512, lane);
    };
    auto load_kt = [&](int64_t c) {
        const T* p = (const T*)a.prep.kt + ((slot0 + c) * a.sh.hk + hk) * (DK / 16) * 1024 + lane * 8;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int s = 0; s < 2; ++s) KT[m][s] = load_raw(p + ((wave * MT + m) * 2 + s) * 512, true);
    };
    auto put_state = [&]() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int t = wave * MT + m;
                const float x[4] = {S[m][j][0], S[m][j][1], S[m][j][2], S[m][j][3]};
                put_rows<NS>(&l.s[t >> 1][j][0][0], 512, t & 1, lane, x);
            }
    };
    // outputs of chunk c from Q S and the fragments of u, one chunk late: these
    // products run while the next chunk's first fragments come from LDS
    f32x4 qs[NT];
    Frag<NO> uf[2][NT];
    auto finish = [&](int64_t c) {
        f32x4 o1[NT] = {};
        mma_each(Pf[0], uf[0], qs);
        if (wave >= 2) mma_each(Pf[1], uf[1], o1);
        const RowBuf b = row_buf(obase + c * kC * hv * (int64_t)dv, len - c * kC, ldo, dv * E);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) x[j] = a.sh.scale * (qs[j][i] + o1[j][i]);
            buf_store<BF, NT>(b, ooff[i], x);
        }
    };
    if (nch > 0) {
        load_k(0);
        load_v(0);
        load_sc(0);
        if (MODE == kScanOut) load_q(0);
        load_t(0);
        load_kt(0);
        if (MODE == kScanOut) load_p(0);
        put_state();
    }
    for (int64_t c = 0; c < nch; ++c) {
        const int64_t nx = c + 1 < nch ? c + 1 : c;  // the last chunk loads itself again
        if (MODE == kScanKeep) {
            const RowBuf b = __builtin_amdgcn_make_buffer_rsrc(
                (T*)a.s0 + ((slot0 + c) * hv + h) * (int64_t)dk * dv, 0, (int)(dk * dv * E), 0x00020000);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) x[j] = S[m][j][i];
                    buf_store<BF, NT>(b, soff[m][i], x);
                }
        }
        lds_barrier();  // the state's fragments are in place
        Frag<NS> sf[KS][NT];
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j) sf[s][j] = get_frag<NS>(&l.s[s][j][0][0], 512, lane);
        __builtin_amdgcn_sched_barrier(0);
        if (MODE == kScanOut && c > 0) {
            finish(c - 1);
            load_p(c);
        }
        f32x4 ks[NT] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) mma_each(to_frag(K[s]), sf[s], ks);
        load_k(nx);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = bet[i] * (col_value(V[i], j) - gam[i] * ks[j][i]);
            put_rows<NS>(&l.e[wave >> 1][j][0][0], 512, wave & 1, lane, x);
        }
        load_v(nx);
        lds_barrier();  // e
        Frag<NS> ef[2][NT];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j) ef[s][j] = get_frag<NS>(&l.e[s][j][0][0], 512, lane);
        __builtin_amdgcn_sched_barrier(0);
        if (MODE == kScanOut) {  // while e's fragments arrive
#pragma unroll
            for (int j = 0; j < NT; ++j) qs[j] = f32x4{};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                Frag<NO> so[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) so[j] = first_parts<NO>(sf[s][j]);
                mma_each(to_frag(Q[s]), so, qs);
            }
            load_q(nx);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) qs[j][i] *= gam[i];
        }
        f32x4 u[NT] = {}, u1[NT] = {};
        mma_each(Tf[0], ef[0], u);
        if (wave >= 2) mma_each(Tf[1], ef[1], u1);
        load_t(nx);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = u[j][i] + u1[j][i];
                y[i] = kap[i] * x[i];
                u[j][i] = x[i];
            }
            if (MODE == kScanOut) put_rows<NO>(&l.u[wave >> 1][j][0][0], 512, wave & 1, lane, x);
            put_rows<NS>(&l.ku[wave >> 1][j][0][0], 512, wave & 1, lane, y);
        }
        if (MODE == kScanKeep) {
            const RowBuf b = row_buf(obase + c * kC * hv * (int64_t)dv, len - c * kC, ldo, dv * E);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) x[j] = u[j][i];
                buf_store<BF, NT>(b, ooff[i], x);
            }
        }
        const float gl = glast;
        load_sc(nx);
        lds_barrier();  // u
        Frag<NS> kf[2][NT];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j) kf[s][j] = get_frag<NS>(&l.ku[s][j][0][0], 512, lane);
        if (MODE == kScanOut)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < NT; ++j) uf[s][j] = get_frag<NO>(&l.u[s][j][0][0], 512, lane);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[m][j][i] *= gl;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_each(to_frag(KT[m][s]), kf[s], S[m]);
        load_kt(nx);
        put_state();
    }
    if (MODE == kScanOut && nch > 0) finish(nch - 1);
    if (a.s_out)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = 16 * (wave * MT + m) + 4 * g + i;
                float x[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) x[j] = S[m][j][i];
                if (cok && k < dk) store_cols<NT>(a.s_out + ((n * hv + h) * dk + k) * dv + c0, x);
            }
}

}  // namespace delta
}  // namespace hy
