// The state scan of the gated delta rule: one workgroup of four waves carries 16 NT
// columns of one (sequence, value head)'s state through its chunks.
//
// Wave w owns tokens 16w .. 16w+15 of a chunk (K S, Q S, T e, P u) and rows
// DK/4 w .. of the state, which stay in its registers in fp32. Every operand element
// on the left of a product is thus read by exactly one wave, straight from memory into
// registers; the right-hand operands (the state's parts, the residual e, the written
// values u) pass between the waves through LDS as fragments, with three barriers a
// chunk. The next chunk's left operands are loaded as soon as this chunk's are used;
// the barriers leave those loads in flight.
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
    static constexpr int KS = DK / 32;
    static constexpr int NU = BF ? 1 : 3;  // parts of u against P: o is rounded to bf16 right after
    alignas(16) __bf16 s[KS][NT][IO::NS][512];
    alignas(16) __bf16 e[2][NT][IO::NS][512];
    alignas(16) __bf16 u[2][NT][NU][512];
    alignas(16) __bf16 ku[2][NT][IO::NS][512];
};

template <bool BF, int DK, int NT, int MODE>
__global__ __launch_bounds__(kThreads) void k_delta_scan(ScanArgs a) {
    using IO = Io<BF>;
    using T = typename IO::T;
    constexpr int KS = DK / 32, MT = DK / 64;
    constexpr int NS = IO::NS, NP = BF ? 1 : 3;
    extern __shared__ __align__(16) unsigned char lds_raw[];
    ScanLds<BF, DK, NT>& l = *reinterpret_cast<ScanLds<BF, DK, NT>*>(lds_raw);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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
    const Range r = seq_range(a.seqs, n);
    const int64_t nch = (r.len + kC - 1) / kC;
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

    const int64_t row = 16 * wave + col;   // token of this lane's operand rows
    const int64_t drow = 16 * wave + 4 * g;  // first of this lane's four result rows
    const T* kp = (const T*)a.k + (r.first + row) * a.sh.ldk + (int64_t)hk * dk + 8 * g;
    const T* qp = (const T*)a.q + (r.first + row) * a.sh.ldq + (int64_t)hk * dk + 8 * g;
    const T* vp = (const T*)a.v + (r.first + drow) * a.sh.ldv + (int64_t)h * dv + c0;
    T* op = (T*)(MODE == kScanOut ? a.o : a.u) + ((r.first + drow) * hv + h) * (int64_t)dv + c0;

    Raw<BF> K[KS], Q[KS], KT[MT][2];
    Frag<NS> Tf[2];
    Frag<NP> Pf[2];
    float V[4][NT];
    f32x4 gam, kap, bet;
    float glast = 0.f;
    auto load_k = [&](int64_t c) {
        const bool ok = c * kC + row < r.len;
#pragma unroll
        for (int s = 0; s < KS; ++s) K[s] = load_raw(kp + c * kC * a.sh.ldk + 32 * s, ok && 32 * s + 8 * g < dk);
    };
    auto load_q = [&](int64_t c) {
        const bool ok = c * kC + row < r.len;
#pragma unroll
        for (int s = 0; s < KS; ++s) Q[s] = load_raw(qp + c * kC * a.sh.ldq + 32 * s, ok && 32 * s + 8 * g < dk);
    };
    auto load_v = [&](int64_t c) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load_cols<NT>(vp + (c * kC + i) * a.sh.ldv, cok && c * kC + drow + i < r.len, V[i]);
    };
    auto load_sc = [&](int64_t c) {
        const float* sc = a.prep.sc + ((r.slot0 + c) * hv + h) * 3 * kC;
        gam = *reinterpret_cast<const f32x4*>(sc + drow);
        kap = *reinterpret_cast<const f32x4*>(sc + kC + drow);
        bet = *reinterpret_cast<const f32x4*>(sc + 2 * kC + drow);
        glast = sc[kC - 1];
    };
    // every fragment of row tile `wave`: one step for tiles 0 and 1, two below
    auto load_t = [&](int64_t c) {
        const __bf16* p = a.prep.t + ((r.slot0 + c) * hv + h) * kTri * NS * 512;
        Tf[0] = get_frag<NS>(p + lower_frag(wave, 0) * NS * 512, 512, lane);
        if (wave >= 2) Tf[1] = get_frag<NS>(p + lower_frag(wave, 1) * NS * 512, 512, lane);
    };
    auto load_p = [&](int64_t c) {
        const __bf16* p = a.prep.p + ((r.slot0 + c) * hv + h) * kTri * NP * 512;
        Pf[0] = get_frag<NP>(p + lower_frag(wave, 0) * NP * 512, 512, lane);
        if (wave >= 2) Pf[1] = get_frag<NP>(p + lower_frag(wave, 1) * NP * 512, 512, lane);
    };
    auto load_kt = [&](int64_t c) {
        const T* p = (const T*)a.prep.kt + ((r.slot0 + c) * a.sh.hk + hk) * (DK / 16) * 1024 + lane * 8;
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
    if (nch > 0) {
        load_k(0);
        load_sc(0);
        load_v(0);
        if (MODE == kScanOut) load_q(0);
        load_t(0);
        if (MODE == kScanOut) load_p(0);
        load_kt(0);
        put_state();
    }
    for (int64_t c = 0; c < nch; ++c) {
        const int64_t nx = c + 1 < nch ? c + 1 : c;  // the last chunk loads itself again
        if (MODE == kScanKeep) {
            T* sp = (T*)a.s0 + ((r.slot0 + c) * hv + h) * (int64_t)dk * dv + c0;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = 16 * (wave * MT + m) + 4 * g + i;
                    float x[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) x[j] = S[m][j][i];
                    if (cok && k < dk) store_cols<NT>(sp + (int64_t)k * dv, x);
                }
        }
        lds_barrier();  // the state's fragments are in place
        f32x4 ks[NT] = {}, qs[NT] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const Frag<IO::NI> ka = to_frag(K[s]);
            Frag<IO::NI> qa;
            if (MODE == kScanOut) qa = to_frag(Q[s]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const Frag<NS> sf = get_frag<NS>(&l.s[s][j][0][0], 512, lane);
                ks[j] = mma(ka, sf, ks[j]);
                if (MODE == kScanOut) {
                    Frag<NP> s1;  // one part of the state against bf16 outputs
#pragma unroll
                    for (int i = 0; i < NP; ++i) s1.p[i] = sf.p[i];
                    qs[j] = mma(qa, s1, qs[j]);
                }
            }
        }
        load_k(nx);
        if (MODE == kScanOut) load_q(nx);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = bet[i] * (V[i][j] - gam[i] * ks[j][i]);
            put_rows<NS>(&l.e[wave >> 1][j][0][0], 512, wave & 1, lane, x);
        }
        load_v(nx);
        lds_barrier();  // e
        f32x4 u[NT] = {};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            u[j] = mma(Tf[0], get_frag<NS>(&l.e[0][j][0][0], 512, lane), u[j]);
            if (wave >= 2) u[j] = mma(Tf[1], get_frag<NS>(&l.e[1][j][0][0], 512, lane), u[j]);
        }
        load_t(nx);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = u[j][i];
                y[i] = kap[i] * u[j][i];
            }
            if (MODE == kScanOut) put_rows<NP>(&l.u[wave >> 1][j][0][0], 512, wave & 1, lane, x);
            put_rows<NS>(&l.ku[wave >> 1][j][0][0], 512, wave & 1, lane, y);
        }
        if (MODE == kScanKeep)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (cok && c * kC + drow + i < r.len) {
                    float x[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) x[j] = u[j][i];
                    store_cols<NT>(op + (c * kC + i) * hv * (int64_t)dv, x);
                }
        lds_barrier();  // u
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[m][j][i] *= glast;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const Frag<NS> uf = get_frag<NS>(&l.ku[s][j][0][0], 512, lane);
#pragma unroll
                for (int m = 0; m < MT; ++m) S[m][j] = mma(to_frag(KT[m][s]), uf, S[m][j]);
            }
        load_kt(nx);
        put_state();
        if (MODE == kScanOut) {
            f32x4 o[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][i] = gam[i] * qs[j][i];
                o[j] = mma(Pf[0], get_frag<NP>(&l.u[0][j][0][0], 512, lane), o[j]);
                if (wave >= 2) o[j] = mma(Pf[1], get_frag<NP>(&l.u[1][j][0][0], 512, lane), o[j]);
            }
            load_p(nx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (cok && c * kC + drow + i < r.len) {
                    float x[NT];
#pragma unroll
                    for (int j = 0; j < NT; ++j) x[j] = a.sh.scale * o[j][i];
                    store_cols<NT>(op + (c * kC + i) * hv * (int64_t)dv, x);
                }
        }
        load_sc(nx);
    }
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
