// The backward's state scan: from the last chunk to the first it carries dS, the gradient
// of the state, and solves for r, the gradient of the residuals. With dS1 the gradient of
// the state behind a chunk and the forward's T, P, decays:
//   dU = P^T (scale dO) + diag(exp(G_last - G)) K dS1,        r = T^T dU,
//   dS0 = exp(G_last) dS1 + Q^T diag(scale exp(G)) dO - K^T diag(exp(G) beta) r.
// The same shape as the forward's scan, and the same division: a state wave for each
// block of 16 columns, in whose registers dS stays (fp32, operands as bf16 parts), and
// here an input wave a block, one chunk ahead, that makes what does not depend on dS
// (P^T dO and Q^T diag(exp(G)) dO) and hands it over in LDS as fp32. The input waves of
// bf16 calls also stage K, Q and dO, half the rows each; fp32 calls have a staging wave.
// Measured as the forward's scan: 401 us, 3.1 us a chunk (2.4 TB/s). Chain and memory bound
// it: with P, dU and r in two parts, and bf16 alone kept, it took 358, without stores 264, without
// the inputs 259, the input waves alone 183. Stores from the input waves (results handed back in
// LDS) took 358 to 386 in place of 358, T^T a chunk ahead in alternating registers 365.
#pragma once
#include "delta_scan.hpp"

namespace hy {
namespace delta {

struct RevArgs {
    Seqs seqs;
    Shape sh;
    const void *q, *k;
    Prep prep;
    const void* dout;      // [tokens][hv][dv]
    const float* ds_out;   // [N][hv][dk][dv] gradient of the final states, or null
    float* ds_in;          // likewise of the initial states (output), or null
    void* ds1;             // dS behind every chunk, as Kept
    void* r;               // likewise
    Pieces pieces;
    int nblk, nb16;
};

template <int DK>
struct RevInputs {  // what an input wave hands over
    alignas(16) f32x4 u[4][64];        // P^T dO, row tiles of tokens
    alignas(16) f32x4 s[DK / 16][64];  // Q^T diag(exp(G)) dO, row tiles of dk
};
template <bool BF, int DK>
struct RevCfg {
    static constexpr int NB = BF ? 2 : 1;
    static constexpr int BUF = BF ? 2 : 1;
    static constexpr bool STAGER = !BF;
    static constexpr int threads = 64 * (2 * NB + (STAGER ? 1 : 0));
    struct None {};
    struct LdsV {
        ColTile<16 * NB> o[BUF];
    };
    struct LdsT {
        Tile<Io<BF>::NI, DK> k[BUF], q[BUF];
        RevInputs<DK> x[NB][2];
    };
    struct Lds : LdsT, std::conditional<BF, LdsV, None>::type {};
};

// ENDS: only dS in front of a piece that starts from zero (the last from ds_out), for
// the pieces before it to carry
template <bool BF, int DK, bool ENDS>
__global__ __launch_bounds__((RevCfg<BF, DK>::threads)) __attribute__((amdgpu_waves_per_eu(1)))
void k_delta_rev(RevArgs a) {
    using IO = Io<BF>;
    using T = typename IO::T;
    using Cfg = RevCfg<BF, DK>;
    constexpr int KS = DK / 32, MT = DK / 16, NB = Cfg::NB, BUF = Cfg::BUF;
    constexpr int NI = IO::NI, NS = IO::NS, NG = IO::NE, NE = ENDS ? NS : IO::NE;
    constexpr uint32_t E = sizeof(T);
    extern __shared__ __align__(16) unsigned char lds_raw[];
    typename Cfg::Lds& l = *reinterpret_cast<typename Cfg::Lds*>(lds_raw);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, col = lane & 15;
    const int64_t bid = blockIdx.x;
    const int64_t pair = bid / (8 * a.nblk) * 8 + (bid & 7);
    const int hv = a.sh.hv;
    if (pair >= a.pieces.slots * hv) return;
    Piece pc;
    if (!find_piece(a.seqs, a.pieces, pair / hv, pc) || (ENDS && pc.s == 0)) return;
    const int64_t n = pc.n;
    const int h = (int)(pair % hv), hk = h / a.sh.group;
    const int64_t first = uniform64(pc.r.first), len = uniform64(pc.r.len), slot0 = uniform64(pc.r.slot0);
    const int behind = __builtin_amdgcn_readfirstlane(pc.count - 1 - pc.s);  // pieces behind this one
    const int nch = (int)((len + kC - 1) / kC);
    const int tail = (int)(len - (int64_t)(nch - 1) * kC);
    const int dk = a.sh.dk, dv = a.sh.dv;
    const int wgcol = (int)(bid / 8 % a.nblk) * NB * 16;
    const uint32_t ldo = (uint32_t)(hv * dv) * E;
    const int64_t krow = (int64_t)kC * a.sh.ldk * E, qrow = (int64_t)kC * a.sh.ldq * E, orow = (int64_t)kC * ldo;
    const unsigned char* kbase = (const unsigned char*)((const T*)a.k + first * a.sh.ldk + (int64_t)hk * dk);
    const unsigned char* qbase = (const unsigned char*)((const T*)a.q + first * a.sh.ldq + (int64_t)hk * dk);
    const unsigned char* obase = (const unsigned char*)((const T*)a.dout + (first * hv + h) * (int64_t)dv);
    // chunks are numbered in the order they are taken: number i is chunk nch - 1 - i
    auto rows_in = [&](int i) { return i == 0 ? tail : kC; };
    // (numbers behind the last: the last again, staged and never read)
    auto load_tile = [&](auto& r, const unsigned char* base, int64_t step, int64_t ld, int i, int w = 0) {
        i = i < nch ? i : nch - 1;
        r.load(plain_buf(base + (nch - 1 - i) * step, (rows_in(i) - 1) * (uint32_t)(ld * E) + dk * E), (uint32_t)(ld * E), dk, lane,
               w);
    };
    auto load_o = [&](auto& r, int i, int w) {
        i = i < nch ? i : nch - 1;
        r.load(plain_buf(obase + (nch - 1 - i) * orow, (rows_in(i) - 1) * ldo + dv * E), ldo, wgcol, dv, lane, w);
    };

    if constexpr (Cfg::STAGER)
        if (wave == waves_of<Cfg>() - 1) {
            // K of number i for the state, Q of number i + 1 for the inputs
            Stage<BF, DK> rk, rq;
            if (nch > 0) {
                load_tile(rq, qbase, qrow, a.sh.ldq, 0);
                load_tile(rk, kbase, krow, a.sh.ldk, 0);
                rq.store(l.q[0], lane);
                rk.store(l.k[0], lane);
                load_tile(rq, qbase, qrow, a.sh.ldq, 1);
                lds_barrier();
                lds_barrier();  // the first inputs are made
                rq.store(l.q[0], lane);
                load_tile(rk, kbase, krow, a.sh.ldk, 1);
                load_tile(rq, qbase, qrow, a.sh.ldq, 2);
                lds_barrier();
            }
            for (int i = 0; i < nch; ++i) {
                lds_barrier();  // K of number i and Q of number i + 1 have been read
                rk.store(l.k[0], lane);
                rq.store(l.q[0], lane);
                load_tile(rk, kbase, krow, a.sh.ldk, i + 2);
                load_tile(rq, qbase, qrow, a.sh.ldq, i + 3);
                lds_barrier();
            }
            return;
        }

    const MinusOne minus(lane);
    const int blk = wgcol / 16 + wave % NB;
    const int c0 = blk * 16 + col;
    const bool cok = c0 < dv;
    auto drow = [&](int t, int i) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1) + i; };
    const uint32_t ooff = cok ? drow(0, 0) * ldo + c0 * E : kNoElem;
    auto rec_buf = [&](int i) {
        return plain_buf(a.prep.rec + ((slot0 + nch - 1 - i) * hv + h) * Rec<BF>::bytes, Rec<BF>::bytes);
    };
    auto back_buf = [&](int i) {
        return plain_buf(a.prep.back + ((slot0 + nch - 1 - i) * hv + h) * Rec<BF>::back, Rec<BF>::back);
    };

    if (wave >= NB) {
        Frag<NG> Pt[kTri];
        f32x4 gam[4];
        uint32_t O[4][4];  // fp32 dO, a chunk ahead
        auto load = [&](int i) {
            const RowBuf rb = rec_buf(i), bb = back_buf(i);
#pragma unroll
            for (int t = 0; t < 4; ++t) gam[t] = buf_f4(rb, drow(t, 0) * 4, Rec<BF>::sc);
#pragma unroll
            for (int f = 0; f < kTri; ++f) Pt[f] = buf_frag<NG>(bb, Rec<BF>::pt, f, lane);
            if constexpr (!BF) {
                const RowBuf ob = plain_buf(obase + (nch - 1 - i) * orow, (rows_in(i) - 1) * ldo + dv * E);
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        O[t][j] = __builtin_amdgcn_raw_buffer_load_b32(ob, (int)(ooff + (32 * (t >> 1) + 4 * (t & 1) + j) * ldo), 0, 0);
            }
        };
        auto inputs = [&](int i) {
            RevInputs<DK>& out = l.x[wave - NB][i & 1];
            const Tile<NI, DK>& q = l.q[i & (BUF - 1)];
            f32x4 o[4];
            Frag<NI> of[2];
            if constexpr (BF) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const u32x2 lo = l.o[i & 1].rows4(lane, 2 * s, 16 * (wave - NB));
                    const u32x2 hi = l.o[i & 1].rows4(lane, 2 * s + 1, 16 * (wave - NB));
                    const u32x4 w = {lo[0], lo[1], hi[0], hi[1]};
                    of[s].p[0] = __builtin_bit_cast(bf16x8, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[2 * s][j] = __uint_as_float(j & 1 ? lo[j >> 1] & 0xffff0000u : lo[j >> 1] << 16);
                        o[2 * s + 1][j] = __uint_as_float(j & 1 ? hi[j >> 1] & 0xffff0000u : hi[j >> 1] << 16);
                    }
                }
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[t][j] = __uint_as_float(O[t][j]);
#pragma unroll
                for (int s = 0; s < 2; ++s) of[s] = pair_frag<NI>(o[2 * s], o[2 * s + 1], minus);
            }
            f32x4 x[4] = {};
            const Frag<NG> p0[2] = {Pt[0], Pt[2]}, p1[4] = {Pt[1], Pt[3], Pt[4], Pt[5]};
            mma_tiles(p0, of[0], x);
            mma_tiles(p1, of[1], x);
#pragma unroll
            for (int t = 0; t < 4; ++t) out.u[t][lane] = a.sh.scale * x[t];
            Frag<NG> gf[2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
                gf[s] = pair_frag<NG>(a.sh.scale * gam[2 * s] * o[2 * s], a.sh.scale * gam[2 * s + 1] * o[2 * s + 1], minus);
            load(i + 1 < nch ? i + 1 : nch - 1);
#pragma unroll
            for (int m = 0; m < MT; m += 2) {
                f32x4 y[2] = {};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Frag<NI> w[2] = {q.cols(lane, m, s), q.cols(lane, m + 1, s)};
                    mma_tiles(w, gf[s], y);
                }
                out.s[m][lane] = y[0];
                out.s[m + 1][lane] = y[1];
            }
        };
        if (nch > 0) load(0);
        if constexpr (Cfg::STAGER) {
            if (nch > 0) {
                lds_barrier();
                inputs(0);
                lds_barrier();
                lds_barrier();
            }
            for (int i = 0; i < nch; ++i) {
                inputs(i + 1);
                lds_barrier();
                lds_barrier();
            }
        } else {
            // each also stages its half of the rows: K of number i + 1 while the state is at i,
            // Q and dO of number i + 2
            Stage<BF, DK, NB> rk, rq;
            StageV<NB> ro;
            const int w = wave - NB;
            auto stage_q = [&](int i) {
                rq.store(l.q[i & 1], lane, w);
                ro.store(l.o[i & 1], lane, w);
                load_tile(rq, qbase, qrow, a.sh.ldq, i + 1, w);
                load_o(ro, i + 1, w);
            };
            auto stage_k = [&](int i) {
                rk.store(l.k[i & 1], lane, w);
                load_tile(rk, kbase, krow, a.sh.ldk, i + 1, w);
            };
            if (nch > 0) {
                load_tile(rq, qbase, qrow, a.sh.ldq, 0, w);
                load_o(ro, 0, w);
                load_tile(rk, kbase, krow, a.sh.ldk, 0, w);
                stage_q(0);
                stage_k(0);
                lds_barrier();
                stage_q(1);
                inputs(0);
                lds_barrier();
            }
            for (int i = 0; i < nch; ++i) {
                stage_k(i + 1);
                stage_q(i + 2);
                __builtin_amdgcn_sched_barrier(0);
                inputs(i + 1);
                lds_barrier();
            }
        }
        return;
    }

    __builtin_amdgcn_s_setprio(3);
    f32x4 S[MT];
    Frag<NS> sf[KS];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = drow(t, i);
            S[t][i] = behind == 0 && a.ds_out && k < dk && cok ? a.ds_out[((n * hv + h) * dk + k) * dv + c0] : 0.f;
        }
    const int64_t bsize = (int64_t)a.nb16 * MT * 256, msize = DK * DK * NS * 2;
    if (!ENDS && behind > 0 && blk < a.nb16) {
        const int64_t at = (uniform64(pc.first) + pc.count - 1) * hv + h;  // the last piece
        carry<NS, DK>(S, a.pieces.b + at * bsize + blk * (MT * 256), -hv * bsize, a.pieces.mt + at * msize, -hv * msize, behind - 1,
                      lane, minus);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) sf[s] = pair_frag<NS>(S[2 * s], S[2 * s + 1], minus);

    Frag<NS> Tt[kTri];
    f32x4 gam[4], kap[4], bet[4];
    float glast = 0.f;
    auto load_sc = [&](int i) {
        const RowBuf rb = rec_buf(i);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            gam[t] = buf_f4(rb, drow(t, 0) * 4, Rec<BF>::sc);
            kap[t] = buf_f4(rb, drow(t, 0) * 4, Rec<BF>::sc + kC * 4);
            bet[t] = buf_f4(rb, drow(t, 0) * 4, Rec<BF>::sc + 2 * kC * 4);
        }
        glast = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rb, 0, Rec<BF>::sc + (kC - 1) * 4, 0));
    };
    auto load_t = [&](int i) {
        const RowBuf bb = back_buf(i);
#pragma unroll
        for (int f = 0; f < kTri; ++f) Tt[f] = buf_frag<NS>(bb, 0, f, lane);
    };
    if (nch > 0) {
        load_sc(0);
        load_t(0);
        lds_barrier();  // Q and dO of the first chunk
        if (Cfg::STAGER) lds_barrier();
        lds_barrier();  // its inputs and K
    }
    using Kp = Kept<BF, KS>;
    constexpr int X2 = NI == 1 ? NE : 6, X3 = NS == 3 ? 6 : NE == 3 ? 5 : 3;  // matrix instructions per product
    for (int i = 0; i < nch; ++i) {
        const int nx = i + 1 < nch ? i + 1 : i;
        const Tile<NI, DK>& K = l.k[i & (BUF - 1)];
        const RevInputs<DK>& in = l.x[wave][i & 1];
        const int64_t fr = ((slot0 + nch - 1 - i) * hv + h) * a.nb16 + blk;  // this block's fragments
        auto keep_s = [&](int s) {
            keep_frag<BF>((unsigned char*)a.ds1 + fr * Kp::state, blk < a.nb16, KS, s, lane, S[2 * s], S[2 * s + 1]);
        };
        auto keep_r = [&](const f32x4(&r)[4], int s) {
            keep_frag<BF>((unsigned char*)a.r + fr * Kp::rows, blk < a.nb16, 2, s, lane, r[2 * s], r[2 * s + 1]);
        };
        if constexpr (!ENDS && !BF) {
#pragma unroll
            for (int s = 0; s < KS; ++s) keep_s(s);
        }
        // dU = P^T dO + diag(exp(G_last - G)) K dS
        f32x4 x[4] = {};
        Frag<NI> ka[2][4];
        auto read_rows = [&](int s) {
#pragma unroll
            for (int t = 0; t < 4; ++t) ka[s & 1][t] = K.rows(lane, t, s);
        };
        read_rows(0);
        read_rows(1);
        f32x4 xu[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) xu[t] = in.u[t][lane];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            mma_tiles(ka[s & 1], sf[s], x);
            if (s + 2 < KS) read_rows(s + 2);
            if constexpr (!ENDS && BF) keep_s(s);
            __builtin_amdgcn_sched_barrier(0);
        }
        Frag<NI> kt[2][MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) kt[1][m] = K.cols(lane, m, 1);
        __builtin_amdgcn_sched_barrier(0);
        Frag<NE> uf[2];
        auto du = [&](int p) {
#pragma unroll
            for (int t = 2 * p; t < 2 * p + 2; ++t) x[t] = kap[t] * x[t] + xu[t];
            uf[p] = pair_frag<NE>(x[2 * p], x[2 * p + 1], minus);
        };
        du(1);
        __builtin_amdgcn_sched_barrier(0);
        // r = T^T dU: rows of the second half depend on the second half of dU only
        f32x4 r[4] = {};
        const Frag<NS> t1[4] = {Tt[1], Tt[3], Tt[4], Tt[5]}, t0[2] = {Tt[0], Tt[2]};
        mma_tiles(t1, uf[1], r);
        du(0);
        interleave<4 * X3, 4, 0>();
        mma_tiles(t0, uf[0], r);
        // -diag(exp(G) beta) r as an operand, the second half first
        Frag<NE> rf[2];
        auto rpart = [&](int p) {
            rf[p] = pair_frag<NE>(-gam[2 * p] * bet[2 * p] * r[2 * p], -gam[2 * p + 1] * bet[2 * p + 1] * r[2 * p + 1], minus);
        };
        rpart(1);
#pragma unroll
        for (int m = 0; m < MT; ++m) S[m] = glast * S[m] + in.s[m][lane];
        __builtin_amdgcn_sched_barrier(0);
        load_t(nx);
#pragma unroll
        for (int m = 0; m < MT; ++m) kt[0][m] = K.cols(lane, m, 0);
        __builtin_amdgcn_sched_barrier(0);
        auto update = [&](int s, int p) {
            const Frag<NI> w[2] = {kt[s][2 * p], kt[s][2 * p + 1]};
            mma_tiles(w, rf[s], S + 2 * p);
        };
        auto parts = [&](int p) { sf[p] = pair_frag<NS>(S[2 * p], S[2 * p + 1], minus); };
#pragma unroll
        for (int p = 0; p < KS; ++p) update(1, p);
        rpart(0);
        interleave<MT * X2, 5, 0>();
        if constexpr (!ENDS && !BF) {
#pragma unroll
            for (int s = 0; s < 2; ++s) keep_r(r, s);
        }
        load_sc(nx);
        __builtin_amdgcn_sched_barrier(0);
        update(0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int p = 1; p < KS; ++p) {
            update(0, p);
            parts(p - 1);
            if constexpr (!ENDS && BF)
                if (p < 3) keep_r(r, p - 1);  // (heads of 64 have one such step: the other half below)
            interleave<2 * X2, 6, 0>();
        }
        if constexpr (!ENDS && BF && KS == 2) keep_r(r, 1);
        parts(KS - 1);
        if (BUF == 1) lds_barrier();
        lds_barrier();
    }
    if constexpr (ENDS) {
        if (blk < a.nb16)
#pragma unroll
            for (int t = 0; t < MT; ++t)
                *reinterpret_cast<f32x4*>(a.pieces.b + ((uniform64(pc.first) + pc.s) * hv + h) * bsize + blk * (MT * 256) +
                                          (t * 64 + lane) * 4) = S[t];
        return;
    }
    if (a.ds_in && pc.s == 0)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = drow(t, i);
                if (cok && k < dk) a.ds_in[((n * hv + h) * dk + k) * dv + c0] = S[t][i];
            }
}

}  // namespace delta
}  // namespace hy
