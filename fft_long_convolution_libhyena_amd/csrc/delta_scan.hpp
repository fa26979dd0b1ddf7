// The state scan of the gated delta rule. A workgroup carries NB blocks of 16 columns of
// one (sequence, value head)'s state through its chunks, or through those of a piece of the
// sequence; three kinds of waves share it:
//   state     one wave a block: e, u and the new state, all in its registers
//   outputs   one wave a block, a chunk behind: o = scale (exp(G) Q S + P u)
//   staging   brings K, Q (and bf16 v) of the next chunks into LDS: the outputs' waves, half
//             the rows each (bf16), or a wave of its own
// The scan that keeps states for the backward has no outputs, and the one that makes the
// ends of pieces has only state waves, four a workgroup, which also stage (bf16).
// The state is fp32 with its bf16 parts beside it as right-hand operands. With rows
// numbered as in tile_row, every result of a chunk (the residual e, the written values u,
// the new state) becomes the next product's operand in the lane that holds it: nothing on
// the way from one state to the next passes through LDS or another wave. The outputs
// are off that way; their wave takes the parts of the state and u from LDS. T, P and the
// decays come as the preparation laid them out, 1 KiB a load, a chunk ahead. One barrier a
// chunk (two where LDS holds one buffer of K and Q only: fp32, three parts).
//
// What bounds it: a state wave is alone on its SIMD, so its instructions (134 matrix, about
// 300 vector for a chunk of a 128 x 16 block) run in order, matrix and vector ones
// alternating; the chain over the chunks is sequential. Measured, 8 sequences of 8192 tokens,
// 6 heads of 128 x 128, bf16: 290 us, 2.3 us a chunk (192 workgroups on 256 CUs; 1.9 TB/s;
// matrix pipes busy 33% of the CUs' cycles); the scan that keeps states, with residuals in two
// parts and 453 MB to write, 300. On the way, for a chunk: tokens and state rows split over four
// waves, operands exchanged in LDS with three barriers, 2.3 us for 32 columns; each wave loading
// K, Q and K^T for itself, 2.0 us for 16 columns (a load of 16 rows of 64 bytes costs 60
// clocks, one of 1 KiB in a row 16).
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
    void* s0;           // state before every chunk, as Kept (for the backward)
    void* u;            // written values, likewise
    Pieces pieces;
    int nblk;           // workgroups per head
    int nbv;            // of them, those on columns of v; the others on M's (ends)
    int nb16;           // blocks of 16 columns per head
};

// outputs; states and written values kept; the ends of pieces
enum { kScanOut = 0, kScanKeep = 1, kScanEnds = 2 };

// The outputs' waves rest for this many 64-clock units after a barrier, while the state
// waves read K: both at once would halve the state's LDS rate where it waits for it (8
// sequences of 8192 tokens: 341 us without the rest, 318 with it).
constexpr int kOutSleep = 8;

// Minus the identity, as left operands that take rows of a 32-row operand back to the
// result tile (t even or odd) they came from.
struct MinusOne {
    bf16x8 a[2];
    __device__ __forceinline__ explicit MinusOne(int lane) {
        const int col = lane & 15, g = lane >> 4;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) a[t][j] = (__bf16)(g == col >> 2 && j == 4 * t + (col & 3) ? -1.f : 0.f);
    }
};
// Eight rows of one column from a pair of result tiles, as an operand. What a part
// leaves of the values (exact in fp32) is a matrix product too, x + (-1) h: two
// instructions on the matrix cores in place of sixteen vector ones.
template <int N>
__device__ __forceinline__ Frag<N> pair_frag(f32x4 a, f32x4 b, const MinusOne& minus) {
    Frag<N> f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const u32x4 w = {pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(b[0], b[1]), pack2(b[2], b[3])};
        f.p[n] = __builtin_bit_cast(bf16x8, w);
        if (n + 1 < N) {
            a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus.a[0], f.p[n], a, 0, 0, 0);
            b = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus.a[1], f.p[n], b, 0, 0, 0);
        }
    }
    return f;
}

template <bool BF, int DK>
struct Exchange {  // the operands of one chunk's outputs
    alignas(16) __bf16 s[DK / 32][Io<BF>::NO][512];
    alignas(16) f32x4 u[4][64];  // as computed: the outputs' wave has time to split it
};
template <bool BF, int DK, int MODE>
struct ScanCfg {
    static constexpr bool OUT = MODE == kScanOut, ENDS = MODE == kScanEnds;
    // column blocks; without outputs to make, the ends' state waves have the CU to themselves
    static constexpr int NB = ENDS ? (BF ? 4 : 3) : BF ? 2 : 1;
    static constexpr int BUF = BF ? 2 : 1;                        // buffers of K and of Q
    static constexpr bool STAGER = !(BF && (OUT || ENDS));       // a wave that only stages
    static constexpr bool SELF = BF && ENDS;                      // the state waves stage
    static constexpr int threads = 64 * ((OUT ? 2 : 1) * NB + (STAGER ? 1 : 0));
    // waves a SIMD: two workgroups share a CU where their LDS lets them (bf16, heads up to 64)
    static constexpr int eu = threads > 256 || (BF && OUT && DK == 64) ? 2 : 1;
    struct None {};
    struct LdsOut {
        Tile<Io<BF>::NI, DK> k[BUF], q[BUF];
        Exchange<BF, DK> x[NB][2];
    };
    struct LdsKeep {
        Tile<Io<BF>::NI, DK> k[BUF];
    };
    struct LdsV {
        ColTile<16 * NB> v[BUF];
    };
    struct Lds : std::conditional<OUT, LdsOut, LdsKeep>::type, std::conditional<BF, LdsV, None>::type {};
};
// v of a chunk, 32 columns, by W waves: 16 rows of 64 bytes an instruction
template <int W>
struct StageV {
    u32x4 r[4 / W];
    __device__ __forceinline__ void load(RowBuf b, uint32_t ld, int col0, int dv, int lane, int w = 0) {
        const int c = col0 + 8 * (lane & 3);
        const uint32_t off = c < dv ? (w * (64 / W) + (lane >> 2)) * ld + c * 2 : kNoElem;
#pragma unroll
        for (int i = 0; i < 4 / W; ++i)
            r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)(off + i * 16 * ld), 0, 0));
    }
    __device__ __forceinline__ void store(ColTile<32>& t, int lane, int w = 0) const {
#pragma unroll
        for (int i = 0; i < 4 / W; ++i)
            *reinterpret_cast<u32x4*>(t.b + (w * (64 / W) + 16 * i + (lane >> 2)) * ColTile<32>::pitch + 16 * (lane & 3)) = r[i];
    }
};

// likewise 64 columns by four waves, 16 rows each: 8 rows of 128 bytes an instruction
struct StageV4 {
    u32x4 r[2];
    __device__ __forceinline__ void load(RowBuf b, uint32_t ld, int col0, int dv, int lane, int w) {
        const int c = col0 + 8 * (lane & 7);
        const uint32_t off = c < dv ? (16 * w + (lane >> 3)) * ld + c * 2 : kNoElem;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)(off + i * 8 * ld), 0, 0));
    }
    __device__ __forceinline__ void store(ColTile<64>& t, int lane, int w) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<u32x4*>(t.b + (16 * w + 8 * i + (lane >> 3)) * ColTile<64>::pitch + 16 * (lane & 7)) = r[i];
    }
};

// The state in front of a piece: the end of the sequence's first piece, carried through
// `steps` more, S = M S + B. b and m point at the first and step from piece to piece
// (the reverse scan goes the other way, with the transposes). M does not depend on the
// state, so its fragments are under way a step (fp32: half a step) ahead.
template <int NS, int DK>
__device__ __forceinline__ void carry(f32x4 (&S)[DK / 16], const float* b, int64_t bstep, const unsigned char* m, int64_t mstep,
                                      int steps, int lane, const MinusOne& minus) {
    constexpr int KS = DK / 32, MT = DK / 16, P = MT / 2, R = NS == 2 ? P : P / 2;
    auto end = [&](const float* p, int t) { return *reinterpret_cast<const f32x4*>(p + (t * 64 + lane) * 4); };
#pragma unroll
    for (int t = 0; t < MT; ++t) S[t] = end(b, t);
    if (steps < 1) return;
    Frag<NS> a[R][2][KS];
    auto load = [&](const unsigned char* p, int i) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int s = 0; s < KS; ++s)
                a[i % R][t][s] = get_frag<NS>(reinterpret_cast<const __bf16*>(p) + ((2 * i + t) * KS + s) * NS * 512, 512, lane);
    };
    m += mstep;
#pragma unroll
    for (int i = 0; i < R; ++i) load(m, i);
    for (int k = 0; k < steps; ++k) {
        b += bstep;
        Frag<NS> f[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) f[s] = pair_frag<NS>(S[2 * s], S[2 * s + 1], minus);
#pragma unroll
        for (int t = 0; t < MT; ++t) S[t] = end(b, t);
        const unsigned char* next = k + 1 < steps ? m + mstep : m;
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Frag<NS> w[2] = {a[i % R][0][s], a[i % R][1][s]};
                mma_tiles(w, f[s], S + 2 * i);
            }
            load(i + R < P ? m : next, (i + R) % P);
        }
        m = next;
    }
}
// a column of M, as a state wave holds it, to where carry takes it: element j of lane
// (row of the tile, eight columns) of fragment (row tile, 32 columns)
template <int NS, int DK>
__device__ __forceinline__ void store_end(unsigned char* m, unsigned char* mt, const f32x4 (&S)[DK / 16], int c0, int lane) {
    constexpr int KS = DK / 32, MT = DK / 16;
    const int g = lane >> 4;
    // the row of M^T that this column is: tile and row in it, inverting tile_row
    const int tm = 2 * (c0 >> 5) + (c0 >> 2 & 1), tr = 4 * (c0 >> 3 & 3) + (c0 & 3);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const f32x4 &x = S[2 * s], &y = S[2 * s + 1];
        const Frag<NS> f = split8<NS>({x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
#pragma unroll
        for (int n = 0; n < NS; ++n) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int tile = 2 * s + (j >> 2), l = 16 * (c0 >> 3 & 3) + 4 * g + (j & 3);
                reinterpret_cast<__bf16*>(m)[((tile * KS + (c0 >> 5)) * NS + n) * 512 + l * 8 + (c0 & 7)] = f.p[n][j];
            }
            if (mt) *reinterpret_cast<bf16x8*>(mt + (((tm * KS + s) * NS + n) * 512 + (16 * g + tr) * 8) * 2) = f.p[n];
        }
    }
    static_assert(MT == 2 * KS, "pairs of tiles");
}

template <class Cfg>
__device__ __forceinline__ constexpr int waves_of() {
    return Cfg::threads / 64;
}

template <bool BF, int DK, int MODE>
__global__ __launch_bounds__((ScanCfg<BF, DK, MODE>::threads)) __attribute__((amdgpu_waves_per_eu((ScanCfg<BF, DK, MODE>::eu))))
void k_delta_scan(ScanArgs a) {
    using IO = Io<BF>;
    using T = typename IO::T;
    using Cfg = ScanCfg<BF, DK, MODE>;
    constexpr bool OUT = Cfg::OUT, ENDS = Cfg::ENDS;
    constexpr int KS = DK / 32, MT = DK / 16, NB = Cfg::NB, BUF = Cfg::BUF;
    // states kept for the backward and at the ends of pieces are carried on in NS parts
    constexpr int NI = IO::NI, NS = IO::NS, NE = OUT ? IO::NE : NS, NP = IO::NP, NO = IO::NO;
    constexpr uint32_t E = sizeof(T);
    extern __shared__ __align__(16) unsigned char lds_raw[];
    typename Cfg::Lds& l = *reinterpret_cast<typename Cfg::Lds*>(lds_raw);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, col = lane & 15;
    // column blocks of one head sit 8 workgroups apart, so that they land on one XCD
    // and share its L2 for the head's operands
    const int64_t bid = blockIdx.x;
    const int64_t pair = bid / (8 * a.nblk) * 8 + (bid & 7);
    const int hv = a.sh.hv;
    if (pair >= a.pieces.slots * hv) return;
    Piece pc;
    if (!find_piece(a.seqs, a.pieces, pair / hv, pc)) return;
    const int64_t n = pc.n;
    const int h = (int)(pair % hv), hk = h / a.sh.group;
    const int64_t first = uniform64(pc.r.first), len = uniform64(pc.r.len), slot0 = uniform64(pc.r.slot0);
    const int64_t pslot = uniform64(pc.first);
    const int ps = __builtin_amdgcn_readfirstlane(pc.s);
    const bool last = pc.s + 1 == pc.count;
    const int wg = (int)(bid / 8 % a.nblk);
    const bool onm = ENDS && wg >= a.nbv;  // columns of M
    if (ENDS && (last || (onm && ps == 0))) return;
    const int nch = (int)((len + kC - 1) / kC);
    const int tail = (int)(len - (int64_t)(nch - 1) * kC);  // rows of the last chunk
    const int dk = a.sh.dk, dv = a.sh.dv;
    const int64_t recstep = (int64_t)hv * Rec<BF>::bytes;
    const unsigned char* rec = a.prep.rec + (slot0 * hv + h) * Rec<BF>::bytes;

    // what a staging wave does for K, Q or v: chunk c stored, chunk c + 1 on its way
    const int64_t krow = (int64_t)kC * a.sh.ldk * E, qrow = (int64_t)kC * a.sh.ldq * E, vrow = (int64_t)kC * a.sh.ldv * E;
    const unsigned char* kbase = (const unsigned char*)((const T*)a.k + first * a.sh.ldk + (int64_t)hk * dk);
    const unsigned char* qbase = OUT ? (const unsigned char*)((const T*)a.q + first * a.sh.ldq + (int64_t)hk * dk) : nullptr;
    const unsigned char* vbase = (const unsigned char*)((const T*)a.v + first * a.sh.ldv + (int64_t)h * dv);
    const int wgcol = (onm ? wg - a.nbv : wg) * NB * 16;
    auto rows_in = [&](int c) { return c + 1 < nch ? kC : tail; };
    // (chunks behind the last: the last again, staged and never read, so that the waves that
    // load have no branches, behind which every wait would be one for all loads)
    auto load_tile = [&](auto& r, const unsigned char* base, int64_t step, int64_t ld, int c, int w = 0) {
        c = c < nch ? c : nch - 1;
        r.load(plain_buf(base + c * step, (rows_in(c) - 1) * (uint32_t)(ld * E) + dk * E), (uint32_t)(ld * E), dk, lane, w);
    };
    auto load_vt = [&](auto& r, int c, int w = 0) {
        c = c < nch ? c : nch - 1;
        r.load(plain_buf(vbase + c * vrow, (rows_in(c) - 1) * (uint32_t)(a.sh.ldv * E) + dv * E), (uint32_t)(a.sh.ldv * E), wgcol,
               onm ? 0 : dv, lane, w);
    };
    if constexpr (Cfg::STAGER)
        if (wave == waves_of<Cfg>() - 1) {
            Stage<BF, DK> rk, rq;
            StageV<1> rv;
            if (nch > 0) {
                load_tile(rk, kbase, krow, a.sh.ldk, 0);
                if constexpr (BF) load_vt(rv, 0);
                rk.store(l.k[0], lane);
                if constexpr (BF) rv.store(l.v[0], lane);
                load_tile(rk, kbase, krow, a.sh.ldk, 1);
                if constexpr (BF) load_vt(rv, 1);
                if constexpr (OUT) load_tile(rq, qbase, qrow, a.sh.ldq, 0);
                lds_barrier();
            }
            for (int c = 0; c < nch; ++c) {
                if (BUF == 1) lds_barrier();  // K of chunk c and Q of chunk c - 1 have been read
                rk.store(l.k[(c + 1) & (BUF - 1)], lane);
                if constexpr (BF) rv.store(l.v[(c + 1) & (BUF - 1)], lane);
                if constexpr (OUT) rq.store(l.q[c & (BUF - 1)], lane);
                load_tile(rk, kbase, krow, a.sh.ldk, c + 2);
                if constexpr (BF) load_vt(rv, c + 2);
                if constexpr (OUT) load_tile(rq, qbase, qrow, a.sh.ldq, c + 1);
                lds_barrier();
            }
            return;
        }

    const MinusOne minus(lane);
    const int blk = wgcol / 16 + wave % NB;
    const int c0 = blk * 16 + col;  // this lane's column
    const bool cok = !onm && c0 < dv;
    const uint32_t ldo = (uint32_t)(hv * dv) * E;
    unsigned char* op = OUT ? (unsigned char*)((T*)a.o + (first * hv + h) * (int64_t)dv) : nullptr;
    // row i of this lane's results in tile t
    auto drow = [&](int t, int i) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1) + i; };
    const uint32_t ooff = cok ? drow(0, 0) * ldo + c0 * E : kNoElem;
    const uint32_t ofull = (kC - 1) * ldo + dv * E, olast = (tail - 1) * ldo + dv * E;
    auto store_rows = [&](const f32x4(&y)[4], int c) {
        const RowBuf b = plain_buf(op, c + 1 < nch ? ofull : olast);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                buf_store<BF>(b, ooff + (32 * (t >> 1) + 4 * (t & 1) + i) * ldo, y[t][i]);
            }
        op += (int64_t)kC * ldo;
    };

    if constexpr (OUT)
        if (wave >= NB) {
            Frag<NP> Pf[kTri];
            f32x4 gam[4];
            auto load = [&]() {
                const RowBuf rb = plain_buf(rec, Rec<BF>::bytes);
#pragma unroll
                for (int t = 0; t < 4; ++t) gam[t] = buf_f4(rb, drow(t, 0) * 4, Rec<BF>::sc);
#pragma unroll
                for (int f = 0; f < kTri; ++f) Pf[f] = buf_frag<NP>(rb, Rec<BF>::p, f, lane);
            };
            // The outputs again where u or S is not finite: u from its residuals, K, v, T and the
            // decays read once more
            auto causal = [&](int c, const auto& q, const auto& in, f32x4(&y)[4]) {
                const uint32_t ldk = (uint32_t)a.sh.ldk * E, ldv = (uint32_t)a.sh.ldv * E;
                const RowBuf kb = plain_buf(kbase + c * krow, (rows_in(c) - 1) * ldk + dk * E), rb = plain_buf(rec, Rec<BF>::bytes);
                const RowBuf vb = plain_buf(vbase + c * vrow, (rows_in(c) - 1) * ldv + dv * E);
                f32x4 e[4] = {}, u[4] = {};
#pragma unroll
                for (int t = 0; t < 4; ++t) y[t] = f32x4{};
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const Frag<NO> sp = get_frag<NO>(&in.s[s][0][0], 512, lane);
                    const int k = 32 * s + 8 * g;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        Raw<BF> r;
                        buf_raw(kb, k < dk ? tile_row(t, col) * ldk + k * E : kNoElem, r);
                        e[t] = mma(to_frag(r), sp, e[t]);
                        y[t] = mma(q.rows(lane, t, s), sp, y[t]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const f32x4 gt = buf_f4(rb, drow(t, 0) * 4, Rec<BF>::sc);
                    y[t] *= gt;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        e[t][i] = fmaf(-gt[i], e[t][i], buf_elem<BF>(vb, cok ? drow(t, i) * ldv + c0 * E : kNoElem));
                }
                const int first = clear_from_first(e, lane);
                {
                    const Frag<IO::NE> half[2] = {pair_frag<IO::NE>(e[0], e[1], minus), pair_frag<IO::NE>(e[2], e[3], minus)};
#pragma unroll
                    for (int f = 0; f < kTri; ++f) {
                        u[tri_row(f)] = mma(buf_frag<NS>(rb, Rec<BF>::t, f, lane), half[tri_half(f)], u[tri_row(f)]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                int from = clear_from_first(u, lane);  // T's diagonal marks tokens, too
                from = from < first ? from : first;
                const Frag<NO> half[2] = {pair_frag<NO>(u[0], u[1], minus), pair_frag<NO>(u[2], u[3], minus)};
#pragma unroll
                for (int f = 0; f < kTri; ++f) {
                    y[tri_row(f)] = mma(buf_frag<NP>(rb, Rec<BF>::p, f, lane), half[tri_half(f)], y[tri_row(f)]);
                    __builtin_amdgcn_sched_barrier(0);
                }
                poison(y, from, lane);
                __builtin_amdgcn_s_waitcnt(0);  // nothing of this is under way where the paths meet again
                __builtin_amdgcn_sched_barrier(0);
            };
            auto outputs = [&](int c) {
                const Exchange<BF, DK>& in = l.x[wave - NB][c & 1];
                const Tile<NI, DK>& q = l.q[c & (BUF - 1)];
                f32x4 y[4] = {};
                Frag<NI> qa[2][4];
                Frag<NO> sp[2];
                auto read = [&](int s) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) qa[s & 1][t] = q.rows(lane, t, s);
                    sp[s & 1] = get_frag<NO>(&in.s[s][0][0], 512, lane);
                };
                read(0);
                read(1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    mma_tiles(qa[s & 1], sp[s & 1], y);
                    if (s + 2 < KS) read(s + 2);
                    __builtin_amdgcn_sched_barrier(0);
                }
                f32x4 u[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) u[t] = in.u[t][lane];
#pragma unroll
                for (int t = 0; t < 4; ++t) y[t] *= gam[t];
                const Frag<NO> u0 = pair_frag<NO>(u[0], u[1], minus), u1 = pair_frag<NO>(u[2], u[3], minus);
                const Frag<NP> p0[4] = {Pf[0], Pf[1], Pf[2], Pf[4]}, p1[2] = {Pf[3], Pf[5]};
                mma_tiles(p0, u0, y);
                mma_tiles(p1, u1, y + 2);
                __builtin_amdgcn_sched_barrier(0);
                if (__builtin_expect(__any(!finite(y[2][0])), 0)) causal(c, q, in, y);  // a row that has met all of u
                if (c + 1 < nch) rec += recstep;
                load();
#pragma unroll
                for (int t = 0; t < 4; ++t) y[t] *= a.sh.scale;
                store_rows(y, c);
            };
            if (nch > 0) load();
            if constexpr (Cfg::STAGER) {
                if (nch > 0) lds_barrier();
                for (int c = 0; c < nch; ++c) {
                    lds_barrier();
                    lds_barrier();
                    outputs(c);
                }
            } else {
                // each also stages its half of the rows: K and v of chunk c + 1 while the state is
                // at c, Q of chunk c
                Stage<BF, DK, NB> rk, rq;
                StageV<NB> rv;
                const int w = wave - NB;
                auto stage = [&](int c) {
                    __builtin_amdgcn_s_sleep(kOutSleep);
                    rk.store(l.k[(c + 1) & 1], lane, w);
                    rv.store(l.v[(c + 1) & 1], lane, w);
                    rq.store(l.q[c & 1], lane, w);
                    load_tile(rk, kbase, krow, a.sh.ldk, c + 2, w);
                    load_vt(rv, c + 2, w);
                    load_tile(rq, qbase, qrow, a.sh.ldq, c + 1, w);
                    __builtin_amdgcn_sched_barrier(0);
                };
                if (nch > 0) {
                    load_tile(rk, kbase, krow, a.sh.ldk, 0, w);
                    load_vt(rv, 0, w);
                    rk.store(l.k[0], lane, w);
                    rv.store(l.v[0], lane, w);
                    load_tile(rk, kbase, krow, a.sh.ldk, 1, w);
                    load_vt(rv, 1, w);
                    load_tile(rq, qbase, qrow, a.sh.ldq, 0, w);
                    lds_barrier();
                    stage(0);
                    lds_barrier();
                }
                for (int c = 1; c < nch; ++c) {
                    stage(c);
                    outputs(c - 1);
                    lds_barrier();
                }
                if (nch > 0) outputs(nch - 1);
            }
            return;
        }

    __builtin_amdgcn_s_setprio(3);  // the sequential part goes first
    f32x4 S[MT];
    Frag<NS> sf[KS];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = drow(t, i);
            S[t][i] = ps == 0 && (ENDS || pc.count == 1) && a.s_in && k < dk && cok ? a.s_in[((n * hv + h) * dk + k) * dv + c0] : 0.f;
            if (onm) S[t][i] = k == c0 ? 1.f : 0.f;
        }
    // A cut sequence's initial state goes to its first piece by way of the last one's unused
    // record: the last piece may have written the final state in its place by then.
    const int64_t bsize = (int64_t)a.nb16 * MT * 256, msize = DK * DK * NS * 2;
    float* bp = a.pieces.b + (pslot * hv + h) * bsize + blk * (MT * 256);  // the first piece's
    const int64_t spare = (pc.count - 1) * (hv * bsize);
    if (pc.count > 1 && !onm && blk < a.nb16) {
        if (!ENDS)
            carry<NS, DK>(S, ps > 0 ? bp : bp + spare, hv * bsize, a.pieces.m + (pslot * hv + h) * msize, hv * msize, ps - 1, lane,
                          minus);
        else if (ps == 0)
#pragma unroll
            for (int t = 0; t < MT; ++t) *reinterpret_cast<f32x4*>(bp + spare + (t * 64 + lane) * 4) = S[t];
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) sf[s] = pair_frag<NS>(S[2 * s], S[2 * s + 1], minus);

    const uint32_t ldv = (uint32_t)a.sh.ldv * E;
    const uint32_t voff = cok ? drow(0, 0) * ldv + c0 * E : kNoElem;
    auto vbuf = [&](int c) { return plain_buf(vbase + c * vrow, (rows_in(c) - 1) * ldv + dv * E); };
    Frag<NS> Tab[BF ? 2 : 1][kTri];  // fp32 has no room for two
    uint32_t V[4][4];  // fp32 only, a chunk ahead; bf16 v comes through LDS
    f32x4 gam[4], kap[4];
    float glast = 0.f;
    auto load_v = [&](const RowBuf& b, int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            V[t][i] = __builtin_amdgcn_raw_buffer_load_b32(b, (int)(voff + (32 * (t >> 1) + 4 * (t & 1) + i) * ldv), 0, 0);
    };
    auto load_gam = [&](const RowBuf& b, int t) { gam[t] = buf_f4(b, drow(t, 0) * 4, Rec<BF>::sc); };
    auto load_kap = [&](const RowBuf& b, int t) { kap[t] = buf_f4(b, drow(t, 0) * 4, Rec<BF>::sc + kC * 4); };
    auto load_last = [&](const RowBuf& b) {
        glast = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, 0, Rec<BF>::sc + (kC - 1) * 4, 0));
    };
    auto load_t = [&](Frag<NS>(&to)[kTri], const RowBuf& b, int f) { to[f] = buf_frag<NS>(b, Rec<BF>::t, f, lane); };
    Stage<BF, DK, Cfg::SELF ? 4 : 1> rk;
    StageV4 rv;
    auto self_load = [&](int c) {
        load_tile(rk, kbase, krow, a.sh.ldk, c, wave);
        load_vt(rv, c, wave);
    };
    auto self_store = [&](int c) {
        if constexpr (Cfg::SELF) {
            rk.store(l.k[c & 1], lane, wave);
            rv.store(l.v[c & 1], lane, wave);
        }
    };
    if (nch > 0) {
        if constexpr (Cfg::SELF) {
            self_load(0);
            self_store(0);
            self_load(1);
        }
        const RowBuf vb = vbuf(0), rb = plain_buf(rec, Rec<BF>::bytes);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (!BF) load_v(vb, t);
            load_gam(rb, t);
            load_kap(rb, t);
        }
        load_last(rb);
#pragma unroll
        for (int f = 0; f < kTri; ++f) load_t(Tab[0], rb, f);
        lds_barrier();  // K of the first chunk is in LDS
    }
    // this block's fragments of the backward, one chunk's behind another's
    const bool kept = MODE == kScanKeep && blk < a.nb16;
    using Kp = Kept<BF, KS>;
    unsigned char* s0p = !kept ? nullptr : (unsigned char*)a.s0 + ((slot0 * hv + h) * a.nb16 + blk) * (int64_t)Kp::state;
    unsigned char* up = !kept ? nullptr : (unsigned char*)a.u + ((slot0 * hv + h) * a.nb16 + blk) * (int64_t)Kp::rows;
    constexpr int X2 = NI == 1 ? NE : 6, X3 = NS == 3 ? 6 : NE == 3 ? 5 : 3;  // matrix instructions per product
    // one chunk; T alternates between two sets of registers
    auto chunk = [&](int c, Frag<NS>(&Tf)[kTri], Frag<NS>(&Tn)[kTri]) {
        if (c + 1 < nch) rec += recstep;  // loaded for the next chunk; the last one reads itself again
        const RowBuf vb = vbuf(c + 1 < nch ? c + 1 : c), rb = plain_buf(rec, Rec<BF>::bytes);
        const Tile<NI, DK>& K = l.k[c & (BUF - 1)];
        if constexpr (MODE == kScanKeep) {
            if (kept)
#pragma unroll
                for (int s = 0; s < KS; ++s) keep_frag<BF>(s0p, true, KS, s, lane, S[2 * s], S[2 * s + 1]);
            s0p += (int64_t)hv * a.nb16 * Kp::state;
        }
        __builtin_amdgcn_sched_barrier(0);
        // e = V - exp(G) K S; LDS reads two steps ahead of their products
        f32x4 x[4] = {};
        Frag<NI> ka[2][4];
        auto read_rows = [&](int s) {
#pragma unroll
            for (int t = 0; t < 4; ++t) ka[s & 1][t] = K.rows(lane, t, s);
        };
        read_rows(0);
        read_rows(1);
        u32x2 v4[4];
        if constexpr (BF) {
#pragma unroll
            for (int t = 0; t < 4; ++t) v4[t] = l.v[c & (BUF - 1)].rows4(lane, t, 16 * wave);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            mma_tiles(ka[s & 1], sf[s], x);
            if constexpr (OUT) {
#pragma unroll
                for (int p = 0; p < NO; ++p) *reinterpret_cast<bf16x8*>(&l.x[wave][c & 1].s[s][p][lane * 8]) = sf[s].p[p];
            }
            if (s + 2 < KS) read_rows(s + 2);
            if constexpr (BF) {
#pragma unroll
                for (int f = s * kTri / KS; f < (s + 1) * kTri / KS; ++f) load_t(Tn, rb, f);
            }
            if constexpr (Cfg::SELF)
                if (s == KS - 1) {
                    self_store(c + 1);
                    self_load(c + 2);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        Frag<NI> kt[2][MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) kt[0][m] = K.cols(lane, m, 0);
        __builtin_amdgcn_sched_barrier(0);
        Frag<NE> ef[2];
        auto residual = [&](int p) {
#pragma unroll
            for (int t = 2 * p; t < 2 * p + 2; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v;
                    if constexpr (BF)
                        v = __uint_as_float(i & 1 ? v4[t][i >> 1] & 0xffff0000u : v4[t][i >> 1] << 16);
                    else
                        v = __uint_as_float(V[t][i]);
                    x[t][i] = fmaf(-gam[t][i], x[t][i], v);
                }
                if (!BF) load_v(vb, t);
                load_gam(rb, t);
            }
            ef[p] = pair_frag<NE>(x[2 * p], x[2 * p + 1], minus);
        };
        residual(0);
        __builtin_amdgcn_sched_barrier(0);
        // u = T diag(beta) e, the second half of e split meanwhile
        f32x4 u[4] = {};
        const Frag<NS> t0[4] = {Tf[0], Tf[1], Tf[2], Tf[4]};
        mma_tiles(t0, ef[0], u);
        residual(1);
        interleave<4 * X3, 4, 1>();
        const Frag<NS> t1[2] = {Tf[3], Tf[5]};
        mma_tiles(t1, ef[1], u + 2);
        Frag<NE> kf[2];
        kf[0] = pair_frag<NE>(kap[0] * u[0], kap[1] * u[1], minus);
#pragma unroll
        for (int m = 0; m < MT; ++m) S[m] *= glast;
        interleave<2 * X3, 12, 0>();
        if constexpr (!BF) {
#pragma unroll
            for (int f = 0; f < kTri; ++f) load_t(Tn, rb, f);
        }
        load_kap(rb, 0);
        load_kap(rb, 1);
        load_last(rb);
#pragma unroll
        for (int m = 0; m < MT; ++m) kt[1][m] = K.cols(lane, m, 1);
        __builtin_amdgcn_sched_barrier(0);
        // S = exp(G_last) S + K^T diag(exp(G_last - G)) u: the second half of u is split
        // during the first products, and the new state's parts two tiles at a time
        auto update = [&](int s, int p) {
            const Frag<NI> w[2] = {kt[s][2 * p], kt[s][2 * p + 1]};
            mma_tiles(w, kf[s], S + 2 * p);
        };
        f32x4 rest[MT];
        auto next_part = [&](int p, int n) {
            const f32x4 &a = rest[2 * p], &b = rest[2 * p + 1];
            const u32x4 w = {pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(b[0], b[1]), pack2(b[2], b[3])};
            sf[p].p[n] = __builtin_bit_cast(bf16x8, w);
            if (n + 1 < NS) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    rest[2 * p + t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus.a[t], sf[p].p[n], rest[2 * p + t], 0, 0, 0);
            }
        };
        auto first_part = [&](int p) {
            rest[2 * p] = S[2 * p];
            rest[2 * p + 1] = S[2 * p + 1];
            next_part(p, 0);
        };
        auto last_parts = [&](int p) {
#pragma unroll
            for (int n = 1; n < NS; ++n) next_part(p, n);
        };
#pragma unroll
        for (int p = 0; p < KS; ++p) update(0, p);
        kf[1] = pair_frag<NE>(kap[2] * u[2], kap[3] * u[3], minus);
        load_kap(rb, 2);
        load_kap(rb, 3);
        interleave<MT * X2, 5, 1>();
        if constexpr (OUT) {
#pragma unroll
            for (int t = 0; t < 4; ++t) l.x[wave][c & 1].u[t][lane] = u[t];
        } else if constexpr (MODE == kScanKeep) {
            if (kept)
#pragma unroll
                for (int s = 0; s < 2; ++s) keep_frag<BF>(up, true, 2, s, lane, u[2 * s], u[2 * s + 1]);
            up += (int64_t)hv * a.nb16 * Kp::rows;
        }
        // the new state's parts, two tiles at a time: first part a step behind the products,
        // its remainder and second part another step, so that none waits for a result
#pragma unroll
        for (int p = 0; p < KS + 2; ++p) {
            if (p < KS) update(1, p);
            if (p >= 1 && p <= KS) first_part(p - 1);
            if (p >= 2) last_parts(p - 2);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (BUF == 1) lds_barrier();  // K may be replaced
        lds_barrier();                // chunk c's operands and the next K are in LDS
    };
    int c = 0;
    for (; c + 1 < nch; c += 2) {
        chunk(c, Tab[0], Tab[BF ? 1 : 0]);
        chunk(c + 1, Tab[BF ? 1 : 0], Tab[0]);
    }
    if (c < nch) chunk(c, Tab[0], Tab[BF ? 1 : 0]);
    if constexpr (ENDS) {
        if (!onm) {
            if (blk < a.nb16)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    *reinterpret_cast<f32x4*>(bp + ps * (hv * bsize) + (t * 64 + lane) * 4) = S[t];
        } else if (c0 < DK) {
            const int64_t at = ((pslot + ps) * hv + h) * msize;
            store_end<NS, DK>(a.pieces.m + at, a.pieces.mt ? a.pieces.mt + at : nullptr, S, c0, lane);
        }
        return;
    }
    if (a.s_out && last)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = drow(t, i);
                if (cok && k < dk) a.s_out[((n * hv + h) * dk + k) * dv + c0] = S[t][i];
            }
}

}  // namespace delta
}  // namespace hy
