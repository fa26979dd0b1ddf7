// The backward's chunk-parallel part: with the state S0 before and its gradient dS1
// behind every chunk, the written values u and the residuals' gradients r, the gradients
// of q, k, v, g and beta. Per chunk and value head, with D_ij = exp(G_i - G_j),
// W_ij = scale D_ij (dO_i . u_j) for j <= i, M_ij = -beta_i D_ij (r_i . u_j) for j < i:
//   dQ = scale diag(exp G) dO S0^T + W K
//   dK = -diag(exp(G) beta) r S0^T + diag(exp(G_last - G)) u dS1^T + W^T Q + (M + M^T) K
//   dV = diag(beta) r,   dbeta_i = r_i . u_i / beta_i
//   dG_i = scale exp(G_i) q_i . (dO S0^T)_i - beta_i exp(G_i) k_i . (r S0^T)_i
//          + sum_j X_ij - sum_j X_ji - exp(G_last - G_i) k_i . (u dS1^T)_i,
//   X_ij = W_ij q_i . k_j + M_ij k_i . k_j,
//   dG_last += sum_i exp(G_last - G_i) k_i . (u dS1^T)_i + exp(G_last) <dS1, S0>,
// and dg_t is the sum of dG_i over i >= t. u_i / beta_i is what the state's answer to k_i
// lacks of v_i. Formed here as that difference, r . v - r . answer, it would keep the roundings
// of both where they cancel (an answer within 1% of v: dbeta 0.18 off); beta = 0 is held at 2^-90.
// A workgroup holds K and Q in LDS and walks over 32 columns of v's width at a time (dO,
// u, r and the states' columns, the next step's loads in flight), bf16 calls in two halves,
// dS1 in the place of S0; wave w has rows 16 w of every product. Bound by bytes and their
// latency with two workgroups a CU: 8 sequences of 8192 tokens, 6 heads of 128 x 128, bf16,
// 378 us (1571 MB, 4.2 TB/s).
#pragma once
#include "delta.hpp"

namespace hy {
namespace delta {

struct GradArgs {
    Seqs seqs;
    Shape sh;
    const void *q, *k, *g, *beta, *dout;
    const void *s0, *ds1, *u, *r;  // as Kept
    void *dq, *dk;       // [tokens][hk][dk]
    void* dv;            // [tokens][hv][dv]
    void *dg, *dbeta;    // [tokens][hv]
};

// R rows of W elements in LDS, natural order; fp32 is split when read
template <bool BF, int R, int W>
struct GradTile;
template <int R, int W>
struct GradTile<true, R, W> {
    using T = __bf16;
    static constexpr int pitch = 2 * W + 16;
    alignas(16) unsigned char b[R * pitch];
    __device__ __forceinline__ u32x4* at16(int row, int e) { return reinterpret_cast<u32x4*>(b + row * pitch + 2 * e); }
    __device__ __forceinline__ float get(int row, int e) const {
        return (float)*reinterpret_cast<const __bf16*>(b + row * pitch + 2 * e);
    }
    __device__ __forceinline__ void put(int row, int e, float x) { *reinterpret_cast<__bf16*>(b + row * pitch + 2 * e) = (__bf16)x; }
    __device__ __forceinline__ Frag<1> rows(int lane, int t, int s) const {
        return Frag<1>{{*reinterpret_cast<const bf16x8*>(b + (16 * t + (lane & 15)) * pitch + 64 * s + 16 * (lane >> 4))}};
    }
    __device__ __forceinline__ Frag<1> cols(int lane, int m, int s) const {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        typedef __attribute__((address_space(3))) s16x4* Lds4;
        const unsigned char* p = b + (32 * s + 8 * (lane >> 4) + ((lane & 15) >> 2)) * pitch + 32 * m + 8 * (lane & 3);
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(p + 4 * pitch));
        return Frag<1>{{__builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7))}};
    }
};
template <int R, int W>
struct GradTile<false, R, W> {
    using T = float;
    static constexpr int pitch = 4 * W + 16;
    alignas(16) unsigned char b[R * pitch];
    __device__ __forceinline__ u32x4* at16(int row, int e) { return reinterpret_cast<u32x4*>(b + row * pitch + 4 * e); }
    __device__ __forceinline__ float get(int row, int e) const { return *reinterpret_cast<const float*>(b + row * pitch + 4 * e); }
    __device__ __forceinline__ void put(int row, int e, float x) { *reinterpret_cast<float*>(b + row * pitch + 4 * e) = x; }
    __device__ __forceinline__ Frag<3> rows(int lane, int t, int s) const {
        float x[8];
        load8(reinterpret_cast<const float*>(b + (16 * t + (lane & 15)) * pitch + 128 * s + 32 * (lane >> 4)), true, x);
        return split8<3>(x);
    }
    __device__ __forceinline__ Frag<3> cols(int lane, int m, int s) const {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = get(32 * s + 8 * (lane >> 4) + i, 16 * m + (lane & 15));
        return split8<3>(x);
    }
};

// W rows (state rows or tokens) of 32 columns out of the scans' fragments, read as an
// operand whose contraction runs over the columns: bf16 stays column by column and is read
// across; fp32 is turned when it is stored.
template <bool BF, int W>
struct StepTile;
template <int W>
struct StepTile<true, W> : GradTile<true, 32, W> {
    __device__ __forceinline__ void put8(int c, int e, const bf16x8& x) { *this->at16(c, e) = __builtin_bit_cast(u32x4, x); }
    __device__ __forceinline__ Frag<1> op(int lane, int m) const { return this->cols(lane, m, 0); }
};
template <int W>
struct StepTile<false, W> : GradTile<false, W, 32> {
    __device__ __forceinline__ void put8(int c, int e, const float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) this->put(e + i, c, x[i]);
    }
    __device__ __forceinline__ Frag<3> op(int lane, int m) const { return this->rows(lane, m, 0); }
};

// A 64 x 64 matrix as a left operand: in bf16 calls two tiles, its parts (with one each dQ and
// dK were off by a fifth more than by their own rounding; 7% of the kernel's time).
template <bool BF>
struct GradMat {
    GradTile<BF, kC, kC> part[BF ? 2 : 1];
    __device__ __forceinline__ void put(int row, int e, float x) {
        part[0].put(row, e, x);
        if constexpr (BF) part[1].put(row, e, x - (float)(__bf16)x);
    }
    __device__ __forceinline__ auto rows(int lane, int t, int s) const {
        if constexpr (BF)
            return Frag<2>{{part[0].rows(lane, t, s).p[0], part[1].rows(lane, t, s).p[0]}};
        else
            return part[0].rows(lane, t, s);
    }
    __device__ __forceinline__ auto cols(int lane, int t, int s) const {
        if constexpr (BF)
            return Frag<2>{{part[0].cols(lane, t, s).p[0], part[1].cols(lane, t, s).p[0]}};
        else
            return part[0].cols(lane, t, s);
    }
};

template <bool BF, int DK>
struct GradLds {
    GradTile<BF, kC, DK> k, q;
    struct Steps {
        GradTile<BF, kC, 32> o;
        StepTile<BF, kC> u[Io<BF>::NK], r[Io<BF>::NK];
        StepTile<BF, DK> st[2];  // bf16: both parts of S0, then of dS1; fp32: S0 and dS1
    };
    struct Mats {
        GradMat<BF> w, n;
    };
    union {
        Steps step;  // 32 columns of v's width
        Mats mat;    // after the last of them
    };
    double G[kC];
    float gam[kC], kap[kC], bet[kC], row[kC], kus[kC], ru[kC];
    float cs[4][kC];
    float red[4];
};

template <bool BF, int DK, bool SHARED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu((BF && !SHARED ? 2 : 1))))
void k_delta_grad(GradArgs a) {
    using T = typename Io<BF>::T;
    constexpr int MT = DK / 16, KS = DK / 32;
    constexpr uint32_t E = sizeof(T);
    constexpr int V = 16 / (int)E, LPR = 32 / V;  // elements of 16 bytes; lanes of a 32-element row
    constexpr int RPP = kThreads / LPR;           // rows one pass of the workgroup stages
    constexpr int NR = kC / RPP;                  // passes for 64 rows
    constexpr int NF = DK / 64;                   // state fragments a wave stages (of 2 KS)
    constexpr int NK = Io<BF>::NK;
    using Kp = Kept<BF, KS>;
    extern __shared__ __align__(16) unsigned char lds_raw[];
    GradLds<BF, DK>& l = *reinterpret_cast<GradLds<BF, DK>*>(lds_raw);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, col = lane & 15;
    const int64_t slot = blockIdx.x;
    const int hk = blockIdx.y;
    Range rg;
    int64_t c, n;
    if (!find_chunk(a.seqs, slot, rg, c, n)) return;
    const int64_t tok = uniform64(rg.first + c * kC);
    const int rows = __builtin_amdgcn_readfirstlane((int)(rg.len - c * kC < kC ? rg.len - c * kC : kC));
    const int hv = a.sh.hv, dk = a.sh.dk, dv = a.sh.dv;
    const uint32_t ldk = (uint32_t)a.sh.ldk * E, ldq = (uint32_t)a.sh.ldq * E, ldo = (uint32_t)(hv * dv) * E;

    {  // K and Q
        const RowBuf kb = row_buf((const T*)a.k + tok * a.sh.ldk + (int64_t)hk * dk, rows, ldk, dk * E);
        const RowBuf qb = row_buf((const T*)a.q + tok * a.sh.ldq + (int64_t)hk * dk, rows, ldq, dk * E);
#pragma unroll
        for (int e = 0; e < kC * (DK / V) / kThreads; ++e) {
            const int x = e * kThreads + tid, t = x / (DK / V), k = x % (DK / V) * V;
            *l.k.at16(t, k) = __builtin_bit_cast(u32x4, buf_f4(kb, k < dk ? t * ldk + k * E : kNoElem, 0));
            *l.q.at16(t, k) = __builtin_bit_cast(u32x4, buf_f4(qb, k < dk ? t * ldq + k * E : kNoElem, 0));
        }
    }
    f32x4 dq[MT] = {}, dkk[MT] = {};
    const int srow = tid / LPR, scol = tid % LPR * V;
    for (int hh = 0; hh < (SHARED ? a.sh.group : 1); ++hh) {
        const int h = hk * a.sh.group + hh;
        const int64_t obase = (tok * hv + h) * (int64_t)dv;
        const int nb16 = (dv + 15) / 16;
        const int64_t fidx = (slot * hv + h) * nb16;  // first block's fragments
        const RowBuf ob = row_buf((const T*)a.dout + obase, rows, ldo, dv * E);
        const RowBuf vo = row_buf((T*)a.dv + obase, rows, ldo, dv * E);
        const RowBuf ub = plain_buf((const unsigned char*)a.u + fidx * Kp::rows, nb16 * Kp::rows);
        const RowBuf rb = plain_buf((const unsigned char*)a.r + fidx * Kp::rows, nb16 * Kp::rows);
        const RowBuf sb = plain_buf((const unsigned char*)a.s0 + fidx * Kp::state, nb16 * Kp::state);
        const RowBuf db = plain_buf((const unsigned char*)a.ds1 + fidx * Kp::state, nb16 * Kp::state);
        // a step's 2 blocks: wave w stages fragment w of the four of u and r and fragments
        // NF w .. of the 2 KS of the states; blocks past the last read zeros
        u32x4 po[NR];
        KeptRaw<BF> pu, pr, ps[NF], pd[NF];
        auto fetch = [&](int c0) {
            const bool ok = c0 + scol < dv;
#pragma unroll
            for (int i = 0; i < NR; ++i)
                po[i] = __builtin_bit_cast(u32x4, buf_f4(ob, ok ? (i * RPP + srow) * ldo + (c0 + scol) * E : kNoElem, 0));
            const uint32_t rows = (c0 / 16) * Kp::rows + w * Kp::frag, states = (c0 / 16) * Kp::state + NF * w * Kp::frag;
            pu.load(ub, rows, lane);
            pr.load(rb, rows, lane);
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                ps[f].load(sb, states + f * Kp::frag, lane);
                pd[f].load(db, states + f * Kp::frag, lane);
            }
        };
        // into LDS: rows' fragment w, all parts; the states', first parts (the second returned)
        auto put_rows = [&](StepTile<BF, kC>(&t)[NK], const KeptRaw<BF>& p) {
            float x[8];
            p.get(x);
            const int c = 16 * (w >> 1) + col, e = 32 * (w & 1) + 8 * g;
            if constexpr (BF) {
                const Frag<NK> f = split8<NK>(x);
#pragma unroll
                for (int n = 0; n < NK; ++n) t[n].put8(c, e, f.p[n]);
            } else {
                t[0].put8(c, e, x);
            }
        };
        auto put_state = [&](const KeptRaw<BF>(&p)[NF], int t) {
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int x = NF * w + f, c = 16 * (x / KS) + col, e = 32 * (x % KS) + 8 * g;  // block x / KS, step x % KS
                float y[8];
                p[f].get(y);
                if constexpr (BF) {
                    const Frag<NK> parts = split8<NK>(y);
#pragma unroll
                    for (int n = 0; n < NK; ++n) l.step.st[n].put8(c, e, parts.p[n]);
                } else {
                    l.step.st[t].put8(c, e, y);
                }
            }
        };
        // <dS1, S0> goes into dg of every token of the chunk and beyond: from all bits of both
        // (from bf16 alone dg was up to 6.7e-3 off where the final states' gradient outweighs
        // the outputs')
        auto dot_states = [&]() {
            float dot = 0.f;
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                float s[8], d[8];
                ps[f].get(s);
                pd[f].get(d);
#pragma unroll
                for (int i = 0; i < 8; ++i) dot = fmaf(s[i], d[i], dot);
            }
            return dot;
        };
        fetch(0);
        if (w == 0) {
            const float bv = buf_elem<BF>(row_buf((const T*)a.beta + tok * hv + h, rows, hv * E, E), lane * (hv * E));
            const double G = chunk_decay(buf_elem<BF>(row_buf((const T*)a.g + tok * hv + h, rows, hv * E, E), lane * (hv * E)), lane);
            const double last = __shfl(G, 63);
            l.G[lane] = G;
            l.gam[lane] = decay(G);
            l.kap[lane] = decay(last - G);
            l.bet[lane] = bv;
        }
        f32x4 dp[4] = {}, z[4] = {}, qs[MT] = {}, rs[MT] = {}, us[MT] = {};
        float sd = 0.f;  // this thread's part of <dS1, S0>
        for (int c0 = 0; c0 < dv; c0 += 32) {
            __syncthreads();  // the step before (or the head before) has read its tiles
#pragma unroll
            for (int i = 0; i < NR; ++i) *l.step.o.at16(i * RPP + srow, scol) = po[i];
            put_rows(l.step.u, pu);
            __builtin_amdgcn_sched_barrier(0);
            put_rows(l.step.r, pr);
            __builtin_amdgcn_sched_barrier(0);
            put_state(ps, 0);
            __builtin_amdgcn_sched_barrier(0);
            sd += dot_states();
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (!BF) {
                put_state(pd, 1);
                if (c0 + 32 < dv) fetch(c0 + 32);
            }
            lds_barrier();
            auto parts = [&](const auto& t, int m) {
                if constexpr (BF)
                    return Frag<2>{{t[0].op(lane, m).p[0], t[1].op(lane, m).p[0]}};
                else
                    return t[0].op(lane, m);
            };
            const auto ao = l.step.o.rows(lane, w, 0);
            const auto ar = parts(l.step.r, w), au = parts(l.step.u, w);
            {  // dv: this lane has eight columns of one token of r
                const int t = 16 * w + col, at = c0 + 8 * g;
                const uint32_t off = at < dv ? t * ldo + at * E : kNoElem;
                const float b = l.bet[t];
                if constexpr (BF) {
                    u32x4 x;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = pack2(b * ((float)ar.p[0][2 * i] + (float)ar.p[1][2 * i]),
                                     b * ((float)ar.p[0][2 * i + 1] + (float)ar.p[1][2 * i + 1]));
                    __builtin_amdgcn_raw_buffer_store_b128(x, vo, (int)off, 0, 0);
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        f32x4 x = *reinterpret_cast<const f32x4*>(l.step.r[0].at16(t, 8 * g + 4 * j));
                        x *= b;
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), vo, (int)(off + 16 * j), 0, 0);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) {
                    const auto b = parts(l.step.u, j);
                    dp[j] = mma(ao, b, dp[j]);
                    z[j] = mma(ar, b, z[j]);
                }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const auto b = parts(l.step.st, m);
                qs[m] = mma(ao, b, qs[m]);
                rs[m] = mma(ar, b, rs[m]);
                if constexpr (!BF) us[m] = mma(au, l.step.st[1].op(lane, m), us[m]);
                if (BF && (m & 1)) __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (BF) {
                lds_barrier();  // S0 has been read
                put_state(pd, 0);
                if (c0 + 32 < dv) fetch(c0 + 32);
                lds_barrier();
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    us[m] = mma(au, parts(l.step.st, m), us[m]);
                    if (m & 1) __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        // the lane anew, so that no address below is formed before the steps and held through them
        int thread = tid;
        asm volatile("" : "+v"(thread));
        const int lane = thread & 63, g = lane >> 4, col = lane & 15;
        // k_i . k_j and q_i . k_j
        f32x4 kk[4] = {}, qk[4] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const auto ka = l.k.rows(lane, w, s), qa = l.q.rows(lane, w, s);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) {
                    const auto b = l.k.rows(lane, j, s);
                    kk[j] = mma(ka, b, kk[j]);
                    qk[j] = mma(qa, b, qk[j]);
                }
        }
        // sums along rows over the sixteen lanes of a row
        auto row_sum = [&](f32x4 x) {
#pragma unroll
            for (int d = 1; d < 16; d <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] += __shfl_xor(x[i], d);
            return x;
        };
        f32x4 qqs = {}, krs = {}, kus = {}, rx = {};
        const int ti = 16 * w + 4 * g;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float kv = l.k.get(ti + i, 16 * m + col);
                qqs[i] = fmaf(l.q.get(ti + i, 16 * m + col), qs[m][i], qqs[i]);
                krs[i] = fmaf(kv, rs[m][i], krs[i]);
                kus[i] = fmaf(kv, us[m][i], kus[i]);
                if (i == 3) __builtin_amdgcn_sched_barrier(0);
            }
        qqs = row_sum(qqs);
        krs = row_sum(krs);
        kus = row_sum(kus);
        const f32x4 gam = *reinterpret_cast<const f32x4*>(l.gam + ti), kap = *reinterpret_cast<const f32x4*>(l.kap + ti);
        const f32x4 bet = *reinterpret_cast<const f32x4*>(l.bet + ti);
        // no branches around single elements: their decays are formed everywhere and selected
        if (col >> 2 == g) {  // this lane has a diagonal element of its wave's tile
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (j == w && (col & 3) == i) l.ru[16 * w + col] = z[j][i];
        }
        float cx[4] = {};
        double Gi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) Gi[i] = l.G[ti + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > w) continue;  // dp and z are zero there
            const int tj = 16 * j + col;
            const double Gj = l.G[tj];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = decay(Gi[i] - Gj);
                const float d = tj <= ti + i ? e : 0.f, ds = tj < ti + i ? e : 0.f;
                const float wv = tj <= ti + i ? a.sh.scale * d * dp[j][i] : 0.f;
                const float dz = tj < ti + i ? ds * z[j][i] : 0.f;
                const float mv = -bet[i] * dz;
                const float x = fmaf(mv, kk[j][i], wv * qk[j][i]);
                rx[i] += x;
                cx[j] += x;
                dp[j][i] = wv;
                z[j][i] = mv;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            cx[j] += __shfl_xor(cx[j], 16);
            cx[j] += __shfl_xor(cx[j], 32);
            if (g == 0) l.cs[w][16 * j + col] = cx[j];
        }
        rx = row_sum(rx);
        if (col == 0) {
            *reinterpret_cast<f32x4*>(l.row + ti) = a.sh.scale * gam * qqs - bet * gam * krs + rx;
            *reinterpret_cast<f32x4*>(l.kus + ti) = kap * kus;
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sd += __shfl_xor(sd, d);
        if (lane == 0) l.red[w] = sd;
        __syncthreads();  // the last step's tiles have been read: W and M take their place
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                l.mat.w.put(ti + i, 16 * j + col, dp[j][i]);
                l.mat.n.put(ti + i, 16 * j + col, z[j][i]);
            }
        __syncthreads();
        if (w == 0) {
            double d = (double)l.row[lane] - l.cs[0][lane] - l.cs[1][lane] - l.cs[2][lane] - l.cs[3][lane] - l.kus[lane];
            double ku = l.kus[lane];
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) ku += __shfl_xor(ku, s);
            if (lane == 63) d += ku + (double)l.gam[63] * ((double)l.red[0] + l.red[1] + l.red[2] + l.red[3]);
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) {
                const double up = __shfl_down(d, s);
                if (lane + s < 64) d += up;
            }
            buf_store<BF>(row_buf((T*)a.dg + tok * hv + h, rows, hv * E, E), lane * (hv * E), (float)d);
            buf_store<BF>(row_buf((T*)a.dbeta + tok * hv + h, rows, hv * E, E), lane * (hv * E), l.ru[lane] / held_beta(l.bet[lane]));
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            dq[m] += a.sh.scale * gam * qs[m];
            dkk[m] += kap * us[m] - gam * bet * rs[m];
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const auto na = l.mat.n.rows(lane, w, s), wa = l.mat.w.rows(lane, w, s);
            const auto nt = l.mat.n.cols(lane, w, s), wt = l.mat.w.cols(lane, w, s);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const auto kc = l.k.cols(lane, m, s);
                if (2 * s <= w) {
                    dq[m] = mma(wa, kc, dq[m]);
                    dkk[m] = mma(na, kc, dkk[m]);
                }
                if (2 * s + 1 >= w) {
                    dkk[m] = mma(nt, kc, dkk[m]);
                    dkk[m] = mma(wt, l.q.cols(lane, m, s), dkk[m]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // whole rows out, through the tiles of K and Q: 16 bytes a lane in place of single elements
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            l.q.put(16 * w + 4 * g + i, 16 * m + col, dq[m][i]);
            l.k.put(16 * w + 4 * g + i, 16 * m + col, dkk[m][i]);
        }
    __syncthreads();
    const uint32_t ldd = (uint32_t)(a.sh.hk * dk) * E;
    const RowBuf qo = row_buf((T*)a.dq + (tok * a.sh.hk + hk) * (int64_t)dk, rows, ldd, dk * E);
    const RowBuf ko = row_buf((T*)a.dk + (tok * a.sh.hk + hk) * (int64_t)dk, rows, ldd, dk * E);
#pragma unroll
    for (int e = 0; e < kC * (DK / V) / kThreads; ++e) {
        const int x = e * kThreads + tid, t = x / (DK / V), k = x % (DK / V) * V;
        const uint32_t off = k < dk ? t * ldd + k * E : kNoElem;
        __builtin_amdgcn_raw_buffer_store_b128(*l.q.at16(t, k), qo, (int)off, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(*l.k.at16(t, k), ko, (int)off, 0, 0);
    }
}

}  // namespace delta
}  // namespace hy
