// Chunk-parallel preparation of the gated delta rule: the decays, T = (I + A)^-1 and
// P of every (chunk, value head), written as matrix-core fragments so that the scans
// read them 16 bytes per lane without staging. Bound by those records' and the operands'
// bytes: 8 sequences of 8192 tokens, 6 heads of 128, bf16, 84 us (367 MB, 4.4 TB/s), for the
// backward, with T^T and P^T, 97 us (480 MB, 5.0 TB/s).
#pragma once
#include "delta.hpp"

namespace hy {
namespace delta {

struct PrepArgs {
    Seqs seqs;
    Shape sh;
    const void *q, *k, *g, *beta;
    Prep out;
};

constexpr int kMP = 68;  // LDS pitch (floats) of a 64 x 64 matrix: rows 16-byte aligned, four banks apart

template <bool BF, int DK>
struct PrepLds {
    using T = typename Io<BF>::T;
    static constexpr int KP = DK + 32 / (int)sizeof(T);  // row pitch of the staged K tile: 32 bytes over spread its reads
    float a[kC][kMP];
    union {
        alignas(16) T rows[kC][KP];  // K, until its products are made
        float p[kC][kMP];            // then P, then T
    };
    double G[kC];
    float beta[kC], kk[kC];
};

// a 64 x 64 matrix in LDS (or its transpose; or with column c scaled by scale[c]) as
// block-triangular A fragments of N parts
template <int N, bool TRANS>
__device__ __forceinline__ void write_tri(const float (*m)[kMP], const float* scale, __bf16* dst, int tid) {
    for (int e = tid; e < kTri * 64; e += kThreads) {
        const int f = e >> 6, lane = e & 63;
        const int i = TRANS ? (f < 4 ? f >> 1 : f - 2) : tri_row(f);
        const int s = TRANS ? (f < 4 ? f & 1 : 1) : tri_half(f);
        const int row = tile_row(i, lane & 15), c0 = 32 * s + 8 * (lane >> 4);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (TRANS ? m[c0 + j][row] : m[row][c0 + j]) * (scale ? scale[c0 + j] : 1.f);
        const Frag<N> fr = split8<N>(x);
#pragma unroll
        for (int n = 0; n < N; ++n) *reinterpret_cast<bf16x8*>(dst + ((int64_t)f * N + n) * 512 + lane * 8) = fr.p[n];
    }
}

// One workgroup per (slot, value head). Tiles of K K^T and Q K^T by bf16 matrix
// products; the 16 x 16 diagonal blocks of I + A inverted by forward substitution in
// fp32 (one wave each), the blocks below by T_ij = -T_ii sum_k A_ik T_kj on the fp32
// matrix instruction, one block diagonal at a time: nothing of T is rounded before
// its parts are written.
template <bool BF, int DK, bool BWD>
__global__ __launch_bounds__(kThreads) void k_delta_prep(PrepArgs a) {
    using IO = Io<BF>;
    using T = typename IO::T;
    extern __shared__ __align__(16) unsigned char lds_raw[];
    PrepLds<BF, DK>& l = *reinterpret_cast<PrepLds<BF, DK>*>(lds_raw);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, col = lane & 15;
    const int64_t slot = blockIdx.x;
    const int h = blockIdx.y, hk = h / a.sh.group;
    Range r;
    int64_t c, n;
    if (!find_chunk(a.seqs, slot, r, c, n)) return;
    const int64_t tok = uniform64(r.first + c * kC);
    const int rows = __builtin_amdgcn_readfirstlane((int)(r.len - c * kC < kC ? r.len - c * kC : kC));
    const int64_t sh_idx = slot * a.sh.hv + h;
    const T* kp = (const T*)a.k + tok * a.sh.ldk + (int64_t)hk * a.sh.dk;
    const T* qp = (const T*)a.q + tok * a.sh.ldq + (int64_t)hk * a.sh.dk;

    // the loads of K and Q are on their way while every wave sums the decays for itself
    constexpr int V = 16 / (int)sizeof(T), NL = kC * (DK / V) / kThreads;
    const uint32_t E = sizeof(T), ldk = (uint32_t)a.sh.ldk * E, ldq = (uint32_t)a.sh.ldq * E;
    const RowBuf kb = row_buf(kp, rows, ldk, a.sh.dk * E), qb = row_buf(qp, rows, ldq, a.sh.dk * E);
    f32x4 kr[NL];
#pragma unroll
    for (int e = 0; e < NL; ++e) {
        const int t = (e * kThreads + tid) / (DK / V), k = (e * kThreads + tid) % (DK / V) * V;
        kr[e] = buf_f4(kb, k < a.sh.dk ? t * ldk + k * E : kNoElem, 0);
    }
    Raw<BF> qr[DK / 32];
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
        const int k0 = 32 * s + 8 * g;
        buf_raw(qb, k0 < a.sh.dk ? (16 * wave + col) * ldq + k0 * E : kNoElem, qr[s]);
    }
    float gv = 0.f, bv = 0.f;
    if (lane < rows) {
        gv = (float)((const T*)a.g)[(tok + lane) * a.sh.hv + h];
        bv = (float)((const T*)a.beta)[(tok + lane) * a.sh.hv + h];
    }
    const double G = chunk_decay(gv, lane);
    if (wave == 0) {
        l.G[lane] = G;
        l.beta[lane] = BWD ? held_beta(bv) : bv;
    } else if (wave == 1) {
        const double last = __shfl(G, 63);
        float* sc = reinterpret_cast<float*>(a.out.rec + sh_idx * Rec<BF>::bytes + Rec<BF>::sc);
        sc[lane] = decay(G);
        sc[kC + lane] = decay(last - G);
        sc[2 * kC + lane] = bv;
    }
#pragma unroll
    for (int e = 0; e < NL; ++e) {
        const int t = (e * kThreads + tid) / (DK / V), k = (e * kThreads + tid) % (DK / V) * V;
        *reinterpret_cast<f32x4*>(&l.rows[t][k]) = kr[e];
    }
    __syncthreads();

    // wave w: row tile w of A and P
    {
        f32x4 kk[4] = {}, qk[4] = {};
        const int row = 16 * wave + col;
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) {
            const int k0 = 32 * s + 8 * g;
            float x[8];
            load8(&l.rows[row][k0], true, x);
            const Frag<IO::NI> ka = split8<IO::NI>(x);
            const Frag<IO::NI> qa = to_frag(qr[s]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= wave) {
                    load8(&l.rows[16 * j + col][k0], true, x);
                    const Frag<IO::NI> kb = split8<IO::NI>(x);
                    kk[j] = mma(ka, kb, kk[j]);
                    qk[j] = mma(qa, kb, qk[j]);
                }
        }
        if (!BWD && col >> 2 == g) {  // this lane has a k_t . k_t
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (j == wave && (col & 3) == i) l.kk[row] = kk[j][i];
        }
        __syncthreads();  // K has been read: P takes its place
        // no branches around single elements: their decays are formed everywhere and selected
        const int t0 = 16 * wave + 4 * g;
        double Gi[4];
        float bi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Gi[i] = l.G[t0 + i];
            bi[i] = l.beta[t0 + i];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int tj = 16 * j + col;
            const double Gj = l.G[tj];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float d = decay(Gi[i] - Gj);
                l.a[t0 + i][tj] = tj < t0 + i ? bi[i] * d * kk[j][i] : 0.f;
                l.p[t0 + i][tj] = tj <= t0 + i ? d * qk[j][i] : 0.f;
            }
        }
    }
    __syncthreads();
    // From the first token on whose k, g or beta is not finite, the rows of A and P are cleared,
    // so that no part of T or P of the tokens in front of it meets it; T's diagonal marks them
    // below (the forward; the backward's gradients reach back anyway).
    int good = kC;
    if (!BWD) {
        const uint64_t bad = __ballot(!(finite(l.kk[lane]) && finite(l.beta[lane]) && finite((float)l.G[lane])));
        if (__builtin_expect(bad != 0, 0)) {
            good = __builtin_ctzll(bad);
            for (int e = good * kC + tid; e < kC * kC; e += kThreads) l.a[e / kC][e % kC] = l.p[e / kC][e % kC] = 0.f;
            __syncthreads();
        }
    }
    if (!BWD)
        write_tri<IO::NP, false>(l.p, nullptr, reinterpret_cast<__bf16*>(a.out.rec + sh_idx * Rec<BF>::bytes + Rec<BF>::p), tid);
    else
        write_tri<IO::NE, true>(l.p, nullptr, reinterpret_cast<__bf16*>(a.out.back + sh_idx * Rec<BF>::back + Rec<BF>::pt), tid);
    __syncthreads();

    // T over P. Diagonal block `wave`: column `col` of the inverse, x_i = e_i - sum_{j<i} A_ij x_j
    {
        const int b = 16 * wave;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == col ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; j += 4) {  // A is zero on and above the diagonal
                const f32x4 row = *reinterpret_cast<const f32x4*>(&l.a[b + i][b + j]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < i) v = fmaf(-row[e], x[j + e], v);
            }
            x[i] = v;
        }
        if (g == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) l.p[b + i][b + col] = x[i];
        // the blocks above the diagonal are zero
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j > wave)
#pragma unroll
                for (int i = 0; i < 4; ++i) l.p[b + 4 * g + i][16 * j + col] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int d = 1; d < 4; ++d) {
        if (wave >= d) {
            const int j = wave - d, b = 16 * wave;
            f32x4 x = {};
            for (int k = j; k < wave; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    x = __builtin_amdgcn_mfma_f32_16x16x4f32(l.a[b + col][16 * k + 4 * s + g],
                                                             l.p[16 * k + 4 * s + g][16 * j + col], x, 0, 0, 0);
            // rows 4g + s of x in this lane: contract over {4g + s : g} at each s
            f32x4 y = {};
#pragma unroll
            for (int s = 0; s < 4; ++s)
                y = __builtin_amdgcn_mfma_f32_16x16x4f32(l.p[b + col][b + 4 * g + s], x[s], y, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) l.p[b + 4 * g + i][16 * j + col] = -y[i];
        }
        __syncthreads();
    }
    if (!BWD && good < kC) {
        if (wave == 0 && lane >= good) {
            l.p[lane][lane] = __builtin_nanf("");
            l.beta[lane] = 1.f;
        }
        __syncthreads();
    }
    write_tri<IO::NS, false>(l.p, l.beta, reinterpret_cast<__bf16*>(a.out.rec + sh_idx * Rec<BF>::bytes), tid);
    if (BWD)
        write_tri<IO::NS, true>(l.p, nullptr, reinterpret_cast<__bf16*>(a.out.back + sh_idx * Rec<BF>::back), tid);
}

}  // namespace delta
}  // namespace hy
