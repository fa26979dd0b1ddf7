// Norms of the queries' and keys' heads with the position rotation in the same pass, and
// their backward, for gfx950. For a head's vector x [dim], weight w (optional) and F
// rotated pairs:
//   n = x s,  s = 1 / sqrt(mean(x^2) + eps) (rms) or 1 / sqrt(sum(x^2) + eps) (l2),
//   y = R (w n),  R turning pair i by position * freq[i];
// backward, with e = R^T dy:  dw = sum over tokens and heads of e n,
//   dx = s (w e - n c sum(w e n)),  c = 1 / dim (rms) or 1 (l2).
//
// One read and one write of every value: bound by memory. A group of G lanes (the power of
// two that gives each 8 elements) holds one head; lane l of the rotated part has four pairs
// whole, either 8 neighbours or 4 elements of each half, so the rotation needs no exchange.
// A group keeps its token and walks over heads, several in flight: the angles'
// reduction (64 bits: positions reach far beyond where a 32-bit product keeps a fraction of
// a turn) and sine are paid once a token and lane. Sums over the 8 elements and the G lanes
// are fp32 (a head whose squares pass 3e38 in sum gives zeros); the weights' gradients are summed in a fixed order (lane, workgroup, then over
// workgroups in 64 bits).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/hyena.h"
#include "plan.hpp"
#include "stream.hpp"

namespace hy {
namespace {

constexpr int kNormThreads = 256;
// Heads in flight per group where a group takes several; one where it has one (5 and 256
// tokens of 12 heads, in a graph: 3.1 and 3.4 us, with four 4.1 and 4.5; 65536 tokens: one
// 85, two 80, four 79 us; backward of 65536 and 16 heads: 89, 97, 92 us).
constexpr int kNormAhead = 4;
// Waves to aim for before a group takes several heads. 2048 tokens: 5.7 us with 2048, 7.4
// with 1024, 9.1 with 4096; backward of 4096 tokens 12.3, 13.0 and 18.6 us, of 16384 25.3,
// 25.3 and 31.4.
constexpr int kNormWaves = 2048;
constexpr int kNormBackWgs = 1024;    // at most, in the backward: partial sums of dw
constexpr int64_t kNormMaxWgs = ((int64_t(1) << 32) - 1) / kNormThreads;  // a launch takes fewer than 2^32 threads

struct NormArgs {
    const void *q, *k;
    int64_t ldq, ldk;
    const int64_t* pos;
    const int32_t* axis;    // [rot]: which of a token's `axes` positions turns a pair, or null (one position)
    int axes;
    const void *dqo, *dko;  // backward: upstream gradients
    void *qo, *ko;          // outputs (forward), dq and dk (backward), dense
    const float *wq, *wk, *freq;
    float* part;            // backward: [workgroups][2][dim] or null
    int64_t tokens;
    int hq, hk, dim, rot, per;  // per: heads a group takes
    float eps, inv_n;           // inv_n: 1 / dim (rms) or 1 (l2)
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4n __attribute__((ext_vector_type(4)));

// eight elements of a head: quads a and b (neighbours unless HALVES); ST: as accesses of a stream (stream.hpp)
template <bool BF, bool HALVES, bool ST>
struct Eight {
    u32x4 r[BF ? 1 : 2];
    __device__ __forceinline__ void load(const void* base, int a, int b, bool ok) {
        if (!ok) {
            r[0] = u32x4{};
            if constexpr (!BF) r[1] = u32x4{};
            return;
        }
        if constexpr (BF) {
            const uint16_t* p = (const uint16_t*)base;
            if constexpr (HALVES) {
                const u32x2 x = load_once<ST>((const u32x2*)(p + 4 * a)), y = load_once<ST>((const u32x2*)(p + 4 * b));
                r[0] = u32x4{x[0], x[1], y[0], y[1]};
            } else {
                r[0] = load_once<ST>((const u32x4*)(p + 4 * a));
            }
        } else {
            r[0] = load_once<ST>((const u32x4*)((const float*)base + 4 * a));
            r[1] = load_once<ST>((const u32x4*)((const float*)base + 4 * b));
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(r[0][i] << 16);
                x[2 * i + 1] = __uint_as_float(r[0][i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i >> 2][i & 3]);
        }
    }
    static __device__ __forceinline__ void store(void* base, int a, int b, const float (&x)[8]) {
        if constexpr (BF) {
            typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
            bf16x8 h;
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = (__bf16)x[i];
            const u32x4 w = __builtin_bit_cast(u32x4, h);
            uint16_t* p = (uint16_t*)base;
            if constexpr (HALVES) {
                store_once<ST>(u32x2{w[0], w[1]}, (u32x2*)(p + 4 * a));
                store_once<ST>(u32x2{w[2], w[3]}, (u32x2*)(p + 4 * b));
            } else {
                store_once<ST>(w, (u32x4*)(p + 4 * a));
            }
        } else {
            store_once<ST>(f32x4n{x[0], x[1], x[2], x[3]}, (f32x4n*)((float*)base + 4 * a));
            store_once<ST>(f32x4n{x[4], x[5], x[6], x[7]}, (f32x4n*)((float*)base + 4 * b));
        }
    }
};

// pair p of a lane: elements p, p + 4 (halves) or 2p, 2p + 1 (neighbours)
template <bool HALVES, bool BACK>
__device__ __forceinline__ void turn(float (&x)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int i = HALVES ? p : 2 * p, j = HALVES ? p + 4 : 2 * p + 1;
        const float a = x[i], b = x[j], sn = BACK ? -s[p] : s[p];
        x[i] = a * c[p] - b * sn;
        x[j] = a * sn + b * c[p];
    }
}

// AXES: a position for each of several axes. One position keeps code of its own: with a choice a token the calls of 5 to
// 16384 tokens of 12 heads of 128 were 1 to 5% slower, 8192 tokens of 5 fp32 heads of 256 19.8 us in place of 17.4.
template <bool BF, int G, bool HALVES, bool BACK, int AHEAD, bool ST, bool AXES>
__global__ __launch_bounds__(kNormThreads) void k_qk_norm(NormArgs a) {
    constexpr int GW = kNormThreads / G;  // groups per workgroup
    using E8 = Eight<BF, HALVES, ST>;
    constexpr int64_t E = BF ? 2 : 4;
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int quads = a.dim / 4, rq = a.rot / 4;
    const bool lok = 8 * lane < a.dim, turns = lane < rq;
    int qa = 2 * lane, qb = 2 * lane + 1;
    if (HALVES) {
        qa = turns ? lane : 2 * rq + 2 * (lane - rq);
        qb = turns ? rq + lane : qa + 1;
    }
    if (!lok || qb >= quads) qa = qb = 0;
    float w[2][8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const float* wp = t ? a.wk : a.wq;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[t][i] = wp ? wp[4 * (i < 4 ? qa : qb) + (i & 3)] : 1.f;
    }
    float fr[4] = {};
    int ax[AXES ? 4 : 1] = {};
    if (turns)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            fr[p] = a.freq[4 * lane + p];
            if constexpr (AXES) {
                const int i = a.axis[4 * lane + p];
                ax[p] = i < 0 ? 0 : i < a.axes ? i : a.axes - 1;
            }
        }
    float dw[2][8] = {};
    const int heads = a.hq + a.hk;
    const int h0 = blockIdx.y * a.per, h1 = h0 + a.per < heads ? h0 + a.per : heads;
    for (int64_t t0 = (int64_t)blockIdx.x * GW; t0 < a.tokens; t0 += (int64_t)gridDim.x * GW) {
        const int64_t t = t0 + grp;
        const bool tok = t < a.tokens, ok = tok && lok;
        auto src = [&](int h, const void* q, const void* k, int64_t ldq, int64_t ldk) {
            return h < a.hq ? (const char*)q + (t * ldq + (int64_t)h * a.dim) * E
                            : (const char*)k + (t * ldk + (int64_t)(h - a.hq) * a.dim) * E;
        };
        const int64_t dq = (int64_t)a.hq * a.dim, dk = (int64_t)a.hk * a.dim;  // dense row lengths
        E8 x[AHEAD], y[BACK ? AHEAD : 1];
        auto fetch = [&](int h) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const bool in = ok && h + i < h1;
                x[i].load(src(h + i, a.q, a.k, a.ldq, a.ldk), qa, qb, in);
                if constexpr (BACK) y[i].load(src(h + i, a.dqo, a.dko, dq, dk), qa, qb, in);
            }
        };
        fetch(h0);
        float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {};
        if (turns && tok) {
            double pos[AXES ? 4 : 1];
            if constexpr (AXES) {
#pragma unroll
                for (int p = 0; p < 4; ++p) pos[p] = (double)a.pos[t * a.axes + ax[p]];
            } else {
                pos[0] = (double)a.pos[t];
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const double u = pos[AXES ? p : 0] * (double)fr[p] * 0.15915494309189533577;  // turns
                sincospif((float)(2.0 * (u - rint(u))), &s[p], &c[p]);
            }
        }
        for (int h = h0; h < h1; h += AHEAD) {
            float v[AHEAD][8], e[BACK ? AHEAD : 1][8];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                x[i].get(v[i]);
                if constexpr (BACK) y[i].get(e[i]);
            }
            if (h + AHEAD < h1) fetch(h + AHEAD);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int hi = h + i;
                const int kind = hi < a.hq ? 0 : 1;
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
#pragma unroll
                for (int d = 1; d < G; d <<= 1) ss += __shfl_xor(ss, d);
                const float inv = 1.f / sqrtf(fmaf(ss, a.inv_n, a.eps));
                float o[8];
                if constexpr (!BACK) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = v[i][j] * inv * (kind ? w[1][j] : w[0][j]);
                    if (turns) turn<HALVES, false>(o, c, s);
                } else {
                    if (turns) turn<HALVES, true>(e[i], c, s);
                    float along = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float n = v[i][j] * inv, g = e[i][j] * n;
                        // heads past the end were read as zeros
                        dw[0][j] += kind ? 0.f : g;
                        dw[1][j] += kind ? g : 0.f;
                        e[i][j] *= kind ? w[1][j] : w[0][j];
                        along = fmaf(e[i][j], n, along);
                    }
#pragma unroll
                    for (int d = 1; d < G; d <<= 1) along += __shfl_xor(along, d);
                    along *= a.inv_n;
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = inv * (e[i][j] - v[i][j] * inv * along);
                }
                if (ok && hi < h1)
                    E8::store((void*)src(hi, a.qo, a.ko, dq, dk), qa, qb, o);
            }
        }
    }
    if constexpr (BACK)
        if (a.part) {
            __shared__ float red[2][GW][8 * G];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (lok) red[t][grp][4 * (i < 4 ? qa : qb) + (i & 3)] = dw[t][i];
            __syncthreads();
            float* out = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.dim;
            for (int e = threadIdx.x; e < 2 * a.dim; e += kNormThreads) {
                const int t = e / a.dim, d = e % a.dim;
                float sum = 0.f;
                for (int i = 0; i < GW; ++i) sum += red[t][i][d];
                out[e] = sum;
            }
        }
}

// sums of the workgroups' partial gradients: 32 columns x 32 rows of threads, each row's
// partials four at a time (with 8 rows one at a time, 1024 partials took 32 us)
__global__ __launch_bounds__(1024) void k_qk_norm_dw(const float* part, int64_t n, int dim, float* dwq, float* dwk) {
    __shared__ double red[32][33];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + c;
    double s = 0;
    if (e < 2 * dim) {
        int64_t i = r;
        for (; i + 96 < n; i += 128) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = part[(i + 32 * j) * 2 * dim + e];
            s += ((double)x[0] + x[1]) + ((double)x[2] + x[3]);
        }
        for (; i < n; i += 32) s += (double)part[i * 2 * dim + e];
    }
    red[r][c] = s;
    __syncthreads();
    for (int d = 16; d > 0; d >>= 1) {
        if (r < d) red[r][c] += red[r + d][c];
        __syncthreads();
    }
    if (r == 0 && e < 2 * dim) {
        float* o = e < dim ? dwq : dwk;
        if (o) o[e % dim] = (float)red[0][c];
    }
}

int group_lanes(int64_t dim) {
    int g = 1;
    while (8 * g < dim) g <<= 1;
    return g;
}

struct NormGrid {
    unsigned x, y;
    int per;
};
NormGrid norm_grid(const hyena_qk_norm_params_t& p, int64_t tokens, bool back) {
    const int64_t heads = p.heads_q + p.heads_k, gw = kNormThreads / group_lanes(p.dim);
    const int64_t wgs = (tokens + gw - 1) / gw;  // with every head of a token in one group
    // a group takes several heads (and the angles once for them) when that leaves enough waves
    int64_t per = wgs * (kNormThreads / 64) * heads / kNormWaves;
    per = per < 1 ? 1 : (per > heads ? heads : per);
    NormGrid g;
    g.per = (int)per;
    g.y = (unsigned)((heads + per - 1) / per);
    int64_t x = wgs < 1 ? 1 : wgs;
    if (back) {
        const int64_t most = kNormBackWgs / g.y < 1 ? 1 : kNormBackWgs / g.y;
        x = x > most ? most : x;
    }
    g.x = (unsigned)(x < kNormMaxWgs ? x : kNormMaxWgs);  // a workgroup walks over the tokens beyond
    return g;
}

// No fewer workgroups than the backward of so many tokens or fewer has: with more tokens a group takes more heads, so
// their number falls now and then.
int64_t norm_covering_wgs(const hyena_qk_norm_params_t& p, int64_t tokens) {
    const int64_t heads = p.heads_q + p.heads_k, gw = kNormThreads / group_lanes(p.dim);
    const int64_t all = (tokens + gw - 1) / gw * heads, most = heads > kNormBackWgs ? heads : kNormBackWgs;
    return all < most ? all : most;
}
size_t norm_part_bytes(int64_t wgs, int64_t dim) { return (size_t)wgs * 2 * (size_t)dim * sizeof(float); }

// Whether a call's accesses are marked as a stream's (stream.hpp): it moves more than the Infinity Cache holds, and
// what the lanes of a head reach with one instruction, `run` bytes behind each other, is whole lines. Of neighbours in
// fp32 an instruction reaches 16 bytes of every 32, of halves with a rest that is not rotated as well.
template <bool BF, bool HALVES, bool BACK>
bool norm_streams(const NormArgs& a) {
    constexpr int64_t E = BF ? 2 : 4;
    if (a.tokens * (a.hq + a.hk) * a.dim * E * (BACK ? 3 : 2) <= kInfinityCache) return false;
    const int64_t run = HALVES ? (2 * a.rot == a.dim ? a.rot * E : 0) : BF ? a.dim * E : 0;
    if (!run || (run | a.ldq * E | a.ldk * E) % kLine) return false;
    return whole_lines(a.q) && whole_lines(a.k) && whole_lines(a.qo) && whole_lines(a.ko) &&
           (!BACK || (whole_lines(a.dqo) && whole_lines(a.dko)));
}

template <bool BF, int G, bool HALVES, bool BACK, bool AXES>
void launch_norm_g(const NormArgs& a, const NormGrid& g, hipStream_t st) {
    const dim3 grid(g.x, g.y), block(kNormThreads);
    if constexpr (8 * G * (BF ? 2 : 4) / (HALVES ? 2 : 1) >= kLine && (BF || HALVES))  // heads of G lanes fill lines
        if (g.per > 1 && norm_streams<BF, HALVES, BACK>(a)) {
            hipLaunchKernelGGL((k_qk_norm<BF, G, HALVES, BACK, kNormAhead, true, AXES>), grid, block, 0, st, a);
            return;
        }
    if (g.per > 1)
        hipLaunchKernelGGL((k_qk_norm<BF, G, HALVES, BACK, kNormAhead, false, AXES>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((k_qk_norm<BF, G, HALVES, BACK, 1, false, AXES>), grid, block, 0, st, a);
}

template <bool BF, bool HALVES, bool BACK, bool AXES>
hipError_t launch_norm_t(const NormArgs& a, const NormGrid& g, hipStream_t st) {
    switch (group_lanes(a.dim)) {
        case 1: launch_norm_g<BF, 1, HALVES, BACK, AXES>(a, g, st); break;
        case 2: launch_norm_g<BF, 2, HALVES, BACK, AXES>(a, g, st); break;
        case 4: launch_norm_g<BF, 4, HALVES, BACK, AXES>(a, g, st); break;
        case 8: launch_norm_g<BF, 8, HALVES, BACK, AXES>(a, g, st); break;
        case 16: launch_norm_g<BF, 16, HALVES, BACK, AXES>(a, g, st); break;
        default: launch_norm_g<BF, 32, HALVES, BACK, AXES>(a, g, st); break;
    }
    return hipGetLastError();
}

template <bool BACK, bool AXES>
hipError_t launch_norm_a(bool bf, bool halves, const NormArgs& a, const NormGrid& g, hipStream_t st) {
    if (bf) return halves ? launch_norm_t<true, true, BACK, AXES>(a, g, st) : launch_norm_t<true, false, BACK, AXES>(a, g, st);
    return halves ? launch_norm_t<false, true, BACK, AXES>(a, g, st) : launch_norm_t<false, false, BACK, AXES>(a, g, st);
}
template <bool BACK>
hipError_t launch_norm(bool bf, bool halves, const NormArgs& a, const NormGrid& g, hipStream_t st) {
    return a.axis ? launch_norm_a<BACK, true>(bf, halves, a, g, st) : launch_norm_a<BACK, false>(bf, halves, a, g, st);
}

hyena_status_t norm_check_params(const hyena_qk_norm_params_t* p, int64_t tokens) {
    if (!p || p->heads_q < 1 || p->heads_k < 1 || p->dim < 1 || p->rot < 0 || tokens < 0) return HYENA_ERR_INVALID_ARG;
    if (p->dtype != HYENA_F32 && p->dtype != HYENA_BF16) return HYENA_ERR_INVALID_ARG;
    if (p->kind != HYENA_NORM_RMS && p->kind != HYENA_NORM_L2) return HYENA_ERR_INVALID_ARG;
    if (p->layout != HYENA_ROT_HALVES && p->layout != HYENA_ROT_PAIRS) return HYENA_ERR_INVALID_ARG;
    if (!(p->eps > 0.f && p->eps <= 3.402823466e38f) || 2 * p->rot > p->dim) return HYENA_ERR_INVALID_ARG;
    if (((uintptr_t)p->w_q | (uintptr_t)p->w_k | (uintptr_t)p->freq) & 3u) return HYENA_ERR_INVALID_ARG;
    if (p->rot > 0 && !p->freq) return HYENA_ERR_INVALID_ARG;
    if (p->dim % 8 || p->dim > 256 || p->rot % 4 || p->heads_q > 65535 || p->heads_q + p->heads_k > 65535 ||
        tokens > (int64_t(1) << 31))
        return HYENA_ERR_UNSUPPORTED;
    return HYENA_OK;
}

hyena_status_t norm_check(const hyena_qk_norm_params_t* p, int64_t tokens, const void* q, int64_t ldq, const void* k,
                          int64_t ldk, const int64_t* positions, NormArgs& a) {
    const hyena_status_t st = norm_check_params(p, tokens);
    if (st != HYENA_OK) return st;
    const int64_t v = p->dtype == HYENA_BF16 ? 8 : 4;
    if (ldq < p->heads_q * p->dim || ldk < p->heads_k * p->dim || ldq % v || ldk % v || ldq > (int64_t(1) << 31) ||
        ldk > (int64_t(1) << 31))
        return HYENA_ERR_INVALID_ARG;
    if (tokens > 0 && (!q || !k || !aligned16(q) || !aligned16(k) || (p->rot > 0 && !positions)))
        return HYENA_ERR_INVALID_ARG;
    if ((uintptr_t)positions & 7u) return HYENA_ERR_INVALID_ARG;
    a = NormArgs{};
    a.q = q;
    a.k = k;
    a.ldq = ldq;
    a.ldk = ldk;
    a.pos = positions;
    a.wq = p->w_q;
    a.wk = p->w_k;
    a.freq = p->freq;
    a.tokens = tokens;
    a.hq = (int)p->heads_q;
    a.hk = (int)p->heads_k;
    a.dim = (int)p->dim;
    a.rot = (int)p->rot;
    a.eps = p->eps;
    a.inv_n = p->kind == HYENA_NORM_RMS ? 1.f / (float)p->dim : 1.f;
    return HYENA_OK;
}

// the forward of both entry points (axis null: one position a token)
hyena_status_t norm_forward(const hyena_qk_norm_params_t* params, const int32_t* axis, int64_t axes, int64_t tokens,
                            const void* q, int64_t ldq, const void* k, int64_t ldk, const int64_t* positions,
                            void* q_out, void* k_out, hipStream_t stream) {
    NormArgs a;
    const hyena_status_t st = norm_check(params, tokens, q, ldq, k, ldk, positions, a);
    if (st != HYENA_OK) return st;
    if (tokens > 0 && (!q_out || !k_out)) return HYENA_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(k_out)) return HYENA_ERR_INVALID_ARG;
    if (tokens == 0) return HYENA_OK;
    a.axis = axis;
    a.axes = (int)axes;
    a.qo = q_out;
    a.ko = k_out;
    const NormGrid g = norm_grid(*params, tokens, false);
    a.per = g.per;
    const bool halves = params->layout == HYENA_ROT_HALVES && params->rot > 0;
    const hipError_t e = launch_norm<false>(params->dtype == HYENA_BF16, halves, a, g, stream);
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

hyena_status_t norm_backward(const hyena_qk_norm_params_t* params, const int32_t* axis, int64_t axes, int64_t tokens,
                             const void* q, int64_t ldq, const void* k, int64_t ldk, const int64_t* positions,
                             const void* dq_out, const void* dk_out, void* dq, void* dk, float* dw_q, float* dw_k,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
    NormArgs a;
    const hyena_status_t st = norm_check(params, tokens, q, ldq, k, ldk, positions, a);
    if (st != HYENA_OK) return st;
    const void* rows[] = {dq_out, dk_out, dq, dk};
    for (const void* p : rows)
        if ((tokens > 0 && !p) || !aligned16(p)) return HYENA_ERR_INVALID_ARG;
    if (((uintptr_t)dw_q | (uintptr_t)dw_k) & 3u) return HYENA_ERR_INVALID_ARG;
    const bool sums = dw_q || dw_k;
    const NormGrid g = norm_grid(*params, tokens, true);
    const size_t need = sums && tokens > 0 ? norm_part_bytes((int64_t)g.x * g.y, params->dim) : 0;
    if (need && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    if (need && !aligned16(workspace)) return HYENA_ERR_INVALID_ARG;
    hipError_t e = hipSuccess;
    if (tokens > 0) {
        a.axis = axis;
        a.axes = (int)axes;
        a.dqo = dq_out;
        a.dko = dk_out;
        a.qo = dq;
        a.ko = dk;
        a.part = sums ? (float*)workspace : nullptr;
        a.per = g.per;
        const bool halves = params->layout == HYENA_ROT_HALVES && params->rot > 0;
        e = launch_norm<true>(params->dtype == HYENA_BF16, halves, a, g, stream);
    }
    if (e == hipSuccess && sums) {  // without tokens: zeros
        const int64_t n = tokens > 0 ? (int64_t)g.x * g.y : 0;
        hipLaunchKernelGGL(k_qk_norm_dw, dim3((unsigned)((2 * params->dim + 31) / 32)), dim3(1024), 0, stream,
                           (const float*)workspace, n, (int)params->dim, dw_q, dw_k);
        e = hipGetLastError();
    }
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

// what the entry points with several axes check in front of the rest
hyena_status_t axes_check(const hyena_qk_norm_params_t* p, const int32_t* axis, int64_t axes) {
    if (!p || axes < 1 || ((uintptr_t)axis & 3u) || (p->rot > 0 && !axis)) return HYENA_ERR_INVALID_ARG;
    return axes > 8 ? HYENA_ERR_UNSUPPORTED : HYENA_OK;
}

}  // namespace
}  // namespace hy

extern "C" {

hyena_status_t hyena_qk_norm_forward(const hyena_qk_norm_params_t* params, int64_t tokens, const void* q, int64_t ldq,
                                     const void* k, int64_t ldk, const int64_t* positions, void* q_out, void* k_out,
                                     hipStream_t stream) {
    return hy::norm_forward(params, nullptr, 1, tokens, q, ldq, k, ldk, positions, q_out, k_out, stream);
}

hyena_status_t hyena_qk_norm_axes_forward(const hyena_qk_norm_params_t* params, const int32_t* axis, int64_t axes,
                                          int64_t tokens, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                          const int64_t* positions, void* q_out, void* k_out, hipStream_t stream) {
    const hyena_status_t st = hy::axes_check(params, axis, axes);
    if (st != HYENA_OK) return st;
    return hy::norm_forward(params, axis, axes, tokens, q, ldq, k, ldk, positions, q_out, k_out, stream);
}

size_t hyena_qk_norm_backward_workspace_bytes(const hyena_qk_norm_params_t* params, int64_t tokens) {
    if (hy::norm_check_params(params, tokens) != HYENA_OK || tokens == 0) return 0;
    return hy::norm_part_bytes(hy::norm_covering_wgs(*params, tokens), params->dim);
}

hyena_status_t hyena_qk_norm_backward(const hyena_qk_norm_params_t* params, int64_t tokens, const void* q, int64_t ldq,
                                      const void* k, int64_t ldk, const int64_t* positions, const void* dq_out,
                                      const void* dk_out, void* dq, void* dk, float* dw_q, float* dw_k, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
    return hy::norm_backward(params, nullptr, 1, tokens, q, ldq, k, ldk, positions, dq_out, dk_out, dq, dk, dw_q, dw_k,
                             workspace, workspace_bytes, stream);
}

hyena_status_t hyena_qk_norm_axes_backward(const hyena_qk_norm_params_t* params, const int32_t* axis, int64_t axes,
                                           int64_t tokens, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                           const int64_t* positions, const void* dq_out, const void* dk_out, void* dq,
                                           void* dk, float* dw_q, float* dw_k, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
    const hyena_status_t st = hy::axes_check(params, axis, axes);
    if (st != HYENA_OK) return st;
    return hy::norm_backward(params, axis, axes, tokens, q, ldq, k, ldk, positions, dq_out, dk_out, dq, dk, dw_q, dw_k,
                             workspace, workspace_bytes, stream);
}

}  // extern "C"
