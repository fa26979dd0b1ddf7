// Root-mean-square norm with the residual's addition in the same pass, its output
// optionally in 8 bits, and its backward. For a token's row x [dim]:
//   s = residual + x,   y = s inv w,   inv = 1 / sqrt(mean(s^2) + eps);
// s is normed as the fp32 sum and rounded when it is stored. In 8 bits (e4m3) a row, or
// each block of 128 columns of it, is divided by its scale, the largest |y| / 448.
// Backward, from the stored s and the gradients dy and ds_out of both outputs:
//   ds = inv w dy - s inv^3 mean(w dy s) + ds_out,   dw = sum over rows of dy s inv.
//
// Every value is read and written once: bound by memory. A row belongs to R threads (a
// wave up to 1024 columns, 256 threads up to 8192, then 512) and stays in their registers between the
// sum and the result: K pieces of 4 neighbours a thread, piece k of thread t at columns
// 4 (k R + t). So 128 columns are 32 lanes of one wave and a block's largest value needs
// no LDS. Threads walk over rows; the weights are loaded once. 65536 x 768 in bf16 take 70 us (5.7 TB/s), 16384 x
// 2048 to 8 bits from an fp32 residual 65 (5.7; a wave a row, 32 values a lane: 82), the backward of
// 65536 x 768 with the residual in fp32 135 (5.9).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hyena.h"
#include "plan.hpp"
#include "stream.hpp"

namespace hy {
namespace {

constexpr int64_t kRmsMaxDim = 16384;
constexpr float kE4m3Most = 448.f;

struct RmsArgs {
    const void *x, *res;
    int64_t ldx, ldres;
    const float* w;
    void *y, *sum;
    float* scales;
    const void *dy, *ds;  // backward: upstream gradients (res is s)
    void *dx, *dres;
    float* part;          // backward: [workgroups][dim] or null
    int64_t rows;
    int dim, block, nscales;
    float eps, inv_n;
};

typedef uint32_t u32x2r __attribute__((ext_vector_type(2)));
typedef float f32x4r __attribute__((ext_vector_type(4)));

// four neighbours of a row; ST: as accesses of a stream (stream.hpp)
template <bool BF, bool ST>
struct Four;
template <bool ST>
struct Four<true, ST> {
    u32x2r r;
    __device__ __forceinline__ void load(const void* row, int e) { r = load_once<ST>((const u32x2r*)((const uint16_t*)row + e)); }
    __device__ __forceinline__ void get(float (&x)[4]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[2 * i] = __uint_as_float(r[i] << 16);
            x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(void* row, int e, const float (&x)[4]) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        store_once<ST>(bf16x4{(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]}, (bf16x4*)((uint16_t*)row + e));
    }
};
template <bool ST>
struct Four<false, ST> {
    f32x4r r;
    __device__ __forceinline__ void load(const void* row, int e) { r = load_once<ST>((const f32x4r*)((const float*)row + e)); }
    __device__ __forceinline__ void get(float (&x)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = r[i];
    }
    static __device__ __forceinline__ void store(void* row, int e, const float (&x)[4]) {
        store_once<ST>(f32x4r{x[0], x[1], x[2], x[3]}, (f32x4r*)((float*)row + e));
    }
};

// N sums (or maxima) over the R threads of a row; every thread gets them
template <int R, int N, bool MAX>
__device__ __forceinline__ void row_reduce(float (&v)[N], float* lds) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float o = __shfl_xor(v[n], d);
            v[n] = MAX ? fmaxf(v[n], o) : v[n] + o;
        }
    if constexpr (R > 64) {
        constexpr int W = R / 64;
        const int wave = threadIdx.x >> 6;
        __syncthreads();  // the row before has been read
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) lds[wave * N + n] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float t = lds[n];
            for (int w = 1; w < W; ++w) t = MAX ? fmaxf(t, lds[w * N + n]) : t + lds[w * N + n];
            v[n] = t;
        }
    }
}

// a / b, from r = 1 / b rounded to nearest: the quotient's error is found exactly and taken off, so what lies
// halfway between two 8-bit values is met as in a division, at 4 operations in place of some 10 (16384 x 2048
// to 8 bits 64.7 us, with the product alone 64.5; 8192 x 8192 96.1 and 94.7)
__device__ __forceinline__ float quotient(float a, float b, float r) {
    const float q = a * r;
    return copysignf(fmaf(fmaf(-q, b, a), r, q), a);
}

// XB, SB: x and y, the residual and the sum are bf16 (otherwise fp32); Q: output in 8 bits
template <bool XB, bool SB, bool Q, bool ST, int R, int K>
__global__ __launch_bounds__(R < 256 ? 256 : R) void k_residual_norm(RmsArgs p) {
    constexpr int kPer = R < 256 ? 256 / R : 1;  // rows a workgroup
    constexpr int XE = XB ? 2 : 4, SE = SB ? 2 : 4;
    __shared__ float lds[R > 64 ? 2 * (R / 64) : 1];
    const int t = threadIdx.x % R;
    float w[K][4];
    int col[K];
    bool ok[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 4 * (k * R + t);
        ok[k] = c < p.dim;
        col[k] = ok[k] ? c : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[k][i] = p.w ? p.w[col[k] + i] : 1.f;
    }
    const int64_t step = (int64_t)gridDim.x * kPer;
    Four<XB, ST> x[K];
    Four<SB, ST> r[K];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k].load((const char*)p.x + row * p.ldx * XE, col[k]);
            if (p.res) r[k].load((const char*)p.res + row * p.ldres * SE, col[k]);
        }
    };
    // every thread of a workgroup takes the same number of rounds
    for (int64_t r0 = (int64_t)blockIdx.x * kPer; r0 < p.rows; r0 += step) {
        const int64_t mine = r0 + threadIdx.x / R;
        const bool in = mine < p.rows;
        const int64_t row = in ? mine : p.rows - 1;
        fetch(row);
        float s[K][4], ss[1] = {};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k].get(s[k]);
            if (p.res) {
                float o[4];
                r[k].get(o);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[k][i] += o[i];
            }
            if (p.sum && in && ok[k]) Four<SB, ST>::store((char*)p.sum + row * p.dim * SE, col[k], s[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) ss[0] = ok[k] ? fmaf(s[k][i], s[k][i], ss[0]) : ss[0];
        }
        row_reduce<R, 1, false>(ss, lds);
        const float inv = 1.f / sqrtf(fmaf(ss[0], p.inv_n, p.eps));
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[k][i] = s[k][i] * inv * w[k][i];
        if constexpr (!Q) {
            if (in)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (ok[k]) Four<XB, ST>::store((char*)p.y + row * p.dim * XE, col[k], s[k]);
        } else {
            float most[K];
#pragma unroll
            for (int k = 0; k < K; ++k)
                most[k] = ok[k] ? fmaxf(fmaxf(fabsf(s[k][0]), fabsf(s[k][1])), fmaxf(fabsf(s[k][2]), fabsf(s[k][3]))) : 0.f;
            if (p.block) {
#pragma unroll
                for (int d = 1; d < 32; d <<= 1)
#pragma unroll
                    for (int k = 0; k < K; ++k) most[k] = fmaxf(most[k], __shfl_xor(most[k], d));
            } else {
                float all[1] = {most[0]};
#pragma unroll
                for (int k = 1; k < K; ++k) all[0] = fmaxf(all[0], most[k]);
                row_reduce<R, 1, true>(all, lds + (R > 64 ? R / 64 : 0));
#pragma unroll
                for (int k = 0; k < K; ++k) most[k] = all[0];
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                // not below 2^-126, so that its inverse is finite
                const float scale = most[k] > 0.f ? fmaxf(most[k] / kE4m3Most, 1.17549435e-38f) : 1.f;
                const float by = 1.f / scale;
                if (in && ok[k]) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = quotient(s[k][i], scale, by);
                    int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
                    q = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], q, true);
                    store_once<ST>(q, (int*)((char*)p.y + row * p.dim + col[k]));
                    if (p.block ? (t & 31) == 0 : k == 0 && t == 0)
                        p.scales[row * p.nscales + (p.block ? col[k] / 128 : 0)] = scale;
                }
            }
        }
    }
}

template <bool XB, bool SB, bool ST, int R, int K>
__global__ __launch_bounds__(R < 256 ? 256 : R) void k_residual_norm_back(RmsArgs p) {
    constexpr int kPer = R < 256 ? 256 / R : 1;
    constexpr int XE = XB ? 2 : 4, SE = SB ? 2 : 4;
    __shared__ float lds[R > 64 ? 2 * (R / 64) : 1];
    const int t = threadIdx.x % R;
    float w[K][4], dw[K][4] = {};
    int col[K];
    bool ok[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = 4 * (k * R + t);
        ok[k] = c < p.dim;
        col[k] = ok[k] ? c : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[k][i] = p.w ? p.w[col[k] + i] : 1.f;
    }
    const int64_t step = (int64_t)gridDim.x * kPer;
    for (int64_t r0 = (int64_t)blockIdx.x * kPer; r0 < p.rows; r0 += step) {
        const int64_t mine = r0 + threadIdx.x / R;
        const bool in = mine < p.rows;
        const int64_t row = in ? mine : p.rows - 1;
        Four<SB, ST> sr[K], dr[K];
        Four<XB, ST> yr[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            sr[k].load((const char*)p.res + row * p.ldres * SE, col[k]);
            yr[k].load((const char*)p.dy + row * p.dim * XE, col[k]);
            if (p.ds) dr[k].load((const char*)p.ds + row * p.dim * SE, col[k]);
        }
        float s[K][4], d[K][4], v[2] = {};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            sr[k].get(s[k]);
            yr[k].get(d[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[0] = ok[k] ? fmaf(s[k][i], s[k][i], v[0]) : v[0];
                v[1] = ok[k] ? fmaf(s[k][i], d[k][i] * w[k][i], v[1]) : v[1];
            }
        }
        row_reduce<R, 2, false>(v, lds);
        const float inv = 1.f / sqrtf(fmaf(v[0], p.inv_n, p.eps));
        const float along = v[1] * inv * p.inv_n * inv;  // mean(w dy s) inv^2
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float o[4], e[4] = {};
            if (p.ds) dr[k].get(e);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dw[k][i] += in ? d[k][i] * (s[k][i] * inv) : 0.f;
                o[i] = fmaf(inv, d[k][i] * w[k][i] - s[k][i] * along, e[i]);
            }
            if (in && ok[k]) {
                if (p.dx) Four<XB, ST>::store((char*)p.dx + row * p.dim * XE, col[k], o);
                if (p.dres) Four<SB, ST>::store((char*)p.dres + row * p.dim * SE, col[k], o);
            }
        }
    }
    if (p.part) {
        float* out = p.part + (int64_t)blockIdx.x * p.dim;
        if constexpr (R >= 256) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (ok[k]) *(f32x4r*)(out + col[k]) = f32x4r{dw[k][0], dw[k][1], dw[k][2], dw[k][3]};
        } else {
            __shared__ f32x4r red[kPer][R * K];
#pragma unroll
            for (int k = 0; k < K; ++k)
                red[threadIdx.x / R][k * R + t] = f32x4r{dw[k][0], dw[k][1], dw[k][2], dw[k][3]};
            __syncthreads();
            for (int c = threadIdx.x; 4 * c < p.dim; c += 256) {
                f32x4r sum = red[0][c];
                for (int i = 1; i < kPer; ++i) sum += red[i][c];
                *(f32x4r*)(out + 4 * c) = sum;
            }
        }
    }
}

// sums of the workgroups' partial gradients: 32 columns x 32 rows of threads
__global__ __launch_bounds__(1024) void k_residual_norm_dw(const float* part, int64_t n, int dim, float* dw) {
    __shared__ double red[32][33];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5, e = blockIdx.x * 32 + c;
    double s = 0;
    if (e < dim) {
        int64_t i = r;
        for (; i + 96 < n; i += 128) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = part[(i + 32 * j) * dim + e];
            s += ((double)x[0] + x[1]) + ((double)x[2] + x[3]);
        }
        for (; i < n; i += 32) s += (double)part[i * dim + e];
    }
    red[r][c] = s;
    __syncthreads();
    for (int d = 16; d > 0; d >>= 1) {
        if (r < d) red[r][c] += red[r + d][c];
        __syncthreads();
    }
    if (r == 0 && e < dim) dw[e] = (float)red[0][c];
}

int64_t rms_rows(int64_t dim) { return dim <= 1024 ? 4 : 1; }  // rows a workgroup

// Workgroups of the forward: two rounds where there are enough rows, at most 8192 (65536 x 768: 2048, 4096, 8192
// and 16384 workgroups 81, 76, 73 and 81 us; 8192 x 4096: 47, 47, 52 and 52).
int64_t rms_forward_wgs(int64_t rows, int64_t dim) {
    const int64_t n = (rows + rms_rows(dim) - 1) / rms_rows(dim);
    return n <= 4096 ? n : n < 16384 ? (n + 1) / 2 : 8192;
}

// Workgroups of the backward, each with partial sums of dw. Two a CU read the longest runs that still
// hide the latency; rows of one piece need more (us, 256, 384, 512 and 768 of them: 65536 x 768 of bf16 100, 77, 70, 74,
// with the residual in fp32 135, 151, 140, 151; 16384 x 2048 118, 94, 93, 96; 65536 x 128 with 256, 512 and 1024 55,
// 32, 25). Sending for the next row early gains nothing on top.
int64_t rms_back_wgs(int64_t rows, int64_t dim) {
    const int64_t n = (rows + rms_rows(dim) - 1) / rms_rows(dim), most = dim <= 256 ? 1024 : 512;
    return n < most ? n : most;
}

// f.template go<R, K>() for the threads of a row and the pieces of one that dim needs
template <class F>
void by_dim(int dim, F f) {
    if (dim <= 256) f.template go<64, 1>();
    else if (dim <= 512) f.template go<64, 2>();
    else if (dim <= 768) f.template go<64, 3>();
    else if (dim <= 1024) f.template go<64, 4>();
    else if (dim <= 2048) f.template go<256, 2>();
    else if (dim <= 4096) f.template go<256, 4>();
    else if (dim <= 8192) f.template go<256, 8>();
    else f.template go<512, 8>();
}

template <bool XB, bool SB>
struct RmsForward {
    const RmsArgs& a;
    hipStream_t st;
    template <int R, int K>
    void go() const {
        const dim3 grid((unsigned)rms_forward_wgs(a.rows, a.dim)), block(R < 256 ? 256 : R);
        constexpr int XE = XB ? 2 : 4, SE = SB ? 2 : 4;
        const int64_t bytes = a.rows * a.dim * (XE + (a.res ? SE : 0) + (a.sum ? SE : 0) + (a.scales ? 1 : XE));
        // Up to 1024 bf16 columns only rows of whole lines (stream.hpp); 300 MiB, unmarked and marked: 264 columns 70.6
        // and 81.6 us, 520 65.6 and 72.4, 1000 63.3 and 65.5, 1544 67.2 and 67.8, 8200 76.7 and 74.8; in fp32 1000
        // columns 61.3 and 58.8. The backward is at most 4% slower so marked (40 columns 264 and 275), up to 8% faster.
        const bool stream = bytes > kInfinityCache && (!XB || a.dim > 1024 || a.dim % (kLine / XE) == 0);
        if (a.scales && stream)
            hipLaunchKernelGGL((k_residual_norm<XB, SB, true, true, R, K>), grid, block, 0, st, a);
        else if (a.scales)
            hipLaunchKernelGGL((k_residual_norm<XB, SB, true, false, R, K>), grid, block, 0, st, a);
        else if (stream)
            hipLaunchKernelGGL((k_residual_norm<XB, SB, false, true, R, K>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((k_residual_norm<XB, SB, false, false, R, K>), grid, block, 0, st, a);
    }
};
template <bool XB, bool SB>
struct RmsBackward {
    const RmsArgs& a;
    hipStream_t st;
    template <int R, int K>
    void go() const {
        const dim3 grid((unsigned)rms_back_wgs(a.rows, a.dim)), block(R < 256 ? 256 : R);
        constexpr int XE = XB ? 2 : 4, SE = SB ? 2 : 4;
        const int64_t bytes = a.rows * a.dim * (SE + XE + (a.ds ? SE : 0) + (a.dx ? XE : 0) + (a.dres ? SE : 0));
        if (bytes > kInfinityCache)
            hipLaunchKernelGGL((k_residual_norm_back<XB, SB, true, R, K>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((k_residual_norm_back<XB, SB, false, R, K>), grid, block, 0, st, a);
    }
};

template <template <bool, bool> class F>
hipError_t launch_rms(const hyena_residual_norm_params_t& p, const RmsArgs& a, hipStream_t st) {
    if (p.dtype == HYENA_F32) by_dim(a.dim, F<false, false>{a, st});
    else if (p.residual_dtype == HYENA_F32) by_dim(a.dim, F<true, false>{a, st});
    else by_dim(a.dim, F<true, true>{a, st});
    return hipGetLastError();
}

hyena_status_t rms_check(const hyena_residual_norm_params_t* p, int64_t rows) {
    if (!p || p->dim < 1 || rows < 0 || (p->block != 0 && p->block != 128)) return HYENA_ERR_INVALID_ARG;
    if (p->dtype != HYENA_F32 && p->dtype != HYENA_BF16) return HYENA_ERR_INVALID_ARG;
    if (p->residual_dtype != HYENA_F32 && p->residual_dtype != HYENA_BF16) return HYENA_ERR_INVALID_ARG;
    if (!(p->eps > 0.f && p->eps <= 3.402823466e38f) || ((uintptr_t)p->w & 3u)) return HYENA_ERR_INVALID_ARG;
    if (p->dtype == HYENA_F32 && p->residual_dtype == HYENA_BF16) return HYENA_ERR_UNSUPPORTED;
    if (p->dim % 8 || p->dim > kRmsMaxDim || rows > (int64_t(1) << 31)) return HYENA_ERR_UNSUPPORTED;
    return HYENA_OK;
}

RmsArgs rms_args(const hyena_residual_norm_params_t& p, int64_t rows) {
    RmsArgs a{};
    a.w = p.w;
    a.rows = rows;
    a.dim = (int)p.dim;
    a.block = (int)p.block;
    a.nscales = p.block ? (int)((p.dim + 127) / 128) : 1;
    a.eps = p.eps;
    a.inv_n = 1.f / (float)p.dim;
    return a;
}

bool rms_bad_ld(int64_t ld, int64_t dim, hyena_dtype_t t) {
    return ld < dim || ld % (t == HYENA_BF16 ? 8 : 4) || ld > (int64_t(1) << 31);
}

}  // namespace
}  // namespace hy

extern "C" {

hyena_status_t hyena_residual_norm_forward(const hyena_residual_norm_params_t* params, int64_t rows, const void* x,
                                           int64_t ldx, const void* residual, int64_t ldr, void* y, float* scales,
                                           void* sum, hipStream_t stream) {
    using hy::aligned16;
    const hyena_status_t st = hy::rms_check(params, rows);
    if (st != HYENA_OK) return st;
    if (rows > 0 && (!x || !y)) return HYENA_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(y) || !aligned16(sum) || ((uintptr_t)scales & 3u))
        return HYENA_ERR_INVALID_ARG;
    if (hy::rms_bad_ld(ldx, params->dim, params->dtype)) return HYENA_ERR_INVALID_ARG;
    if (residual && hy::rms_bad_ld(ldr, params->dim, params->residual_dtype)) return HYENA_ERR_INVALID_ARG;
    if (rows == 0) return HYENA_OK;
    hy::RmsArgs a = hy::rms_args(*params, rows);
    a.x = x;
    a.ldx = ldx;
    a.res = residual;
    a.ldres = ldr;
    a.y = y;
    a.scales = scales;
    a.sum = sum;
    return hy::launch_rms<hy::RmsForward>(*params, a, stream) == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

size_t hyena_residual_norm_backward_workspace_bytes(const hyena_residual_norm_params_t* params, int64_t rows) {
    if (hy::rms_check(params, rows) != HYENA_OK || rows == 0) return 0;
    return (size_t)hy::rms_back_wgs(rows, params->dim) * (size_t)params->dim * sizeof(float);
}

hyena_status_t hyena_residual_norm_backward(const hyena_residual_norm_params_t* params, int64_t rows, const void* s,
                                            int64_t lds, const void* dy, const void* dsum, void* dx, void* dresidual,
                                            float* dw, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    using hy::aligned16;
    const hyena_status_t st = hy::rms_check(params, rows);
    if (st != HYENA_OK) return st;
    if (rows > 0 && (!s || !dy || (!dx && !dresidual && !dw))) return HYENA_ERR_INVALID_ARG;
    const void* all[] = {s, dy, dsum, dx, dresidual};
    for (const void* q : all)
        if (!aligned16(q)) return HYENA_ERR_INVALID_ARG;
    if (((uintptr_t)dw & 3u) || hy::rms_bad_ld(lds, params->dim, params->residual_dtype)) return HYENA_ERR_INVALID_ARG;
    const size_t need = dw ? hyena_residual_norm_backward_workspace_bytes(params, rows) : 0;
    if (need && (!workspace || workspace_bytes < need)) return HYENA_ERR_WORKSPACE;
    if (need && !aligned16(workspace)) return HYENA_ERR_INVALID_ARG;
    hipError_t e = hipSuccess;
    if (rows > 0) {
        hy::RmsArgs a = hy::rms_args(*params, rows);
        a.res = s;
        a.ldres = lds;
        a.dy = dy;
        a.ds = dsum;
        a.dx = dx;
        a.dres = dresidual;
        a.part = dw ? (float*)workspace : nullptr;
        e = hy::launch_rms<hy::RmsBackward>(*params, a, stream);
    }
    if (e == hipSuccess && dw) {  // without rows: zeros
        const int64_t n = rows > 0 ? hy::rms_back_wgs(rows, params->dim) : 0;
        hipLaunchKernelGGL(hy::k_residual_norm_dw, dim3((unsigned)((params->dim + 31) / 32)), dim3(1024), 0, stream,
                           (const float*)workspace, n, (int)params->dim, dw);
        e = hipGetLastError();
    }
    return e == hipSuccess ? HYENA_OK : HYENA_ERR_DEVICE;
}

}  // extern "C"
