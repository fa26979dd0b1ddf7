/*
 * libhyena — the Hyena operator forward hot path, its backward, the whole
 * operator forward, the implicit filter generator, the HyenaND variants
 * (per-sample filters, circular plans, gated 2-D and 3-D long convolutions), and for
 * layers that mix Hyena with linear attention the gated delta rule and the gated linear
 * recurrence (whole sequences, their backward, single tokens against a pool of states), the
 * norm of queries and keys with position rotation and the residual norm in front of a
 * layer, on AMD MI355X (gfx950).
 *
 * The operator (HyenaDNA walkthrough, section 2.1, the Hyena operator module and
 * its forward pass; section 2.2, the long-filter module and its FFT convolution).
 * For each channel d < D and time t < L, with u the in-projected activation of
 * (N+1)*D channels:
 *   uc[c][t] = w[c][0] u[c][t-2] + w[c][1] u[c][t-1] + w[c][2] u[c][t],
 *              u[c][t'] = 0 for t' < 0 (a causal width-3 depthwise filter);
 *   x_i[d] = uc[i*D + d] for i < N (the gates), v_0[d] = uc[N*D + d] (the value);
 *   for o = 0 .. N-2 (the gates taken from x_{N-1} down to x_1):
 *       g_o     = v_o (.) x_{N-1-o}
 *       v_{o+1} = h[o] * g_o + bias[o] g_o
 *   y = v_{N-1} (.) x_0,
 * with (.) the elementwise product and * the causal per-channel long convolution
 *   (h * g)[t] = sum_{s <= t} h[s] g[t - s],
 * evaluated by FFT on the sequence zero-padded to 2L (the HyenaND summary's
 * boundary handling; the Hyena Hierarchy concept page, section 3.2, FFT
 * acceleration). hyena_operator_forward adds the module's in/out projections and
 * its (B, L, D) <-> (B, D, L) transposes around the path; dropout is the identity; the
 * short Conv1d bias is taken as zero.
 *
 * Conventions for every call:
 *  - Device pointers are plain device memory on the device that was current when
 *    the plan was created; that device must be current for every later call.
 *    The caller owns every buffer; libhyena never frees caller memory.
 *  - Tensors are dense and row-major (C order) with the shapes given below and
 *    16-byte aligned base pointers. Outputs must not alias inputs.
 *  - Calls that take a stream enqueue work on it and return without
 *    synchronising; results are ready when the stream reaches that point.
 *  - Errors are reported by return value; nothing throws across this ABI.
 *    Argument errors are detected on the host before any HIP call is made.
 *  - A plan is immutable after creation (apart from the GEMM state the operator
 *    entry points attach under a lock) and may be shared between host threads;
 *    concurrent calls need distinct workspaces and outputs.
 */
#ifndef LIBHYENA_HYENA_H
#define LIBHYENA_HYENA_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct hyena_plan_s* hyena_plan_t; /* opaque */

/* Element type of u_proj and y. All parameters (short_w, h, bias) and every
 * intermediate are fp32; bf16 outputs are rounded to nearest even. */
typedef enum { HYENA_F32 = 0, HYENA_BF16 = 1 } hyena_dtype_t;

typedef enum {
    HYENA_OK = 0,
    HYENA_ERR_INVALID_ARG = 1, /* NULL pointer, bad size or shape, misaligned pointer */
    HYENA_ERR_UNSUPPORTED = 2, /* valid request outside what the library implements */
    HYENA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required */
    HYENA_ERR_DEVICE = 4       /* no usable HIP device, allocation or launch failure */
} hyena_status_t;

/* Which kernel family runs a plan.
 *   LDS       one launch; the whole transform of a (b, d) row stays in LDS
 *             (L <= 16384).
 *   FOURSTEP  three passes per recurrence step (column FFTs, row FFTs with
 *             the spectrum multiply, inverse columns with the gate) over
 *             chunks of rows; any order, 256 <= L <= 2^20. At order 2 with
 *             L = 2^16 or 2^17 the chunks are pipelined: one launch runs the
 *             three passes on three consecutive chunks.
 *   PARTITIONED  the same causal convolution with the filter cut into
 *             blocks of Q = 4096 taps (uniformly partitioned overlap-save):
 *             two LDS-resident launches per recurrence step (transforms of
 *             2Q-sample windows of v; block-Toeplitz sums of window and
 *             filter-block spectra, inverse transforms and the gate), no
 *             transposed tile. Zero-padded plans with 8192 <= L <= 131072;
 *             hyena_backward does not take these plans.
 * AUTO picks LDS when L <= 16384 and FOURSTEP otherwise. */
typedef enum {
    HYENA_PATH_AUTO = 0,
    HYENA_PATH_LDS = 1,
    HYENA_PATH_FOURSTEP = 2,
    /* 3 is unused (HYENA_ERR_INVALID_ARG) */
    HYENA_PATH_PARTITIONED = 4
} hyena_path_t;

/* Create a plan for sequence length L, operator width D and recurrence order
 * N = `order` (N-1 long filters, N gates). Requirements: L a power of two in
 * [16, 2^20], D >= 1, 2 <= order <= 8, dtype one of hyena_dtype_t.
 * Builds the twiddle tables on the host in fp64 and uploads them to the current
 * device (the plan owns that memory; hyena_plan_destroy releases it).
 * Returns HYENA_ERR_INVALID_ARG / HYENA_ERR_UNSUPPORTED for bad arguments,
 * HYENA_ERR_DEVICE when no HIP device is usable. *out is set only on success. */
hyena_status_t hyena_plan_create(hyena_plan_t* out, int64_t L, int64_t D, int order, hyena_dtype_t dtype);

/* As hyena_plan_create, with an explicit kernel family. HYENA_PATH_LDS needs
 * L <= 16384; HYENA_PATH_FOURSTEP needs L >= 256; HYENA_PATH_PARTITIONED needs
 * 8192 <= L <= 131072 and no flags. The spectrum layout depends on the
 * path (PARTITIONED holds the 2Q-point spectra of
 * each filter's L/Q blocks, [o][d][block][Q], in the LDS layout), so a spectrum
 * must be made by a plan whose path uses the same layout as the plan that
 * consumes it. */
hyena_status_t hyena_plan_create_path(hyena_plan_t* out, int64_t L, int64_t D, int order, hyena_dtype_t dtype,
                                      hyena_path_t path);

/* Plan options (bit flags for hyena_plan_create_ex). */
enum {
    /* Circular long convolution (the HyenaND summary's boundary handling offers
     * circular convolution for periodic data besides zero padding to double the
     * grid):  conv(v, h)[t] = sum_{s < L} h[s] v[(t - s) mod L]. The L samples are
     * transformed as they are (an L-point real transform, no zero padding); the
     * short conv keeps its causal zero padding. Requires L >= 32; the LDS path
     * serves L <= 32768. hyena_backward takes circular plans on the LDS path. */
    HYENA_FLAG_CIRCULAR = 1
};

/* As hyena_plan_create_path, with option flags (0 or HYENA_FLAG_CIRCULAR).
 * HYENA_ERR_INVALID_ARG for unknown flag bits; HYENA_ERR_UNSUPPORTED for a
 * circular plan with L < 32 or on the partitioned path. */
hyena_status_t hyena_plan_create_ex(hyena_plan_t* out, int64_t L, int64_t D, int order, hyena_dtype_t dtype,
                                    hyena_path_t path, uint32_t flags);

/* Release a plan and its device tables. NULL is a no-op returning HYENA_OK.
 * The caller must ensure no enqueued work still uses the plan. */
hyena_status_t hyena_plan_destroy(hyena_plan_t plan);

/* The path a plan resolved to (HYENA_PATH_LDS, HYENA_PATH_FOURSTEP or
 * HYENA_PATH_PARTITIONED), or HYENA_PATH_AUTO for a NULL plan. */
hyena_path_t hyena_plan_path(hyena_plan_t plan);

/* Bytes of the opaque spectrum buffer: (N-1) * D * L complex fp32 values, i.e.
 * 8 * (N-1) * D * L (L/2 complex values per filter for a circular plan).
 * Returns 0 for a NULL plan. */
size_t hyena_spectrum_bytes(hyena_plan_t plan);

/* Workspace for a forward over batch B: 0 on the LDS path. On the four-step
 * path this is the recommended size, in tiles of 8*L bytes per (b, d) row held
 * in flight: at order 2 with L = 2^16 or 2^17, three tile slots of
 * min(B*D, 128) rows (the pipelined launches); otherwise up to 128 MiB of
 * tiles. Any workspace of at least 8*L bytes (one row) is accepted: a
 * pipelined forward needs three slots of min(B*D, 32) rows and otherwise runs
 * chunk by chunk, and a larger one lets more rows run per launch. The
 * partitioned path likewise, with 8*L bytes per row at order 2 and 12*L bytes
 * per row above (the gated output of a step is held for the next). The choice
 * of chunks never changes the result: every chunking gives the same bits.
 * Returns 0 for a NULL plan or B < 1. */
size_t hyena_workspace_bytes(hyena_plan_t plan, int64_t B);

/* The real FFT of the long filters, once per plan (the filter spectrum of the
 * causal convolution; HyenaDNA walkthrough section 2.2, fftconv).
 *   h    [N-1][D][L] fp32, device: filter o of channel d at h[(o*D + d)*L + t]
 *   spec device buffer of hyena_spectrum_bytes(plan) bytes, written in the
 *        plan's private layout (the 2L-point spectrum bins 0..L of each
 *        zero-padded filter, scaled by 2^-(log2 L + 2)).
 * Enqueued on `stream`. HYENA_ERR_INVALID_ARG for NULL pointers or misaligned
 * buffers; HYENA_ERR_DEVICE if the launch fails or the plan's device is not
 * current. */
hyena_status_t hyena_filter_spectrum(hyena_plan_t plan, const float* h, void* spec, hipStream_t stream);

/* Spectra of per-sample long filters, for input-dependent convolutions (the
 * HyenaND summary's methodology: kernels conditioned on each input sample, one
 * global FFT path). hyena_filter_spectrum for B filter sets at once:
 *   h    [B][N-1][D][L] fp32, device: the filters of sample b at h + b*(N-1)*D*L
 *   spec device buffer of B * hyena_spectrum_bytes(plan) bytes; sample b's
 *        spectrum starts at byte b * hyena_spectrum_bytes(plan).
 * Errors as hyena_filter_spectrum; HYENA_ERR_INVALID_ARG also for B < 1 or
 * B*(N-1)*D > 2^24. */
hyena_status_t hyena_filter_spectrum_batched(hyena_plan_t plan, int64_t B, const float* h, void* spec,
                                             hipStream_t stream);

/* The forward hot path for a batch of B sequences.
 *   u_proj  [B][(N+1)*D][L] of the plan dtype, device: channel i*D + d is gate
 *           x_i for i < N and channel N*D + d is the value v (the in-projected,
 *           rearranged activation)
 *   short_w [(N+1)*D][3] fp32, device: PyTorch Conv1d taps; uc[t] =
 *           w[0]*u[t-2] + w[1]*u[t-1] + w[2]*u[t] with u[t<0] = 0
 *   spec    from hyena_filter_spectrum of a plan with the same L, D, order, path
 *   bias    [N-1][D] fp32, device: the bias skip term of step o is bias[o][d]*v
 *   y       [B][D][L] of the plan dtype, device (output, before the transpose
 *           to [B][L][D])
 *   workspace / workspace_bytes: device scratch, at least 8*L bytes on the
 *           four-step path and 8*L (order 2) or 12*L bytes on the partitioned
 *           path (see hyena_workspace_bytes); ignored (may be NULL) on the LDS
 *           path. Contents on entry are irrelevant.
 * Enqueued on `stream`; no host synchronisation. Errors: HYENA_ERR_INVALID_ARG
 * (NULL/misaligned pointers, B < 1 or B*D*L too large), HYENA_ERR_WORKSPACE,
 * HYENA_ERR_DEVICE (launch failure, wrong current device). */
hyena_status_t hyena_forward(hyena_plan_t plan, int64_t B, const void* u_proj, const float* short_w,
                             const void* spec, const float* bias, void* y, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/* Parameters of the input-dependent kernel synthesis (HyenaND summary, method:
 * input-dependent kernels through registers and FiLM, kernel synthesis, kernel
 * parametrisation). With A = axes, W = width, M = layers, Z = zdim and
 * C = channels; all arrays fp32, row-major, device, 16-byte aligned:
 *   w_first  [W][A]      first layer, on the coordinates
 *   w_hidden [M-1][W][W] further layers (may be NULL when M = 1); row = output unit
 *   b_layer  [M][W]      layer biases
 *   omega    [M][W]      sine frequency of every hidden unit
 *   film_g [M][W][Z], film_gb [M][W]   FiLM scale  gamma_l = film_g[l] z + film_gb[l]
 *   film_b [M][W][Z], film_bb [M][W]   FiLM shift  beta_l  = film_b[l] z + film_bb[l]
 *   w_out [C][W], b_out [C]            affine output layer, one row per kernel
 *   win_mu [C][A], win_sigma [C][A]    Gaussian window of every kernel
 * Layer l maps h_l to h_{l+1} = sin(omega_l * (gamma_l * (W_l h_l + b_l) + beta_l))
 * with h_0 the coordinate c of a grid point; the kernel is
 *   K_k(c) = exp(-1/2 sum_i ((c_i - mu_ki) / sigma_ki)^2) * (w_out[k] . h_M + b_out[k]).
 * The grid has grid[i] points on axis i (axis 0 slowest; grid[i] for i >= axes is
 * ignored). Point j of a causal axis of n points sits at c = j / n; a signed axis
 * (bit i of signed_axes set) holds the wrapped offsets j (j < n/2) and j - n
 * (j >= n/2) at c = 2 * offset / n. 1-D Hyena filters use one causal axis of L
 * points with C = (N-1)*D (kernel o*D + d is filter o of channel d); the 2-D and
 * 3-D steps use signed axes on their kernel grid (2H x 2W, or H x W for a
 * circular plan) with C = D. */
typedef struct hyena_synth_params_s {
    int64_t axes;          /* 1, 2 or 3 */
    int64_t grid[3];       /* points per axis; at most 2^28 points in all */
    uint32_t signed_axes;  /* bit i: axis i holds signed offsets */
    int64_t width;         /* W: 8, 16, 32 or 64 */
    int64_t layers;        /* M: 1 .. 16 */
    int64_t zdim;          /* Z: 1 .. 256 */
    int64_t channels;      /* C: 1 .. 2^24 */
    const float* w_first;
    const float* w_hidden;
    const float* b_layer;
    const float* omega;
    const float* film_g;
    const float* film_gb;
    const float* film_b;
    const float* film_bb;
    const float* w_out;
    const float* b_out;
    const float* win_mu;
    const float* win_sigma;
} hyena_synth_params_t;

/* Synthesise B samples' kernels from their control vectors:
 *   z [B][Z] fp32, device: the control vector of every sample (derived by the
 *     model from its register tokens)
 *   k [B][C][grid points] fp32, device (output): kernel kk of sample b at
 *     k + (b*C + kk) * points, points in row-major grid order; for 1-D filters this
 *     is the [B][N-1][D][L] input of hyena_filter_spectrum_batched.
 * Enqueued on `stream` on the current device (no plan). HYENA_ERR_INVALID_ARG for
 * NULL or misaligned pointers, B < 1, sizes below 1 or signed bits beyond the axes;
 * HYENA_ERR_UNSUPPORTED for a width other than 8/16/32/64, more than 16 layers,
 * Z > 256, more than 2^28 grid points, B > 65535 or C > 2^24; HYENA_ERR_DEVICE if
 * the launch fails. */
hyena_status_t hyena_kernel_synthesis(const hyena_synth_params_t* params, int64_t B, const float* z, float* k,
                                      hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): hyena_forward with no
 * workspace argument and no allocation of any kind. The four-step and
 * partitioned paths keep their tiles in a scratch array of
 * HYENA_NOALLOC_SCRATCH_BYTES bytes that the library holds in device memory on
 * every GPU it runs on, from load until the process ends (the LDS path needs
 * none); chunks of rows are sized to it, so long rows run fewer rows per launch
 * than with the recommended workspace (the results are the same bits).
 * Every call on one GPU shares that GPU's array: calls that overlap in time on
 * one GPU (on different streams, or from different host threads without
 * ordering) race and give undefined results. The array's contents on entry are
 * irrelevant. Same arguments, results and errors as hyena_forward otherwise;
 * HYENA_ERR_WORKSPACE if one row's tiles exceed the array (not reachable with
 * the supported sizes), HYENA_ERR_DEVICE if the array's address cannot be
 * obtained on the current device. */
#define HYENA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
hyena_status_t hyena_forward_noalloc(hyena_plan_t plan, int64_t B, const void* u_proj, const float* short_w,
                                     const void* spec, const float* bias, void* y, hipStream_t stream);

/* hyena_forward with a filter set per sample (input-dependent long convolutions,
 * the HyenaND summary's methodology): sample b is convolved with the filters whose
 * spectrum hyena_filter_spectrum_batched wrote at byte b * hyena_spectrum_bytes
 * of `spec` (B spectra, B as in this call); short_w and bias stay shared. Same
 * arguments, workspace, results and errors as hyena_forward otherwise. */
hyena_status_t hyena_forward_per_sample(hyena_plan_t plan, int64_t B, const void* u_proj, const float* short_w,
                                        const void* spec, const float* bias, void* y, void* workspace,
                                        size_t workspace_bytes, hipStream_t stream);

/* hyena_forward with per-kernel timing, for measurement. HIP events are
 * recorded on `stream` around every kernel launch of this forward; the call
 * then waits for the last event (so it is synchronous), and writes elapsed
 * milliseconds summed per kernel family into ms[6]:
 *   ms[0] the single kernel of the LDS path, ms[1] four-step pass A (column
 *   FFTs of the gated input), ms[2] pass B (row FFTs, spectrum multiply,
 *   inverse rows), ms[3] pass C (inverse columns and gate; for order > 2 it
 *   also carries the next step's pass A), ms[4] first event to last event,
 *   ms[5] the pipelined four-step launches (each runs all three passes, on
 *   different chunks). On the partitioned path ms[1] is pass 1 (window
 *   transforms) and ms[2] pass 2 (block sums, inverse transforms, gate).
 * Same arguments, results and errors as hyena_forward; HYENA_ERR_INVALID_ARG
 * also for ms == NULL or more than 4096 events. */
hyena_status_t hyena_forward_timed(hyena_plan_t plan, int64_t B, const void* u_proj, const float* short_w,
                                   const void* spec, const float* bias, void* y, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream, float* ms);

/* Bytes of workspace hyena_backward needs for batch B.
 * LDS path: per (b, d) row the N-1 product spectra that the batch sums of dh are
 * taken from, the gated-input spectra of steps 0..N-3 and the values v_1..v_{N-2}
 * (8 bytes per complex or pair value), then 3 floats of short-conv tap sums per
 * (b, channel): 8*B*D*((2N-3)*L + (N-2)*L/2) + 12*B*(N+1)*D.
 * Four-step path: per (b, d) row N+1 L-point complex tiles (the transform, the
 * N-1 gated inputs after their column transforms, the row's share of dh after the
 * inverse rows), N-2
 * fp32 rows of recomputed values and N+1 fp32 staging rows; and 12*(N+1) bytes
 * of tap sums per (row, column block); each region 256-byte aligned. A circular
 * plan (LDS path only) counts L/2-point transforms and L sample pairs per value.
 * Returns 0 for a NULL plan, B < 1, or a circular four-step plan. */
size_t hyena_backward_workspace_bytes(hyena_plan_t plan, int64_t B);

/* Backward of the forward hot path: given the upstream gradient dy of y, the
 * gradients of the same scalar loss with respect to u_proj, short_w, the long
 * filters h (time domain, i.e. through hyena_filter_spectrum) and bias. They
 * follow from the forward's definitions (HyenaDNA walkthrough, section 2.1,
 * HyenaOperator.forward; section 2.2, HyenaFilter.forward and fftconv) by the
 * chain rule; the adjoint of the causal convolution with h is the correlation
 * corr(a, h)[t] = sum_{s >= t} h[s-t] a[s], taken through the same zero-padded
 * 2L-point spectra with the filter spectrum conjugated.
 *   u_proj, short_w, spec, bias: the forward's inputs (spec from
 *           hyena_filter_spectrum of this plan)
 *   dy      [B][D][L] of the plan dtype, device
 *   du_proj [B][(N+1)*D][L] of the plan dtype, device (output; bf16 rounded to
 *           nearest even)
 *   dshort_w [(N+1)*D][3] fp32, dh [N-1][D][L] fp32, dbias [N-1][D] fp32, device
 *           (outputs; the batch sums are complete, not accumulated into the
 *           buffers' previous contents)
 *   workspace / workspace_bytes: device scratch of at least
 *           hyena_backward_workspace_bytes(plan, B); contents on entry irrelevant.
 * Both paths have a backward for every order. For a circular plan (LDS path
 * only; a circular four-step plan gives HYENA_ERR_UNSUPPORTED) the correlations
 * are circular too (corr(a, k)[t] = sum_s k[(s - t) mod L] a[s]), dh has L taps
 * per filter and the short conv's transpose keeps its causal form. Every sum over the batch
 * or over workgroups is taken in a fixed order (no atomics), so results are
 * bitwise reproducible.
 * Enqueued on `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL or misaligned
 * pointers, B < 1), HYENA_ERR_UNSUPPORTED, HYENA_ERR_WORKSPACE,
 * HYENA_ERR_DEVICE (launch failure, wrong current device). Outputs must not
 * alias inputs or each other. */
hyena_status_t hyena_backward(hyena_plan_t plan, int64_t B, const void* u_proj, const float* short_w,
                              const void* spec, const float* bias, const void* dy, void* du_proj, float* dshort_w,
                              float* dh, float* dbias, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace hyena_backward_per_sample needs for batch B: as
 * hyena_backward_workspace_bytes, except on the four-step path, where B*D floats
 * of per-sample dbias terms are added. Returns 0 for a NULL plan, B < 1, or a
 * circular four-step plan. */
size_t hyena_backward_per_sample_workspace_bytes(hyena_plan_t plan, int64_t B);

/* Backward of hyena_forward_per_sample (a filter set per sample, the HyenaND
 * summary's input-dependent convolutions): spec holds the B spectra of
 * hyena_filter_spectrum_batched, and sample b's filter gradient is its own, so
 *   dh      [B][N-1][D][L] fp32, device (output): dh[b] is the gradient with
 *           respect to sample b's filters h[b] [N-1][D][L]
 * while dshort_w and dbias, whose parameters every sample shares, are batch sums
 * as in hyena_backward. Every other argument, the workspace (of at least
 * hyena_backward_per_sample_workspace_bytes(plan, B)), the fixed summation order
 * and the errors are those of hyena_backward; in addition HYENA_ERR_INVALID_ARG
 * when B*(N-1)*D*L exceeds 2^35 (dh alone would pass 128 GiB). */
hyena_status_t hyena_backward_per_sample(hyena_plan_t plan, int64_t B, const void* u_proj, const float* short_w,
                                         const void* spec, const float* bias, const void* dy, void* du_proj,
                                         float* dshort_w, float* dh, float* dbias, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace hyena_operator_forward needs for batch B: the in-projected
 * activation u_proj, the path output y, either the identity short-conv taps
 * (bf16 plans with D a multiple of 64, whose input projection is fused with the
 * short conv) or, for the other plans, x and w_in with the input-bias term
 * appended to each row (B*L + (N+1)*D rows of Dp = D + 1 rounded up to 8
 * values), 32 MiB of GEMM scratch and the path's own workspace
 * (hyena_workspace_bytes), each 256-byte aligned. Returns 0 for a NULL plan or
 * B < 1. */
size_t hyena_operator_workspace_bytes(hyena_plan_t plan, int64_t B);

/* The whole operator forward around the hot path (HyenaDNA walkthrough, section
 * 2.1, HyenaOperator.forward): in_proj, the (B, L, D) -> (B, D, L) transpose, the
 * hot path as in hyena_forward, the transpose back, out_proj:
 *   u_proj[b][c][t] = sum_k w_in[c][k] x[b][t][k] + b_in[c]
 *   out[b][t][j]    = sum_d w_out[j][d] y[b][d][t] + b_out[j]
 *   x     [B][L][D] of the plan dtype, device
 *   w_in  [(N+1)*D][D], b_in [(N+1)*D], w_out [D][D], b_out [D]: the projections'
 *         weights and biases (PyTorch nn.Linear layout), plan dtype, device
 *   short_w, spec, bias: as in hyena_forward
 *   out   [B][L][D] of the plan dtype, device (output)
 *   workspace: at least hyena_operator_workspace_bytes(plan, B) bytes.
 * bf16 plans with D a multiple of 64: the input projection runs in libhyena's own
 * bf16 matrix-core kernel, one launch over every sequence, fused with b_in and
 * the short conv (applied to the fp32 sums, then rounded once to bf16); the path
 * then runs with identity taps. Other plans: the input projection is a hipBLASLt
 * GEMM per sequence (u_proj rounded to the plan dtype) and the path applies the
 * short conv. The output projection of bf16 plans with D a multiple of 64 and L
 * a multiple of 8 runs in libhyena's own bf16 matrix-core kernel, one launch over
 * every sequence (fp32 accumulation, b_out added, rounded once); otherwise it is a
 * hipBLASLt GEMM per sequence (fp32 accumulation). hipBLASLt's heuristic choice of
 * kernel is used unless hyena_operator_tune has run on the plan. The first call
 * on a plan attaches the
 * GEMM state to it (a hipBLASLt handle and descriptors), so calls on one plan are
 * serialised internally; hyena_plan_destroy releases it. The call never waits on
 * the device.
 * Enqueued on `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL or misaligned
 * pointers, B < 1, sizes too large), HYENA_ERR_WORKSPACE, HYENA_ERR_UNSUPPORTED
 * (no GEMM kernel for these shapes), HYENA_ERR_DEVICE, and those of
 * hyena_forward. Outputs must not alias inputs. */
hyena_status_t hyena_operator_forward(hyena_plan_t plan, int64_t B, const void* x, const void* w_in,
                                      const void* b_in, const float* short_w, const void* spec, const float* bias,
                                      const void* w_out, const void* b_out, void* out, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/* Times hipBLASLt's candidate kernels for this plan's projection GEMMs on the
 * given buffers (a few calls each) and keeps the fastest for later calls on the
 * plan. Same arguments and errors as hyena_operator_forward; it overwrites `out`
 * and the workspace with scratch values and returns after the stream has finished
 * (a blocking call, made once before timing-sensitive use). */
hyena_status_t hyena_operator_tune(hyena_plan_t plan, int64_t B, const void* x, const void* w_in, const void* b_in,
                                   const float* short_w, const void* spec, const float* bias, const void* w_out,
                                   const void* b_out, void* out, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/* hyena_operator_forward with timing: HIP events around the three stages on
 * `stream`; waits for the last one and writes milliseconds into ms[4]:
 * ms[0] input projection (with the bias or tap fill; the short conv as well on the
 * fused bf16 path), ms[1] the hot path, ms[2] output
 * projection, ms[3] total. HYENA_ERR_INVALID_ARG also for ms == NULL. */
hyena_status_t hyena_operator_forward_timed(hyena_plan_t plan, int64_t B, const void* x, const void* w_in,
                                            const void* b_in, const float* short_w, const void* spec,
                                            const float* bias, const void* w_out, const void* b_out, void* out,
                                            void* workspace, size_t workspace_bytes, hipStream_t stream,
                                            float* ms);

/* Parameters of the implicit long-filter generator (HyenaDNA walkthrough, section
 * 2.2, HyenaFilter). With E = emb_dim (odd, 3..127), K = (E-1)/2 bands,
 * W = width (8, 16, 32 or 64), M = num_inner (0..16) and C = (N-1)*D of the plan;
 * all arrays fp32, row-major, device, 16-byte aligned:
 *   band_freq [K]      frequencies f_k of the positional sine/cosine bands
 *   w_in [W][E], b_in [W]                 first Linear (PyTorch nn.Linear layout)
 *   w_inner [M][W][W], b_inner [M][W]     inner Linears (may be NULL when M = 0)
 *   sin_freq [W]       frequency of the Sin activation, shared by all its uses
 *   w_out [C][W]       output Linear, no bias; row c = o*D + d
 *   alpha [C]          modulation rates */
typedef struct hyena_filter_mlp_s {
    int64_t emb_dim;
    int64_t width;
    int64_t num_inner;
    const float* band_freq;
    const float* w_in;
    const float* b_in;
    const float* w_inner;
    const float* b_inner;
    const float* sin_freq;
    const float* w_out;
    const float* alpha;
} hyena_filter_mlp_t;

/* The implicit long filters of the plan (HyenaDNA walkthrough, section 2.2,
 * HyenaFilter.filter: positional embedding, the Linear/Sin stack, modulation; and
 * the [L, (N-1)*D] -> [N-1][D][L] reshape of section 2.1). For tau = 0..L-1, t = tau/L:
 *   z    = (t, sin(2 pi f_1 t) .. sin(2 pi f_K t), cos(2 pi f_1 t) .. cos(2 pi f_K t))
 *   a    = sin(sin_freq * (w_in z + b_in)),  then M times  a = sin(sin_freq * (w_inner[m] a + b_inner[m]))
 *   h[o][d][tau] = exp(-alpha[c] t) * sum_j w_out[c][j] a[j],   c = o*D + d
 * (the pages give the structure but not these formulas: the positional features,
 * the Sin activation and the modulation are this library's readings of them).
 *   h [N-1][D][L] fp32, device (output): the layout hyena_filter_spectrum takes.
 * The positional features are evaluated in fp64 and rounded once; the stack runs
 * in fp32; exp(-alpha t) is evaluated as 2^(alpha * (-t log2 e)) with the hardware
 * exp2 (relative error about 1e-7). Enqueued on `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL plan, mlp or
 * h, NULL arrays, even or too small emb_dim, misaligned pointers),
 * HYENA_ERR_UNSUPPORTED (width not 8/16/32/64, emb_dim > 127, num_inner > 16),
 * HYENA_ERR_DEVICE. h must not alias the parameters. */
hyena_status_t hyena_implicit_filter(hyena_plan_t plan, const hyena_filter_mlp_t* mlp, float* h,
                                     hipStream_t stream);

/* ------------------------------------------------------------------------
 * 2-D long convolution (HyenaND summary, methodology: global convolution on the
 * native N-d grid by an N-d FFT; the non-circular mode zero-pads the input to
 * double the grid in every dimension). One gated step per (b, d) image, as one
 * step of the 1-D recurrence above:
 *   s = v * g            (g optional: s = v when NULL)
 *   c[p][q] = sum_{i < 2H, j < 2W} k[i][j] s_pad[(p - i) mod 2H][(q - j) mod 2W]
 *   y = (c + bias * s) * x   (x optional),     p < H, q < W,
 * where s_pad is s zero-padded to 2H x 2W and the kernel k is given on the
 * doubled grid: rows i >= H and columns j >= W hold the negative offsets i - 2H
 * and j - 2W, so a causal kernel (zero outside [0,H) x [0,W)) and a centred one
 * are both expressible. (How the HyenaND operator synthesises its kernels and
 * what short convolution it applies on a grid are not on the pages; this is the
 * convolution step on its own.)
 * ------------------------------------------------------------------------ */
typedef struct hyena_plan2d_s* hyena_plan2d_t; /* opaque */

/* Plan for H x W images (powers of two, 16 <= H <= 512, 32 <= W <= 512) of D
 * channels; dtype of v, g, x and y as for the 1-D plans. The plan owns its
 * twiddle tables on the current device. Errors as hyena_plan_create. */
hyena_status_t hyena_plan2d_create(hyena_plan2d_t* out, int64_t H, int64_t W, int64_t D, hyena_dtype_t dtype);

/* As hyena_plan2d_create, with option flags (0 or HYENA_FLAG_CIRCULAR). A circular
 * plan convolves the grid periodically (the HyenaND summary's boundary handling
 * for periodic systems), with the kernel k[D][H][W] on the grid itself:
 *   c[p][q] = sum_{i < H, j < W} k[i][j] s[(p - i) mod H][(q - j) mod W];
 * its spectrum is D * H * (W/2 + 1) complex values (rfft2 of the H x W kernel,
 * scaled by 1/(2 * H * W)), its workspace 4*H*W bytes per image; 32 <= H <= 1024,
 * 64 <= W <= 1024. HYENA_ERR_INVALID_ARG for unknown flag bits. */
hyena_status_t hyena_plan2d_create_ex(hyena_plan2d_t* out, int64_t H, int64_t W, int64_t D, hyena_dtype_t dtype,
                                      uint32_t flags);

/* Release a 2-D plan. NULL is a no-op. */
hyena_status_t hyena_plan2d_destroy(hyena_plan2d_t plan);

/* Bytes of a 2-D kernel spectrum: D * 2H * (W + 1) complex fp32 values, the
 * doubled grid's real-transform bins (numpy.fft.rfft2 layout) of each channel,
 * scaled by 1/(4 * 2H * W). Returns 0 for a NULL plan. */
size_t hyena_spectrum2d_bytes(hyena_plan2d_t plan);

/* Workspace for hyena_conv2d_forward over batch B: any size of at least one
 * image tile (8 * H * W bytes) is accepted; this is the recommended size (up to
 * 128 MiB of tiles per launch). Returns 0 for a NULL plan or B < 1. */
size_t hyena_workspace2d_bytes(hyena_plan2d_t plan, int64_t B);

/* Kernel spectra, once per plan.
 *   k    [D][2H][2W] fp32, device: the kernels on the doubled grid
 *   spec device buffer of hyena_spectrum2d_bytes(plan) bytes (output)
 * Enqueued on `stream`. HYENA_ERR_INVALID_ARG for NULL or misaligned pointers,
 * HYENA_ERR_DEVICE for launch failures or a wrong current device. */
hyena_status_t hyena_filter_spectrum2d(hyena_plan2d_t plan, const float* k, void* spec, hipStream_t stream);

/* The gated 2-D long convolution above for B x D images.
 *   v    [B][D][H][W] of the plan dtype, device
 *   g, x [B][D][H][W] of the plan dtype, device, or NULL (no gate)
 *   spec from hyena_filter_spectrum2d of this plan; bias [D] fp32, device
 *   y    [B][D][H][W] of the plan dtype, device (output; must not alias inputs)
 *   workspace / workspace_bytes: at least 8*H*W bytes (see hyena_workspace2d_bytes)
 * Three passes per chunk of images: column FFTs of the gated image, row FFTs with
 * the spectrum multiply and the inverse rows, inverse columns with the gate; all
 * intermediates fp32. Enqueued on `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL or
 * misaligned pointers, B < 1, B*D > 2^24), HYENA_ERR_WORKSPACE, HYENA_ERR_DEVICE. */
hyena_status_t hyena_conv2d_forward(hyena_plan2d_t plan, int64_t B, const void* v, const void* g, const void* x,
                                    const void* spec, const float* bias, void* y, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/* Input-dependent kernels (the HyenaND summary's methodology: a kernel set per
 * input sample): hyena_filter_spectrum2d for B kernel sets at once,
 *   k    [B][D][2H][2W] fp32, device; spec: B * hyena_spectrum2d_bytes(plan) bytes,
 *        sample b's spectrum at byte b * hyena_spectrum2d_bytes(plan),
 * and the forward in which image (b, d) uses sample b's kernel d (bias shared).
 * Errors as the calls above; HYENA_ERR_INVALID_ARG also for B < 1 or B*D > 2^24. */
hyena_status_t hyena_filter_spectrum2d_batched(hyena_plan2d_t plan, int64_t B, const float* k, void* spec,
                                               hipStream_t stream);
hyena_status_t hyena_conv2d_forward_per_sample(hyena_plan2d_t plan, int64_t B, const void* v, const void* g,
                                               const void* x, const void* spec, const float* bias, void* y,
                                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * 3-D long convolution: the 2-D step above with one more grid axis (HyenaND
 * summary, methodology: the N-d FFT convolution on the native grid, zero-padded
 * to double the grid in every dimension). One gated step per (b, d) volume:
 *   s = v * g            (g optional)
 *   c[a][p][q] = sum_{l < 2A, i < 2H, j < 2W} k[l][i][j]
 *                s_pad[(a - l) mod 2A][(p - i) mod 2H][(q - j) mod 2W]
 *   y = (c + bias * s) * x   (x optional),     a < A, p < H, q < W,
 * with the kernel given on the doubled grid (an index >= the axis length holds
 * the negative offset, as in 2-D).
 * ------------------------------------------------------------------------ */
typedef struct hyena_plan3d_s* hyena_plan3d_t; /* opaque */

/* Plan for A x H x W volumes (powers of two, 16 <= A, H <= 512, 32 <= W <= 512,
 * A*H*W <= 2^24) of D channels; dtype of v, g, x and y as for the 1-D plans. The
 * plan owns its twiddle tables on the current device. Errors as
 * hyena_plan_create. */
hyena_status_t hyena_plan3d_create(hyena_plan3d_t* out, int64_t A, int64_t H, int64_t W, int64_t D,
                                   hyena_dtype_t dtype);

/* As hyena_plan3d_create, with option flags (0 or HYENA_FLAG_CIRCULAR): a
 * circular plan convolves the volume periodically with the kernel k[D][A][H][W]
 * on the grid itself; its spectrum is D * A * H * (W/2 + 1) complex values
 * (rfftn of the kernel, scaled by 1/(2 * A * H * W)), its workspace 4*A*H*W
 * bytes per volume; 32 <= A, H <= 1024, 64 <= W <= 1024. */
hyena_status_t hyena_plan3d_create_ex(hyena_plan3d_t* out, int64_t A, int64_t H, int64_t W, int64_t D,
                                      hyena_dtype_t dtype, uint32_t flags);

/* Release a 3-D plan. NULL is a no-op. */
hyena_status_t hyena_plan3d_destroy(hyena_plan3d_t plan);

/* Bytes of a 3-D kernel spectrum: D * 2A * 2H * (W + 1) complex fp32 values, the
 * doubled grid's real-transform bins (numpy.fft.rfftn layout) of each channel,
 * scaled by 1/(4 * 2A * 2H * W). Returns 0 for a NULL plan. */
size_t hyena_spectrum3d_bytes(hyena_plan3d_t plan);

/* Workspace for hyena_conv3d_forward over batch B: any size of at least one
 * volume's tiles is accepted: for a zero-padded plan 24 * A * H * W bytes, or
 * 8 * A * H * W when a depth slice's height x row transform (2H x W packed points)
 * has at most 4096 points (the slab pass keeps one tile); 4 * A * H * W bytes for a
 * circular plan. This is the recommended size (up to 192 MiB of tiles per launch).
 * Returns 0 for a NULL plan or B < 1. */
size_t hyena_workspace3d_bytes(hyena_plan3d_t plan, int64_t B);

/* Kernel spectra, once per plan.
 *   k    [D][2A][2H][2W] fp32, device: the kernels on the doubled grid
 *   spec device buffer of hyena_spectrum3d_bytes(plan) bytes (output)
 * Enqueued on `stream`. HYENA_ERR_INVALID_ARG for NULL or misaligned pointers,
 * HYENA_ERR_DEVICE for launch failures or a wrong current device. */
hyena_status_t hyena_filter_spectrum3d(hyena_plan3d_t plan, const float* k, void* spec, hipStream_t stream);

/* The gated 3-D long convolution above for B x D volumes.
 *   v    [B][D][A][H][W] of the plan dtype, device
 *   g, x [B][D][A][H][W] of the plan dtype, device, or NULL (no gate)
 *   spec from hyena_filter_spectrum3d of this plan; bias [D] fp32, device
 *   y    [B][D][A][H][W] of the plan dtype, device (output; must not alias inputs)
 *   workspace / workspace_bytes: at least one volume's tiles (hyena_workspace3d_bytes)
 * Five passes per chunk of volumes: column FFTs over a of the gated volume and
 * over h, row FFTs over w with the spectrum multiply and the inverse rows, inverse
 * columns over h and over a with the gate; all intermediates fp32. When a pair of
 * depth slices fits one workgroup's LDS (the sizes above), the middle three run as
 * one pass per slice pair on chip. Enqueued on
 * `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL or misaligned pointers, B < 1,
 * B*D > 2^24), HYENA_ERR_WORKSPACE, HYENA_ERR_DEVICE. */
hyena_status_t hyena_conv3d_forward(hyena_plan3d_t plan, int64_t B, const void* v, const void* g, const void* x,
                                    const void* spec, const float* bias, void* y, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/* A kernel set per input sample, as for 2-D: k [B][D][2A][2H][2W] fp32 gives B
 * spectra of hyena_spectrum3d_bytes(plan) bytes each; volume (b, d) uses sample
 * b's kernel d. */
hyena_status_t hyena_filter_spectrum3d_batched(hyena_plan3d_t plan, int64_t B, const float* k, void* spec,
                                               hipStream_t stream);
hyena_status_t hyena_conv3d_forward_per_sample(hyena_plan3d_t plan, int64_t B, const void* v, const void* g,
                                               const void* x, const void* spec, const float* bias, void* y,
                                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Gated delta rule: a causal mixer of linear cost beside the long convolutions
 * above, with a state of constant size. Every sequence and value head has a
 * state S [dim_k][dim_v]; for each token in order, with the log decay g (g <= 0
 * forgets, 0 keeps) and the write strength beta,
 *   S <- exp(g) S;   S <- S + beta k (v - S^T k)^T;   o = scale S^T q,
 * so the state's answer to the key k moves from S^T k towards v. The value heads
 * share query and key heads in groups: value head h uses query/key head
 * h / (heads_v / heads_k). Keys should have at most unit length (hyena_qk_norm_*
 * gives it): with beta in [0, 1] the update is then a contraction.
 *
 * The calls take no plan: they run on the current device, which must be the one
 * that holds the buffers. States are fp32 [dim_k][dim_v], row-major. Tokens lie
 * behind each other, either as N sequences of tokens / N each (seq_start NULL) or
 * packed, sequence n being tokens seq_start[n] .. seq_start[n+1]-1 (N + 1 offsets
 * in device memory, not decreasing, seq_start[N] <= tokens; sequences may be
 * empty). Offsets are read on the device: ones that break this rule give undefined
 * results but no access outside the buffers. Rows that belong to no sequence are
 * neither read nor written.
 * ------------------------------------------------------------------------ */
typedef struct hyena_delta_params_s {
    int64_t heads_k, heads_v; /* heads_v a multiple of heads_k */
    int64_t dim_k, dim_v;     /* multiples of 8; dim_k <= 128, dim_v <= 256 */
    hyena_dtype_t dtype;      /* of q, k, v, g, beta, o and their gradients */
    float scale;              /* of the queries, usually dim_k^-1/2; finite */
} hyena_delta_params_t;

/* Device arrays of one call. Token t's heads lie behind each other at
 *   q + t*ldq, k + t*ldk [heads_k][dim_k],   v + t*ldv [heads_v][dim_v]
 * (elements; q, k and v may be column ranges of one projection's rows); ld* at
 * least the heads' width, a multiple of 16 bytes and at most 2^22.
 * g, beta [tokens][heads_v], dense, aligned to their elements. */
typedef struct hyena_delta_inputs_s {
    const void* q;
    int64_t ldq;
    const void* k;
    int64_t ldk;
    const void* v;
    int64_t ldv;
    const void* g;
    const void* beta;
} hyena_delta_inputs_t;

/* Bytes of workspace hyena_delta_forward needs (the triangular factors and decays of
 * chunks of 64 tokens; states between the pieces of long sequences). Returns 0 for arguments that
 * the call would refuse, and where there are no tokens. seq_start is not read:
 * only whether it is NULL matters. */
size_t hyena_delta_workspace_bytes(const hyena_delta_params_t* params, int64_t N, int64_t tokens,
                                   const int64_t* seq_start);

/* The gated delta rule over whole sequences, in chunks of 64 tokens on the matrix
 * cores.
 *   state_in  [N][heads_v][dim_k][dim_v] fp32, device, or NULL (zeros)
 *   o         [tokens][heads_v][dim_v] of the dtype, device (output)
 *   state_out [N][heads_v][dim_k][dim_v] fp32, device (output), or NULL; may be
 *             state_in itself. An empty sequence passes its state on.
 *   workspace at least hyena_delta_workspace_bytes(...) bytes, 16-byte aligned
 * The state is held in fp32 from the first token to the last; bf16 outputs are
 * rounded once from sums whose operands are bf16 or sums of two bf16 parts, fp32
 * results have the accuracy of fp32 products. Decays below exp(-200) count as 0 and
 * g = -inf resets the state. A value that is not finite (but for g = -inf) spoils its token
 * and what follows in the sequence, as in the recurrence, and nothing in front of it: of v
 * in its column, of k, g and beta in their value heads. One of q spoils its token alone. Every sum has a fixed order: results are bitwise
 * reproducible, and those of a sequence of up to 1536 tokens do not depend on the other
 * sequences of the call. Longer ones are cut into pieces that run side by side where the
 * call has few (sequence, head) pairs; how is a rule on the sizes, N and tokens among
 * them, and another cut may round differently. Outputs must not alias inputs, but for
 * state_out. Enqueued on `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL or misaligned
 * pointers, sizes below 1, tokens not a multiple of N without seq_start, heads_v not a
 * multiple of heads_k, bad ld or scale), HYENA_ERR_UNSUPPORTED (dims outside the ranges
 * above, heads_v > 65535, heads_k * dim_k or heads_v * dim_v > 2^22, N > 2^24,
 * tokens > 2^31, more than 2^30 (chunk, head) or 2^26 (sequence, head) pairs, or a launch
 * of 2^32 threads or more: 256 for each chunk, and for each (sequence, head) pair 256 for
 * every 32 columns of dim_v, in fp32 192 for every 16), HYENA_ERR_WORKSPACE,
 * HYENA_ERR_DEVICE. */
hyena_status_t hyena_delta_forward(const hyena_delta_params_t* params, int64_t N, int64_t tokens,
                                   const int64_t* seq_start, const hyena_delta_inputs_t* in, const float* state_in,
                                   void* o, float* state_out, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/* Zeros the rows of `count` (1 to 8) arrays [tokens][row_bytes] that belong to no sequence
 * of a packed call, those in front of seq_start[0] and from seq_start[N] on: outputs of the
 * calls here leave them as they were, and gradients of inputs that were not read are 0.
 * arrays and row_bytes are host arrays; each array and row 2-byte aligned. Offsets outside
 * [0, tokens] are held to it. Enqueued on `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL or
 * misaligned pointers, N < 1, tokens < 0, count or a row's size out of range),
 * HYENA_ERR_DEVICE. */
hyena_status_t hyena_delta_clear_rows(int64_t N, int64_t tokens, const int64_t* seq_start, int count,
                                      void* const* arrays, const int64_t* row_bytes, hipStream_t stream);

/* Bytes of workspace hyena_delta_backward needs: the forward's, the states before and
 * the state gradients behind every chunk of 64 tokens, and two arrays of o's shape, all at
 * three (bf16) or four bytes a value. Returns 0 as hyena_delta_workspace_bytes. */
size_t hyena_delta_backward_workspace_bytes(const hyena_delta_params_t* params, int64_t N, int64_t tokens,
                                            const int64_t* seq_start);

/* Backward of hyena_delta_forward: with the forward's inputs and the gradients
 *   dout       [tokens][heads_v][dim_v] of the dtype, of o
 *   dstate_out [N][heads_v][dim_k][dim_v] fp32, of the final states, or NULL (zeros)
 * of one scalar, its gradients with respect to every input (outputs, dense):
 *   dq, dk [tokens][heads_k][dim_k], dv [tokens][heads_v][dim_v], dg, dbeta
 *   [tokens][heads_v] of the dtype, rounded once from fp32 sums (over the value heads
 *   that share a key head, too); dstate_in [N][heads_v][dim_k][dim_v] fp32, or NULL.
 * The states are computed again from the inputs; nothing of the forward call is kept.
 * Operands of bf16 calls are bf16 or sums of two bf16 parts, the states and their
 * gradients stay fp32 along both scans. Values that are not finite spoil the gradients of
 * their sequence's earlier tokens, too. dbeta is formed from the residual v - answer itself and stays exact where
 * the state predicts v; for it, strengths below 2^-90 count as 2^-90. Every sum has a fixed
 * order: results are bitwise reproducible. Rows that belong to no sequence are left as they were. Arguments, workspace (of at least
 * hyena_delta_backward_workspace_bytes) and errors otherwise as in
 * hyena_delta_forward. Outputs must not alias inputs or each other. */
hyena_status_t hyena_delta_backward(const hyena_delta_params_t* params, int64_t N, int64_t tokens,
                                    const int64_t* seq_start, const hyena_delta_inputs_t* in, const float* state_in,
                                    const void* dout, const float* dstate_out, void* dq, void* dk, void* dv, void* dg,
                                    void* dbeta, float* dstate_in, void* workspace, size_t workspace_bytes,
                                    hipStream_t stream);

/* The recurrent form: T further tokens (one when answering token by token, a few
 * drafted ones) of each of B rows, row b's tokens at b*T .. b*T + T - 1 of the
 * inputs and of o [B*T][heads_v][dim_v].
 *   states [num_states][heads_v][dim_k][dim_v] fp32, device: read and updated in
 *          place, once each
 *   slots  [B] int32, device: the state of every row, or NULL (row b has state b,
 *          num_states >= B). Rows that name the same slot are taken in order, as
 *          successive tokens of it. A row whose slot is outside [0, num_states) gives
 *          zeros and touches no state (rows that pad a captured batch).
 * All arithmetic is fp32. Enqueued on `stream`; no workspace. Errors as
 * hyena_delta_forward, of N = B and tokens = B*T, but for the launch: HYENA_ERR_UNSUPPORTED
 * where 64 threads for every 32 columns of dim_v (at most 256) of each (row, head) pair
 * are 2^32 or more; HYENA_ERR_INVALID_ARG also for
 * B, T or num_states below 1 and for NULL slots with num_states < B. */
hyena_status_t hyena_delta_step(const hyena_delta_params_t* params, int64_t B, int64_t T,
                                const hyena_delta_inputs_t* in, float* states, int64_t num_states,
                                const int32_t* slots, void* o, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Norms of queries and keys for each head, with the position rotation in the same
 * pass. For the vector x [dim] of one head of one token, weight w and F = rot pairs:
 *   n = x / sqrt(mean(x^2) + eps)  (HYENA_NORM_RMS)
 *   n = x / sqrt(sum(x^2) + eps)   (HYENA_NORM_L2: unit length, what the gated delta
 *                                   rule wants of its keys)
 *   y = n * w, then for i < F the pair (y[i], y[i+F]) (HYENA_ROT_HALVES) or
 *   (y[2i], y[2i+1]) (HYENA_ROT_PAIRS) turned by the angle position * freq[i]:
 *   (a, b) -> (a cos - b sin, a sin + b cos).
 * Angles are formed and reduced in fp64, everything else is fp32 and rounded once. The
 * squares of a head sum up below 3e38 (elements to 1e18): past that the head's result is 0.
 * ------------------------------------------------------------------------ */
typedef enum { HYENA_NORM_RMS = 0, HYENA_NORM_L2 = 1 } hyena_norm_t;
typedef enum { HYENA_ROT_HALVES = 0, HYENA_ROT_PAIRS = 1 } hyena_rot_t;

typedef struct hyena_qk_norm_params_s {
    int64_t heads_q, heads_k;
    int64_t dim;         /* a multiple of 8, at most 256 */
    int64_t rot;         /* F: rotated pairs, a multiple of 4, 2 F <= dim; 0 for none */
    hyena_norm_t kind;
    hyena_rot_t layout;
    hyena_dtype_t dtype; /* of q, k, their outputs and gradients */
    float eps;           /* above 0, finite */
    const float* w_q;    /* [dim] fp32, device, shared by the heads, or NULL (ones) */
    const float* w_k;
    const float* freq;   /* [F] fp32, device: radians per position; NULL if F = 0 */
} hyena_qk_norm_params_t;

/* q [tokens][heads_q][dim] with ldq elements between tokens (at least the heads'
 * width, a multiple of 16 bytes, at most 2^31; a column range of a projection's rows
 * may be given as it lies), k likewise; positions [tokens] int64, device (NULL if
 * F = 0); q_out, k_out dense (outputs). Runs on the current device, no plan.
 * Enqueued on `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL or misaligned pointers,
 * bad sizes, ld, eps, kind or layout), HYENA_ERR_UNSUPPORTED (dim or rot outside the
 * ranges above, more than 65535 heads in all, tokens > 2^31), HYENA_ERR_DEVICE. */
hyena_status_t hyena_qk_norm_forward(const hyena_qk_norm_params_t* params, int64_t tokens, const void* q, int64_t ldq,
                                     const void* k, int64_t ldk, const int64_t* positions, void* q_out, void* k_out,
                                     hipStream_t stream);

/* Bytes of workspace that hold for hyena_qk_norm_backward of so many tokens or fewer where it
 * sums weight gradients (partial sums of at most 1024 workgroups, or one a head where there
 * are more). Returns 0 for arguments that the call would refuse and for tokens = 0. */
size_t hyena_qk_norm_backward_workspace_bytes(const hyena_qk_norm_params_t* params, int64_t tokens);

/* Backward: the gradients dq, dk (dense, outputs) of q and k, and dw_q, dw_k [dim] fp32
 * of the weights (outputs; NULL where not wanted; of the ones, where the weight is
 * NULL), for the gradients dq_out, dk_out (dense) of the forward's outputs. Weight
 * gradients are complete sums over tokens and heads in a fixed order. workspace: as
 * above, 16-byte aligned; ignored where neither weight gradient is asked for. Errors
 * as the forward's, and HYENA_ERR_WORKSPACE. Outputs must not alias inputs. */
hyena_status_t hyena_qk_norm_backward(const hyena_qk_norm_params_t* params, int64_t tokens, const void* q, int64_t ldq,
                                      const void* k, int64_t ldk, const int64_t* positions, const void* dq_out,
                                      const void* dk_out, void* dq, void* dk, float* dw_q, float* dw_k, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/* The same with a position of its own for every axis that a token lies on (time, height and
 * width of a video's patches, say): positions [tokens][axes] int64, device, and pair i
 * turns by positions[t][axis[i]] * freq[i]. axis [F] int32, device (NULL if F = 0); values
 * outside [0, axes) are held to it. How the pairs are shared out, in sections or by turns, is
 * axis alone. 1 <= axes <= 8. Workspace, layout and errors otherwise as above;
 * HYENA_ERR_INVALID_ARG also for axes < 1 and a NULL or misaligned axis,
 * HYENA_ERR_UNSUPPORTED for axes > 8. */
hyena_status_t hyena_qk_norm_axes_forward(const hyena_qk_norm_params_t* params, const int32_t* axis, int64_t axes,
                                          int64_t tokens, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                          const int64_t* positions, void* q_out, void* k_out, hipStream_t stream);
hyena_status_t hyena_qk_norm_axes_backward(const hyena_qk_norm_params_t* params, const int32_t* axis, int64_t axes,
                                           int64_t tokens, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                           const int64_t* positions, const void* dq_out, const void* dk_out, void* dq,
                                           void* dk, float* dw_q, float* dw_k, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream);

/* ------------------------------------------------------------------------
 * Gated linear recurrence: a causal mixer whose state is one value a channel. For
 * every channel of a sequence, with the pre-activations r and i, the channel's rate c > 0
 * and the state h, for each token in order
 *   log a = -c sig(r);   h <- a h + sqrt(1 - a^2) sig(i) x;   y = h,   sig(z) = 1 / (1 + exp(-z)).
 *
 * The calls take no plan: they run on the current device, which must be the one
 * that holds the buffers. Tokens lie behind each other as for the gated delta rule: N
 * sequences of tokens / N each (seq_start NULL), or packed with N + 1 offsets in device
 * memory under the same rules. Rows that belong to no sequence are not read; in outputs they are
 * left as they were or, where `clear` asks for it, set to 0.
 * ------------------------------------------------------------------------ */
#define HYENA_RECURRENCE_CARRY 80 /* tokens between the states that the forward keeps for its backward */

typedef struct hyena_recurrence_params_s {
    int64_t dim;         /* channels: a multiple of 8, at most 2^20 */
    hyena_dtype_t dtype; /* of x, r, i, y and their gradients */
    int clear;           /* not 0: rows of y, dx, dr and di that belong to no sequence become 0 */
    const float* rate;   /* [dim] fp32, device: c, a normal number above 0 */
} hyena_recurrence_params_t;

/* Token t's channels lie at x + t*ldx, r + t*ldr, i + t*ldi (elements; column ranges of one
 * projection's rows may be given as they lie); ld* at least dim, a multiple of 16 bytes and at
 * most 2^22 (hyena_recurrence_step: 2^31). */
typedef struct hyena_recurrence_inputs_s {
    const void* x;
    int64_t ldx;
    const void* r;
    int64_t ldr;
    const void* i;
    int64_t ldi;
} hyena_recurrence_inputs_t;

/* Bytes of workspace that hold for hyena_recurrence_forward and for its calls of fewer tokens or
 * channels, so that one workspace, sized for the largest call, serves them all. Returns 0 for arguments
 * that the call would refuse, and where there are no tokens. seq_start is not read. */
size_t hyena_recurrence_workspace_bytes(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                        const int64_t* seq_start);

/* The recurrence over whole sequences.
 *   state_in  [N][dim] fp32, device, or NULL (zeros)
 *   y         [tokens][dim] of the dtype, device (output)
 *   state_out [N][dim] fp32, device (output), or NULL; may be state_in itself. An empty sequence
 *             passes its state on.
 *   carries   [ceil(tokens / HYENA_RECURRENCE_CARRY)][dim] fp32, device (output), or NULL: the states
 *             in front of rows 0, 80, 160, ..., which spare hyena_recurrence_backward a pass over
 *             the inputs
 *   workspace at least hyena_recurrence_workspace_bytes(...) bytes, 16-byte aligned
 * All arithmetic is fp32 and y is rounded once. A value that is not finite spoils its channel of its
 * sequence from its token on and nothing else. Every sum has a fixed order: results are bitwise
 * reproducible; where a sequence lies among the rows, and how many there are, may change their
 * rounding. Outputs must not alias inputs, but for state_out. Enqueued on `stream`. Errors:
 * HYENA_ERR_INVALID_ARG (NULL or misaligned
 * pointers, sizes below 1, tokens not a multiple of N without seq_start, bad ld),
 * HYENA_ERR_UNSUPPORTED (dim not a multiple of 8 or above 2^20, N > 2^24, or 2^23 or more pairs of 80
 * tokens and 128 channels: above 671088560 tokens, of more than 128 channels fewer), HYENA_ERR_WORKSPACE,
 * HYENA_ERR_DEVICE. */
hyena_status_t hyena_recurrence_forward(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                        const int64_t* seq_start, const hyena_recurrence_inputs_t* in,
                                        const float* state_in, void* y, float* state_out, float* carries,
                                        void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace that hold for hyena_recurrence_backward, with carries or (NULL) without, and for
 * its calls of fewer tokens or channels; the pointers are not followed. Returns 0 as
 * hyena_recurrence_workspace_bytes. */
size_t hyena_recurrence_backward_workspace_bytes(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                                 const int64_t* seq_start, const float* carries);

/* Backward of hyena_recurrence_forward: with the forward's inputs and the gradients
 *   dy         [tokens][dim] of the dtype, of y
 *   dstate_out [N][dim] fp32, of the final states, or NULL (zeros)
 * of one scalar, its gradients with respect to every input (outputs, dense): dx, dr, di
 * [tokens][dim] of the dtype, drate [dim] fp32 (the whole sum over the tokens) and dstate_in [N][dim]
 * fp32 or NULL. carries: what the forward of the same inputs and states wrote, or NULL (then they
 * are computed again). Where sqrt(1 - a^2) falls to 0 (r far below 0), dr goes to 0 with it. Values that
 * are not finite spoil their channel's gradients in their sequence, in front of them too, and the
 * channel's drate. Sums and errors otherwise as the forward's. Outputs must not alias inputs or
 * each other. */
hyena_status_t hyena_recurrence_backward(const hyena_recurrence_params_t* params, int64_t N, int64_t tokens,
                                         const int64_t* seq_start, const hyena_recurrence_inputs_t* in,
                                         const float* state_in, const float* carries, const void* dy,
                                         const float* dstate_out, void* dx, void* dr, void* di, float* drate,
                                         float* dstate_in, void* workspace, size_t workspace_bytes,
                                         hipStream_t stream);

/* The recurrent form: T further tokens of each of B rows, row b's at b*T .. b*T + T - 1 of the
 * inputs and of y [B*T][dim]; states [num_states][dim] fp32, read and updated in place once each; slots
 * [B] int32 or NULL, both exactly as for hyena_delta_step: rows that name the same slot are
 * successive tokens of it, a slot outside [0, num_states) gives zeros. Enqueued on `stream`; no
 * workspace. Errors as hyena_recurrence_forward, but for its limit of pairs: HYENA_ERR_UNSUPPORTED where
 * 2^24 pairs of a row and 512 channels are reached, and for B or T > 2^24 or B*T > 2^31 - 256; and
 * HYENA_ERR_INVALID_ARG for B, T or num_states below 1 and for NULL slots with num_states < B. */
hyena_status_t hyena_recurrence_step(const hyena_recurrence_params_t* params, int64_t B, int64_t T,
                                     const hyena_recurrence_inputs_t* in, float* states, int64_t num_states,
                                     const int32_t* slots, void* y, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Residual norm: the addition to the residual stream and the root-mean-square norm in front of
 * the next layer in one pass. For a token's row x [dim]:
 *   s = residual + x,   y = s / sqrt(mean(s^2) + eps) * w.
 * The norm is that of the fp32 sum; s is rounded to the residual's type where it is stored. In 8
 * bits (e4m3: 4 exponent and 3 mantissa bits, no infinities) y is divided by the scale of its
 * row or block of 128 columns, the largest |y| there / 448 (at least 2^-126; 1 where all are 0),
 * and rounded to nearest even. Sums are fp32; the squares of a row sum up below 3e38: past that y is 0. An
 * infinity or NaN spoils its row; 8-bit scales come from the values that are not NaN.
 * ------------------------------------------------------------------------ */
typedef struct hyena_residual_norm_params_s {
    int64_t dim;                  /* a multiple of 8, at most 16384 */
    hyena_dtype_t dtype;          /* of x, y and their gradients */
    hyena_dtype_t residual_dtype; /* of the residual, s and their gradients; HYENA_F32 where dtype is */
    int64_t block;                /* of 8-bit outputs: 128 columns a scale, or 0: one a row */
    float eps;                    /* above 0, finite */
    const float* w;               /* [dim] fp32, device, or NULL (ones) */
} hyena_residual_norm_params_t;

/* x [rows][dim] with ldx elements between rows (at least dim, a multiple of 16 bytes, at most 2^31);
 * residual likewise, or NULL (s = x); y [rows][dim], dense: of the dtype, or where scales is not NULL in 8
 * bits, with scales [rows][1 or ceil(dim / 128)] fp32; sum [rows][dim], dense: s, or NULL. Runs on
 * the current device, no plan. y, scales and sum must not alias the inputs, but sum may be the
 * residual itself where that is dense. Enqueued on `stream`. Errors: HYENA_ERR_INVALID_ARG (NULL or
 * misaligned pointers, bad sizes, ld, eps, block or types), HYENA_ERR_UNSUPPORTED (dim outside the
 * range above, a bf16 residual of fp32
 * rows, rows > 2^31), HYENA_ERR_DEVICE. */
hyena_status_t hyena_residual_norm_forward(const hyena_residual_norm_params_t* params, int64_t rows, const void* x,
                                           int64_t ldx, const void* residual, int64_t ldr, void* y, float* scales,
                                           void* sum, hipStream_t stream);

/* Bytes of workspace hyena_residual_norm_backward needs where it sums the weight's gradient (partial
 * sums of at most 1024 workgroups). Returns 0 for arguments that the call would refuse and for rows = 0. */
size_t hyena_residual_norm_backward_workspace_bytes(const hyena_residual_norm_params_t* params, int64_t rows);

/* Backward: for the stored sums s [rows][dim] (with lds elements between rows, as ldx) and the gradients dy (of the
 * dtype, dense) of y and dsum (of the residual's type, dense; NULL: zeros) of s, the gradient of x and of the
 * residual, which is one and the same, rounded to either type: dx [rows][dim] of the dtype and
 * dresidual of the residual's, dense (outputs; NULL where not wanted, not all three), and dw [dim]
 * fp32 (output, or
 * NULL), a complete sum in a fixed order. An output in 8 bits has the gradients of the values before
 * they were rounded. workspace: as above, 16-byte aligned; ignored without dw. Errors as the forward's, and
 * HYENA_ERR_WORKSPACE. Outputs must not alias inputs, but dresidual may be dsum. */
hyena_status_t hyena_residual_norm_backward(const hyena_residual_norm_params_t* params, int64_t rows, const void* s,
                                            int64_t lds, const void* dy, const void* dsum, void* dx, void* dresidual,
                                            float* dw, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Static, NUL-terminated description of a status code. */
const char* hyena_status_string(hyena_status_t s);

#ifdef __cplusplus
}
#endif

#endif /* LIBHYENA_HYENA_H */
