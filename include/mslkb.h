/*
 * mslkb.h -- C ABI of libmslkb.so: the FP8 rowwise-scaled grouped GEMM
 * f8f8bf16_rowwise_grouped for NVIDIA GB300 (sm_103a), stacked and dynamic layouts.
 *
 * The operation (MSLK #471 "Back the FP8 rowwise grouped GEMM ops with FlyDSL on ROCm":
 * commit introducing the rowwise scaling scheme; PR Summary table) is, for each group g
 * and every row r that group owns,
 *
 *     out[r, n] = bf16_rne( scale_a[r] * scale_b[g, n] * sum_k A[r, k] * B[g, n, k] )
 *
 * with A and B in OCP FP8 E4M3 ("e4m3fn"), scale_a and scale_b in fp32, the sum held in
 * fp32 and never rounded before the scales are applied (once, after the K loop), and
 * the result rounded to bf16 with round-to-nearest-even.
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 * - Pointers named as device pointers must point to memory the current CUDA device
 *   can access (device or managed memory).  They are owned by the caller, are only
 *   read/written by work enqueued on `stream`, and are not retained after the call
 *   returns.  Every buffer is dense and row-major with the sizes given, but for the inputs
 *   that have a row stride (ld...) among their arguments; other strided views are not
 *   supported (the product's kernel addresses the output as one flat row-major buffer:
 *   MSLK #471, commit rejecting a strided output).
 * - `stream` is a cudaStream_t passed as void*; NULL means the legacy default stream.
 *   Calls are asynchronous: they enqueue work and return without synchronising.
 *   The first call on a device performs one-time set-up (device query, kernel attributes,
 *   driver entry point).  The first call on each stream (outside stream capture) also
 *   allocates that stream's workspace (2 x #SMs x 128 KB of fp32 partial sums for split
 *   tiles, plus counters, among them the tile claim counter of the CTA-pair plans; about
 *   40 MB on GB300), which lasts until mslkb_release_workspace or the end of the process;
 *   later calls on the stream allocate nothing and may be captured in a CUDA graph.  A
 *   call captured on a stream that has no workspace yet runs without splitting tiles and,
 *   on CTA pairs, takes its tiles in a fixed stride (same results within tolerance,
 *   possibly slower).
 *   Calls on one stream share its workspace in stream order; a captured graph keeps the
 *   workspace of the stream it was captured on, so two launches of such graphs, or one
 *   and a call on that stream, must not run at the same time.
 * - Sizes are int64_t.  Errors are reported by the return value; nothing is enqueued
 *   when a call returns anything but MSLKB_OK.  Argument checks happen before any CUDA
 *   call, so a bad argument is reported even where no GPU is present.
 * - The library is compiled for sm_103a only; any other device gives MSLKB_ERR_DEVICE.
 * - Errors found on the device (a wait that timed out, m_sizes that overran total_M)
 *   cannot be returned by an asynchronous call; they are OR-ed into a per-device status
 *   word read by mslkb_get_device_status().
 * - Host threads may call at the same time, on one stream or on several; the library's
 *   tables (device set-up, stream workspaces) are guarded by a lock.
 * - Every kernel launch is enqueued inside an NVTX push/pop range of the domain "mslkb"
 *   whose message is the kernel variant's name (mslkb_variant_name) and whose int64
 *   payload is the rows of A, so a profiler can select this library's launches (ncu:
 *   --nvtx --nvtx-include "mslkb@<variant name>/").  The operators around the product have
 *   one range per call, named as the call without "mslkb_", with its rows.  With no tool attached
 *   the range calls return at once; a launch captured in a CUDA graph replays without them.
 */
#ifndef MSLKB_H_
#define MSLKB_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MSLKB_API __attribute__((visibility("default")))
#else
#define MSLKB_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mslkb_status {
  MSLKB_OK = 0,
  MSLKB_ERR_NULL = 1,   /* a pointer needed for the given sizes is NULL */
  MSLKB_ERR_SHAPE = 2,  /* a size is negative, too large, or N is not a multiple of 8 */
  MSLKB_ERR_ALIGN = 3,  /* out is not 16-byte aligned (ragged layouts: or A / B not
                           16-byte aligned, or their row length not a multiple of 16) */
  MSLKB_ERR_DEVICE = 4, /* the current device is not sm_103 (GB300 / B300) */
  MSLKB_ERR_CUDA = 5,   /* a CUDA runtime or driver call failed; see mslkb_last_cuda_error */
  MSLKB_ERR_TOO_LARGE = 6, /* needs more scratch than the allocation-free entry point holds */
  MSLKB_ERR_DTYPE = 7,     /* an element type that the call does not take */
  MSLKB_ERR_WORKSPACE = 8  /* the workspace is NULL, misaligned or too small */
} mslkb_status;

/* Bits of the device status word (mslkb_get_device_status). */
#define MSLKB_DEV_TIMEOUT 0x1u        /* a pipeline wait in the kernel gave up (~1 s)  */
#define MSLKB_DEV_MSIZES_CLAMPED 0x2u /* m_sizes had a negative entry or summed past total_M */
#define MSLKB_DEV_BAD_SLICE 0x4u      /* ragged K: a slice bound not a multiple of 16 */
#define MSLKB_DEV_BOUNDS 0x8u         /* checked build (libmslkb_checked.so) only: a kernel
                                         index fell outside the buffers of the call; that
                                         access was not made as asked.  Bits 16..23 then name
                                         the kinds of access: 16 group metadata, 17 TMA load
                                         K coordinate, 18 TMA load row / column / group
                                         coordinate, 19 TMA K coordinate not 16-byte aligned,
                                         20 scales, 21 direct output store, 22 TMA output
                                         store, 23 split-tile workspace */

/* Limits. */
#define MSLKB_MAX_GROUPS 1024         /* G (kernel keeps per-group tables in shared memory) */
#define MSLKB_MAX_DIM 2147483647LL    /* every size, and total_M * K, N * K, rows * N ... */

/*
 * Stacked layout (op f8f8bf16_rowwise_grouped_stacked; MSLK #471, PR Summary table:
 * "[G] int64 row counts", and the commits on the packed "sizes" layout and its tile
 * retire guard).
 *
 *   A        device, e4m3 codes [total_M, K]      rows of all groups packed along M
 *   B        device, e4m3 codes [G, N, K]         one [N, K] weight matrix per group
 *   scale_a  device, fp32 [total_M]               one scale per row of A
 *   scale_b  device, fp32 [G, N]                  one scale per (group, column)
 *   m_sizes  device, int64 [G]                    rows per group, in group order
 *   out      device, bf16 [total_M, N]            16-byte aligned
 *
 * Group g owns rows [off_g, off_g + m_g) with off_0 = 0, off_{g+1} = off_g + m_g.
 * Empty groups own no rows and cost no work.  Each m_g is clamped into
 * [0, total_M - off_g]; if any entry needed clamping, MSLKB_DEV_MSIZES_CLAMPED is set in
 * the device status word.  Rows of out past the last group are left untouched.
 * K = 0 writes +0.0 to every owned row (MSLK #471, commit zeroing an empty reduction).
 * Any K >= 0 is accepted: when K is a multiple of 16 and A and B are 16-byte aligned
 * the tiles are fetched by TMA; otherwise a narrower asynchronous copy path is used,
 * with zero fill past K (MSLK #471, commit on the K tail).
 * N must be a multiple of 8, the width of one 16-byte bf16 store (MSLK #471, commits on
 * the N tail and on predicating a store on its last column).
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_rowwise_grouped_stacked(
    const void *A, const void *B, const float *scale_a, const float *scale_b,
    const int64_t *m_sizes, void *out, int64_t total_M, int64_t G, int64_t N, int64_t K,
    void *stream);

/*
 * Dynamic (padded) layout (op f8f8bf16_rowwise_grouped_dynamic; MSLK #471, PR Summary
 * table: "[G, M, K] slabs, runtime valid-row count", commit adding the padded layout and
 * commit adding its test: padding rows asserted zero).
 *
 *   A                   device, e4m3 codes [G * expected_m, K]   one slab per group
 *   B                   device, e4m3 codes [G, N, K]
 *   scale_a             device, fp32 [G * expected_m]
 *   scale_b             device, fp32 [G, N]
 *   zero_start_index_M  device, int64 [G]      valid rows at the top of each slab
 *   out                 device, bf16 [G * expected_m, N], 16-byte aligned
 *
 * Group g owns slab rows [g*E, (g+1)*E) with E = expected_m; the first
 * v_g = min(max(zero_start_index_M[g], 0), E) rows are computed and every other row of
 * the slab is written +0.0, whatever A and scale_a hold there (the zeroed-output
 * contract, folded into the kernel so that every output byte is written once).
 * K and N rules as for the stacked layout.
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_rowwise_grouped_dynamic(
    const void *A, const void *B, const float *scale_a, const float *scale_b,
    const int64_t *zero_start_index_M, void *out, int64_t G, int64_t expected_m,
    int64_t N, int64_t K, void *stream);

/*
 * Offsets layout (2D-3D, the torch-native grouped-mm addressing; MSLK #471, commits
 * decoding group boundaries from an int32 inclusive prefix sum and binding the `_mm` op's
 * 2D-3D rank combination).  As the stacked call, but the groups are given as
 *
 *   offsets  device, int32 [G]   inclusive prefix: group g owns rows
 *                                [offsets[g-1], offsets[g]) with offsets[-1] = 0
 *
 * A row count is the step between successive offsets; a negative step owns no rows and
 * steps past total_M are clamped (both set MSLKB_DEV_MSIZES_CLAMPED), as for m_sizes.
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_rowwise_grouped_offsets(
    const void *A, const void *B, const float *scale_a, const float *scale_b,
    const int32_t *offsets, void *out, int64_t total_M, int64_t G, int64_t N, int64_t K,
    void *stream);

/*
 * Batched layout (3D-3D; MSLK #471, commit adding the layout whose groups all carry their
 * full complement of rows, and the one eliding its retire guard).  Every group owns a full
 * slab of M rows and no metadata is read:
 *
 *   A        device, e4m3 codes [G, M, K]
 *   B        device, e4m3 codes [G, N, K]
 *   scale_a  device, fp32 [G, M]
 *   scale_b  device, fp32 [G, N]
 *   out      device, bf16 [G, M, N], 16-byte aligned
 *
 * M need not divide the tile height: rows past a slab are never written (the next slab's
 * rows belong to the next group).  K and N rules as for the stacked layout.
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_rowwise_grouped_batched(
    const void *A, const void *B, const float *scale_a, const float *scale_b, void *out,
    int64_t G, int64_t M, int64_t N, int64_t K, void *stream);

/*
 * Ragged-N layout (3D-2D; MSLK #471, commit adding the form whose weights are one
 * [total_N, K] matrix that the groups partition by row, results packed side by side).
 * Group g owns the output columns [offsets[g-1], offsets[g]) (offsets[-1] = 0):
 *
 *   out[m, n] = bf16_rne((acc * scale_a[g, m]) * scale_b[n]),
 *   acc = sum_k A[g, m, k] * B[n, k]                       for every n of group g
 *
 *   A        device, e4m3 codes [G, M, K] (one slab of M rows per group), 16-byte aligned
 *   B        device, e4m3 codes [total_N, K], 16-byte aligned
 *   scale_a  device, fp32 [G, M]
 *   scale_b  device, fp32 [total_N]
 *   offsets  device, int32 [G]   inclusive prefix over the columns
 *   out      device, bf16 [M, total_N], 16-byte aligned; columns past offsets[G-1] are
 *            not written
 *
 * K must be a multiple of 16 (TMA rows) and total_N of 8; a group's column count may be
 * anything (its last columns are stored one by one).  Column counts follow the offsets
 * rules of mslkb_f8f8bf16_rowwise_grouped_offsets (clamped at total_N, status bit set).
 * M = 0, G = 0 or total_N = 0: nothing to do.  K = 0: the owned columns are +0.0.
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_rowwise_grouped_n_offsets(
    const void *A, const void *B, const float *scale_a, const float *scale_b,
    const int32_t *offsets, void *out, int64_t G, int64_t M, int64_t total_N, int64_t K,
    void *stream);

/*
 * Ragged-K layout (2D-2D; MSLK #471, commit adding the layout whose groups slice K).
 * Group g contracts over k in [offsets[g-1], offsets[g]) (offsets[-1] = 0) and writes a
 * whole [M, N] slab:
 *
 *   out[g, m, n] = bf16_rne((acc * scale_a[g, m]) * scale_b[g, n]),
 *   acc = sum over the slice of A[m, k] * B[n, k]
 *
 *   A        device, e4m3 codes [M, total_K], 16-byte aligned
 *   B        device, e4m3 codes [N, total_K], 16-byte aligned
 *   scale_a  device, fp32 [G, M]
 *   scale_b  device, fp32 [G, N]
 *   offsets  device, int32 [G]   inclusive prefix over K
 *   out      device, bf16 [G, M, N], 16-byte aligned; every element is written
 *
 * total_K must be a multiple of 16, N of 8, and every slice must start and end on a
 * multiple of 16: a group whose slice does not is not computed -- its slab is written
 * +0.0 and MSLKB_DEV_BAD_SLICE is set.  An empty slice gives +0.0 (the empty sum).
 * Slice bounds are clamped into [0, total_K] as row counts are for the offsets layout.
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_rowwise_grouped_k_offsets(
    const void *A, const void *B, const float *scale_a, const float *scale_b,
    const int32_t *offsets, void *out, int64_t G, int64_t M, int64_t N, int64_t total_K,
    void *stream);

/*
 * Block-scaled (groupwise) stacked layout (MSLK #471, commit introducing the rowwise
 * scheme beside the block scheme the grouped kernel already had: a scale per scale block,
 * applied to each block's partial sum inside the K loop; K and N must cover whole scale
 * blocks).  Scale blocks of 128 along K and N:
 *
 *   out[r, n] = bf16_rne( sum_kb scale_a[r, kb] * scale_b[g, n / 128, kb] * S_kb ),
 *   S_kb = sum over k in [128 kb, 128 kb + 128) of A[r, k] * B[g, n, k]
 *
 *   A, B, m_sizes, out  as for mslkb_f8f8bf16_rowwise_grouped_stacked
 *   scale_a  device, fp32 [total_M, K / 128]
 *   scale_b  device, fp32 [G, N / 128, K / 128]
 *
 * K and N must be multiples of 128 (MSLKB_ERR_SHAPE otherwise); A and B 16-byte aligned
 * (MSLKB_ERR_ALIGN).  Each K block's partial sum is scaled in fp32 on its way from the
 * tensor core into the fp32 accumulator.
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_groupwise_grouped_stacked(
    const void *A, const void *B, const float *scale_a, const float *scale_b,
    const int64_t *m_sizes, void *out, int64_t total_M, int64_t G, int64_t N, int64_t K,
    void *stream);

/*
 * Block-scaled (groupwise) dynamic layout (MSLK #471: the block scheme of the commit
 * introducing the rowwise scheme -- "a compile-time blockscale flag" over the grouped
 * kernel's layouts -- on the padded layout of the PR Summary table and its commit; the
 * padded layout's per-group slab addressing is what a [G, scale_k, M] scale tensor needs).
 * Scale blocks of 128 along K and N:
 *
 *   A                   device, e4m3 codes [G * expected_m, K]   one slab per group
 *   B                   device, e4m3 codes [G, N, K]
 *   scale_a             device, fp32 [G * expected_m, K / 128]   per slab row and K block
 *   scale_b             device, fp32 [G, N / 128, K / 128]
 *   zero_start_index_M  device, int64 [G]      valid rows at the top of each slab
 *   out                 device, bf16 [G * expected_m, N], 16-byte aligned
 *
 *   out[r, n] = bf16_rne( sum_kb scale_a[r, kb] * scale_b[g, n / 128, kb] * S_kb )
 *
 * for the first v_g = min(max(zero_start_index_M[g], 0), E) rows of slab g, +0.0 for the
 * rest of the slab whatever A and scale_a hold there.  K and N must be multiples of 128
 * (MSLKB_ERR_SHAPE otherwise); A and B 16-byte aligned (MSLKB_ERR_ALIGN).
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_groupwise_grouped_dynamic(
    const void *A, const void *B, const float *scale_a, const float *scale_b,
    const int64_t *zero_start_index_M, void *out, int64_t G, int64_t expected_m,
    int64_t N, int64_t K, void *stream);

/*
 * Block-scaled (groupwise) batched layout: the block scaling above on the batched layout
 * (MSLK #471, commit adding the layout whose groups all carry their full complement of
 * rows): every group owns a full slab of M rows and no metadata is read.
 *
 *   A        device, e4m3 codes [G, M, K]
 *   B        device, e4m3 codes [G, N, K]
 *   scale_a  device, fp32 [G, M, K / 128]
 *   scale_b  device, fp32 [G, N / 128, K / 128]
 *   out      device, bf16 [G, M, N], 16-byte aligned
 */
MSLKB_API mslkb_status mslkb_f8f8bf16_groupwise_grouped_batched(
    const void *A, const void *B, const float *scale_a, const float *scale_b, void *out,
    int64_t G, int64_t M, int64_t N, int64_t K, void *stream);

/*
 * Allocation-free stacked call (no counterpart on the pages: an addition of this library).
 *
 * For callers that cannot allocate device memory when they call: plug-ins whose host
 * framework owns every device allocation (and gives a library none of its own), and
 * serving loops that cannot take the device-wide synchronisation a cudaMalloc can cause.
 * Same arguments, layout, results and errors as mslkb_f8f8bf16_rowwise_grouped_stacked;
 * the caller still provides inputs and output.  It calls no cudaMalloc, cudaFree or other
 * allocating routine.
 *
 * Its split-tile scratch (fp32 partial sums and arrival counters) is a static device
 * array of MSLKB_NOALLOC_SCRATCH_BYTES (8 MiB) that every GPU loading the library holds
 * until the process exits.  The plans that split tiles by default (swap-AB tiles, up to
 * 32 rows per group on average, e.g. MoE decode) need at most 2 x #SMs x 16 KB of it; a
 * plan that needs more -- 128-row activation tiles split under mslkb_set_split_k(2), or a
 * device with very many SMs -- returns MSLKB_ERR_TOO_LARGE and launches nothing.  CTA-pair
 * plans take their tiles in a fixed stride here (no claim counter).
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress,
 * once per device, with that device current).  Each call clears the counters it uses on
 * `stream` (cudaMemsetAsync) before its kernel.  All calls share the one array, which
 * keeps the last call's contents: calls that overlap on the GPU (different streams, say)
 * race and must be serialised by the caller.
 */
#define MSLKB_NOALLOC_SCRATCH_BYTES (8u << 20)
MSLKB_API mslkb_status mslkb_f8f8bf16_rowwise_grouped_stacked_noalloc(
    const void *A, const void *B, const float *scale_a, const float *scale_b,
    const int64_t *m_sizes, void *out, int64_t total_M, int64_t G, int64_t N, int64_t K,
    void *stream);

/*
 * Operators around the grouped product in a mixture-of-experts block (additions of this
 * library).  They make the product's operands and use its results:
 *
 *   add_rms_norm_quant -> (router's logits) -> route_experts -> moe_dispatch
 *     -> grouped gate/up product -> swiglu_quant -> grouped down product -> moe_combine
 *
 * Conventions beside those above: `dtype` is the element type of the 16- or 32-bit float
 * tensors of a call (MSLKB_BF16 / FP16 / FP32; MSLKB_ERR_DTYPE otherwise).  Sums, norms and
 * softmax statistics are fp32; every output is rounded once, to nearest even.  Any base
 * alignment that suits the element type is accepted; 16-byte aligned rows take the wide
 * path.  Inputs named with an `ld` argument may be slices of wider rows (ld elements from
 * row to row, ld >= the row's length); everything else is dense.  An output may be the same
 * buffer as an input only where that is said.  Nothing is allocated: the one call that
 * needs scratch takes it as `workspace` (16-byte aligned, contents need not be initialised,
 * not shared by calls that may run at the same time) of at least the bytes that its
 * *_workspace_bytes function returns.  Sums are made in a fixed order, which may depend on the
 * sizes, row strides and alignment of a call: equal inputs in equal layouts give equal bits.
 *
 * e4m3 outputs: one scale per row (groupwise = 0) or per 128 columns (groupwise = 1; the
 * row length must be a multiple of 128).  scale = amax / 448 over the row or block and
 * code = e4m3_rne(value / scale); where amax < 2^-80 the codes are 0 and the scale 1.  For
 * rows of length 0 nothing is written (the torch forms fill in scale 1 and eps^(-1/2)).  A
 * NaN, or an infinity that the formula makes NaN, gives its row or block a NaN scale.
 */
typedef enum mslkb_dtype { MSLKB_BF16 = 0, MSLKB_FP16 = 1, MSLKB_FP32 = 2 } mslkb_dtype;

#define MSLKB_MAX_HIDDEN 32768 /* longest row of the norm and SwiGLU calls */
#define MSLKB_MAX_TOPK 32      /* experts per token */
#define MSLKB_MAX_EXPERTS 1024 /* experts of the routing and dispatch calls */

/*
 * Residual addition, root-mean-square norm and quantisation of T rows of H elements:
 *
 *   h = x + residual (residual NULL: h = x),   rstd = (mean(h^2) + eps)^(-1/2),
 *   y = h * rstd * weight,                     q, scale = e4m3(y)
 *
 *   x, residual   device, dtype [T, H], rows ldx / ldr elements apart
 *   weight        device, [H], dtype, or fp32 if weight_fp32 is not 0
 *   q             device, e4m3 [T, H];  scale  device, fp32 [T] or [T, H / 128]
 *   residual_out  device, dtype [T, H]: h; NULL: not written.  May be residual itself
 *                 (rows H elements apart)
 *   y             device, dtype [T, H], for readers of the unquantised norm; NULL: none
 *   rstd          device, fp32 [T], for the gradient; NULL: none
 *
 * The norm is that of the fp32 sum, before residual_out's rounding.  1e-12 <= eps < 1.
 */
MSLKB_API mslkb_status mslkb_add_rms_norm_quant(
    const void *x, const void *residual, const void *weight, void *q, float *scale,
    void *residual_out, void *y, float *rstd, int64_t T, int64_t H, int64_t ldx, int64_t ldr,
    double eps, int32_t dtype, int32_t weight_fp32, int32_t groupwise, void *stream);

/*
 * Gradient of the norm (the quantisation passes the gradient through):
 *
 *   xhat = h * rstd,  g = dy * weight,
 *   dx = rstd * (g - xhat * mean(g * xhat)) + dresidual,   dweight = sum over rows of dy * xhat
 *
 * dx is the gradient of x and of residual alike; dresidual is the gradient that arrives on
 * residual_out (NULL: none).  dy, h, dresidual, dx are dense dtype [T, H] (dx may be dy or
 * dresidual), rstd fp32 [T], dweight fp32 [H].
 */
MSLKB_API int64_t mslkb_add_rms_norm_quant_backward_workspace_bytes(int64_t T, int64_t H);
MSLKB_API mslkb_status mslkb_add_rms_norm_quant_backward(
    const void *dy, const void *h, const void *weight, const float *rstd, const void *dresidual,
    void *dx, float *dweight, void *workspace, int64_t workspace_bytes, int64_t T, int64_t H,
    int32_t dtype, int32_t weight_fp32, void *stream);

/*
 * Each token's experts and weights from the router's logits:
 *
 *   score  = softmax(logits) or 1 / (1 + exp(-logits))       (MSLKB_SOFTMAX, MSLKB_SIGMOID)
 *   choice = score + bias                                    (bias fp32 [E], or NULL)
 *
 * The E experts form num_groups equal groups (1: none).  A group is worth the sum of its
 * group_top (1 or 2) best choices; the experts of the topk_groups best groups stay, and the
 * top_k best choices among them are taken, best first, the lowest index first among equals.
 * (Softmax without bias and with group_top = 1 orders by the logits themselves.)
 *
 *   ids      device, int32 [T, top_k]
 *   weights  device, fp32 [T, top_k]: scale * score, with renormalize scale * score / (sum of
 *            the taken scores, + 1e-20 for the sigmoid)
 *
 * An expert whose logit is -infinity (or whose choice is) is masked: it is never taken, and
 * a token with fewer than top_k experts left gets id -1 and weight 0 in the rest.  A NaN
 * choice counts as the largest; a NaN logit gives its token NaN weights (a NaN bias does not: it
 * is not in the weights).  logits: dtype [T, E], rows ld apart.
 */
#define MSLKB_SOFTMAX 0
#define MSLKB_SIGMOID 1
MSLKB_API mslkb_status mslkb_route_experts(
    const void *logits, const float *bias, int32_t *ids, float *weights, int64_t T, int64_t E,
    int64_t ld, int64_t top_k, int32_t score, int64_t num_groups, int64_t topk_groups,
    int32_t group_top, int32_t renormalize, double scale, int32_t dtype, void *stream);

/*
 * Gradient of the routing weights for the choice that was made (ids; an id outside [0, E)
 * has none): dlogits dtype [T, E], every element written, dense.  The choice itself and the
 * bias have no gradient.
 */
MSLKB_API mslkb_status mslkb_route_experts_backward(
    const float *dweights, const void *logits, const int32_t *ids, void *dlogits, int64_t T,
    int64_t E, int64_t ld, int64_t top_k, int32_t score, int32_t renormalize, double scale,
    int32_t dtype, void *stream);

/*
 * Packs the tokens' rows by expert into the stacked layout.  The choices (t, j) with
 * 0 <= ids[t, j] < E are ordered by expert, then by t * top_k + j; choice number r becomes
 * row r of x_out.  Choices with another id (a masked slot, an expert of another device) are
 * left out, and rows past the last choice are not written.
 *
 *   x           device, [T, row_bytes] bytes (e4m3 codes, or any other row); rows dense
 *   x_scale     device, fp32 [T, scale_cols]; NULL with scale_cols = 0
 *   ids         device, int32 [T, top_k]
 *   x_out       device, [T * top_k, row_bytes];  scale_out  fp32 [T * top_k, scale_cols]
 *   m_sizes     device, int64 [E]: rows per expert, as the stacked products take them
 *   dest        device, int32 [T, top_k]: the choice's row, -1 if left out
 *
 * T * top_k is limited to MSLKB_MAX_DIM / 2, row_bytes and scale_cols to 2^30.
 */
MSLKB_API mslkb_status mslkb_moe_dispatch(
    const void *x, const float *x_scale, const int32_t *ids, void *x_out, float *scale_out,
    int64_t *m_sizes, int32_t *dest, int64_t T, int64_t top_k, int64_t E, int64_t row_bytes,
    int64_t scale_cols, void *stream);

/*
 * The weighted sum of a token's rows:
 *
 *   out[t] = sum over j of weights[t, j] * rows[dest[t, j]]
 *
 * rows dtype [R, H], dest int32 [T, top_k] (outside [0, R): the choice adds nothing and its
 * row is not read), weights fp32 [T, top_k] (NULL: ones, which makes this the gradient of
 * the dispatch), out dtype [T, H].
 */
MSLKB_API mslkb_status mslkb_moe_combine(const void *rows, const int32_t *dest,
                                         const float *weights, void *out, int64_t T,
                                         int64_t top_k, int64_t H, int64_t R, int32_t dtype,
                                         void *stream);

/*
 * Gradient of the combination: drows[dest[t, j]] = weights[t, j] * dout[t], dweights[t, j] =
 * the dot product of dout[t] and rows[dest[t, j]] (0 where the choice has no row).  Rows of
 * drows that no choice names are not written; two choices must not name one row.
 */
MSLKB_API mslkb_status mslkb_moe_combine_backward(
    const void *dout, const void *rows, const int32_t *dest, const float *weights, void *drows,
    float *dweights, int64_t T, int64_t top_k, int64_t H, int64_t R, int32_t dtype, void *stream);

/*
 * The experts' activation: x dtype [R, 2 * W], rows ldx apart, holds gate and up side by side;
 *
 *   a = gate * sigmoid(gate) * up,    q, scale = e4m3(a)     q [R, W], scale [R] or [R, W / 128]
 *
 * With saved not NULL the input is kept in 8 bits for the gradient: saved e4m3 [R, 2 * W] and
 * saved_scale fp32 [R, 2 * W / 128] (one scale per 128 columns; W a multiple of 128).
 */
MSLKB_API mslkb_status mslkb_swiglu_quant(
    const void *x, void *q, float *scale, void *saved, float *saved_scale, int64_t R, int64_t W,
    int64_t ldx, int32_t dtype, int32_t groupwise, void *stream);

/*
 * Gradient of the activation, dx dtype [R, 2 * W], from dy dtype [R, W] and the kept input:
 *
 *   dgate = dy * up * s * (1 + gate * (1 - s)),   dup = dy * gate * s,   s = sigmoid(gate)
 *
 * saved is the checkpoint with its scales, or the input itself (dtype [R, 2 * W], dense) with
 * saved_scale NULL.
 */
MSLKB_API mslkb_status mslkb_swiglu_quant_backward(const void *dy, const void *saved,
                                                   const float *saved_scale, void *dx, int64_t R,
                                                   int64_t W, int32_t dtype, void *stream);

/*
 * The products by expert in 16 bits (dtype MSLKB_BF16 or MSLKB_FP16; MSLKB_ERR_DTYPE
 * otherwise), for experts that are kept in 16 bits and for the backward pass.  The experts'
 * rows are packed as in the stacked layout: expert g owns m_sizes[g] rows after those of the
 * experts before it, clamped to [0, total_M] as there (MSLKB_DEV_MSIZES_CLAMPED).  Products are
 * exact, sums fp32: the tensor core's of at most 1024 terms (fp32 gradients: 512), which lose up to
 * 2^-23 of the sum for each 16 terms, and these added with rounding.
 * G is limited to MSLKB_MAX_GROUPS, every other size to 2^30, and total_M * N, total_M * K and
 * G * N * K to 2^40 (MSLKB_ERR_SHAPE; a workspace of 0 bytes).  Any size and alignment is
 * accepted; an operand whose rows do not start on 16 bytes, or are not spaced by multiples of 16
 * (its address, ldx, lddy or the matrices' row length), is first copied to rows that do, and a
 * contraction with few output tiles is split into parts whose sums are added in a fixed order.
 * Both take `workspace` (16-byte aligned, contents need not be initialised, not
 * shared by calls that may run at the same time) of at least the bytes that the call's
 * *_workspace_bytes function returns for the same arguments; where that is 0, NULL will do.
 *
 *   out[r, n] = sum over k of x[r, k] * w[g, n, k]      transposed = 0: w [G, N, K]
 *   out[r, n] = sum over k of x[r, k] * w[g, k, n]      transposed = 1: w [G, K, N]
 *
 * for every row r of expert g, rounded once.  The second form takes the forward product's
 * weights as they lie and gives its input's gradient (x is then the gradient of out).
 *
 *   x    device, dtype [total_M, K], rows ldx elements apart
 *   out  device, dtype [total_M, N]; rows past the last expert's are not written.  Must not lie
 *        over elements of x or w, or over m_sizes (MSLKB_ERR_SHAPE)
 *
 * K = 0 writes +0.0 to every owned row.
 */
MSLKB_API int64_t mslkb_grouped_mm_workspace_bytes(const void *x, const void *w, int64_t total_M,
                                                   int64_t G, int64_t N, int64_t K, int64_t ldx,
                                                   int32_t transposed);
MSLKB_API mslkb_status mslkb_grouped_mm(const void *x, const void *w, const int64_t *m_sizes,
                                        void *out, int64_t total_M, int64_t G, int64_t N,
                                        int64_t K, int64_t ldx, int32_t transposed, int32_t dtype,
                                        void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The gradient of each expert's matrix:
 *
 *   dw[g, n, k] = add[g, n, k] + sum over expert g's rows r of dy[r, n] * x[r, k]
 *
 *   dy   device, dtype [total_M, N], rows lddy apart;  x  device, dtype [total_M, K], rows ldx
 *        apart.  Rows past the last expert's are not used, whatever they hold
 *   add  device, [G, N, K] of dw's type: what was accumulated before; NULL: nothing.  May be dw
 *        itself, but must not overlap it otherwise (MSLKB_ERR_SHAPE)
 *   dw   device, [G, N, K], fp32 if dw_fp32 is not 0, else dtype; every element is written (an
 *        expert without rows gets add, or +0.0).  Must not lie over elements of dy or x, or over
 *        m_sizes (MSLKB_ERR_SHAPE)
 */
MSLKB_API int64_t mslkb_grouped_mm_weight_grad_workspace_bytes(const void *dy, const void *x,
                                                               int64_t total_M, int64_t G,
                                                               int64_t N, int64_t K, int64_t lddy,
                                                               int64_t ldx);
MSLKB_API mslkb_status mslkb_grouped_mm_weight_grad(
    const void *dy, const void *x, const int64_t *m_sizes, const void *add, void *dw,
    int64_t total_M, int64_t G, int64_t N, int64_t K, int64_t lddy, int64_t ldx, int32_t dtype,
    int32_t dw_fp32, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The norm of a list of gradients taken together, as one vector:
 *
 *   norm = (sum over all elements of g^2)^(1/2)    kind MSLKB_NORM_2
 *   norm = the largest |g|                         kind MSLKB_NORM_INF
 *
 *   grads    host array of `count` device pointers; tensor i has sizes[i] elements (0: none) of
 *            type dtypes[i] (MSLKB_BF16, MSLKB_FP16 or MSLKB_FP32, which may differ), dense, at
 *            any address that suits its type.  sizes and dtypes are host arrays.  The arrays may
 *            be freed when the call returns
 *   norm     device, fp32: a NaN among the elements makes it NaN, an infinity infinity; else it
 *            is infinite only past fp32's largest number (squares do not overflow)
 *   workspace, workspace_bytes: as for the norm's gradient above, of
 *            mslkb_grad_norm_workspace_bytes(count)
 */
#define MSLKB_NORM_2 0
#define MSLKB_NORM_INF 1
#define MSLKB_MAX_TENSORS 65536
MSLKB_API int64_t mslkb_grad_norm_workspace_bytes(int64_t count);
MSLKB_API mslkb_status mslkb_grad_norm(const void *const *grads, const int64_t *sizes,
                                       const int32_t *dtypes, int64_t count, int32_t kind,
                                       float *norm, void *workspace, int64_t workspace_bytes,
                                       void *stream);

/*
 * The gradients scaled so that their norm does not exceed max_norm:
 *
 *   outs[i] = grads[i] * scale,    scale = 1 where norm + eps <= max_norm, else
 *                                          max_norm / (norm + eps)
 *
 * each product rounded once to its tensor's type; norm is that of grads, as above, in fp32.  The
 * scale is NaN exactly if norm is; an infinite max_norm leaves gradients as they are even if norm
 * is infinite; a finite one scales them by 0 then (an infinite element becomes NaN).  outs[i] may
 * be grads[i] itself (left as it is where scale is 1); otherwise results, norm among them, must not
 * lie over each other or over gradients (MSLKB_ERR_SHAPE).  max_norm >= 0 (it may be infinite, and is if fp32
 * does not hold it), eps >= 0.
 */
MSLKB_API mslkb_status mslkb_clip_grad_norm(const void *const *grads, void *const *outs,
                                            const int64_t *sizes, const int32_t *dtypes,
                                            int64_t count, int32_t kind, double max_norm,
                                            double eps, float *norm, void *workspace,
                                            int64_t workspace_bytes, void *stream);

/* Static description of a status code.  Never NULL. */
MSLKB_API const char *mslkb_status_string(mslkb_status status);

/* The cudaError_t (or, for a failed tensor-map encode, the CUresult) behind the last
 * MSLKB_ERR_CUDA returned on this thread. */
MSLKB_API int mslkb_last_cuda_error(void);

/*
 * Reads the device status word of the current device and clears it.  Enqueued on
 * `stream` and then waits for that stream, so it orders after earlier calls on it.
 * flags: host pointer receiving the MSLKB_DEV_* bits.  When the word reports a timeout,
 * the split-tile arrival counters of every stream workspace on the device are cleared as
 * well (a kernel that gave up may have left them short), on `stream`: call it while no
 * other stream runs this library's kernels on the device.
 */
MSLKB_API mslkb_status mslkb_get_device_status(void *stream, uint32_t *flags);

/*
 * Kernel variants and the plan the host would choose.  Pure host code: no CUDA call.
 * layout: 0 = stacked (rows = total_M), 1 = dynamic (rows = expected_m per group),
 *         2 = ragged N (rows = M, N = total_N), 3 = ragged K (rows = M, K = total_K),
 *         4 = block-scaled stacked (rows = total_M), 5 = block-scaled dynamic or batched
 *         (rows = expected_m per group).
 * num_sms: streaming multiprocessors of the target device.
 * a_align / b_align: the byte alignment of the A and B base addresses (e.g. 256).
 */
typedef struct mslkb_plan_info {
  int32_t variant;      /* index into the variant table, see mslkb_variant_name */
  int32_t swap_ab;      /* 1: weights take the MMA M side and tokens the N side */
  int32_t tile_m;       /* activation rows per tile */
  int32_t tile_n;       /* weight rows (output columns) per tile */
  int32_t stages;       /* shared-memory pipeline depth */
  int32_t tma;          /* 1: TMA loads; 0: cp.async loader */
  int32_t copy_width;   /* bytes per asynchronous copy of the cp.async loader */
  int32_t grid;         /* persistent CTAs launched */
  int32_t threads;      /* threads per CTA */
  int32_t smem_bytes;   /* dynamic shared memory per CTA */
  int64_t tiles_bound;  /* host upper bound on output tiles */
  int32_t split_k;      /* 1: the last waves' tiles are split along K over all CTAs */
  int32_t reserved;
} mslkb_plan_info;

MSLKB_API mslkb_status mslkb_plan(int32_t layout, int64_t rows, int64_t G, int64_t N, int64_t K,
                        int32_t num_sms, int64_t a_align, int64_t b_align,
                        mslkb_plan_info *info);

/* Number of kernel variants and the name of one (NULL past the end). */
MSLKB_API int32_t mslkb_num_variants(void);
MSLKB_API const char *mslkb_variant_name(int32_t variant);

/*
 * Resources of one kernel variant on the current device: CTAs that fit on one SM (the
 * library needs 1) and registers per thread.  Makes CUDA calls (device query, kernel
 * attributes); the library runs the same check before a variant's first launch.
 */
MSLKB_API mslkb_status mslkb_variant_resources(int32_t variant, int32_t *blocks_per_sm,
                                               int32_t *regs_per_thread);

/*
 * Failure detection (an addition of this library; the pages have no counterpart).  Every
 * wait of the kernels' pipelines is bounded: a wait that runs past the limit (default
 * ~1 s) makes the kernel give up, record MSLKB_DEV_TIMEOUT in the device status word, let
 * its copies in flight land, free its tensor memory and return, so the context stays
 * usable.  mslkb_set_wait_timeout_us sets the limit for the following launches (0: the
 * default; otherwise at least 1000 us, else MSLKB_ERR_SHAPE).
 */
MSLKB_API mslkb_status mslkb_set_wait_timeout_us(int64_t us);

/*
 * Frees the split-tile workspace of `stream` on the current device (see the conventions
 * above), after waiting for the work already enqueued on `stream`.  The next call on that
 * stream allocates a new one.  A CUDA graph captured on the stream keeps the address of
 * the workspace it was captured with: destroy such graphs first.  A stream with no
 * workspace: nothing to do.  Other streams' workspaces are not touched.
 */
MSLKB_API mslkb_status mslkb_release_workspace(void *stream);

/* Number of stream workspaces the library holds on the current device. */
MSLKB_API int32_t mslkb_workspace_count(void);

/* Library version, as major * 10000 + minor * 100 + patch. */
MSLKB_API int32_t mslkb_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MSLKB_H_ */
