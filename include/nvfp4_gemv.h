/*
 * nvfp4_gemv.h: C ABI of the GB300 (sm_103a) NVFP4 block-scaled batched GEMV.
 *
 * The operation (kernelbot "nvfp4-gemv" submission 103289, `cute_kernel`:
 * each output accumulates a*sfa*b*sfb over K in FP32 and is stored with
 * `.to(Float16)`; submission 69953's docstring names the shapes):
 *
 *   c[m,l] = fp16( sum_{k<K} E2M1(a[m,k,l]) * E4M3(sfa[m,k/16,l])
 *                          * E2M1(b[k,l])   * E4M3(sfb[k/16,l]) )
 *
 * Element formats: E2M1 is FP4 (sign, 2 exponent bits, 1 mantissa bit; no
 * Inf/NaN); E4M3 is finite-only FP8 (0x7F/0xFF are NaN).  Two E2M1 codes are
 * packed per byte along K, the lower k in the low nibble (the pages' torch
 * tensors are `float4_e2m1fn_x2`, so "k is halved").  One E4M3 scale covers
 * 16 consecutive K elements (`sf_vec_size = 16`).
 *
 * Memory layouts (all row-major, batch L outermost; submission 103289's
 * `cute_jit_kernel` gives A the strides (k, 1, m*k) and c the strides
 * (1, 1, m)):
 *   a   : uint8 [L][M][K/2]          packed E2M1, row stride K/2 bytes
 *   b   : uint8 [L][K/2]             packed E2M1 (dense: no N padding)
 *   c   : fp16  [L][M]               output, written, never read
 *   sfa, sfb in one of two layouts, chosen by `sf_layout`:
 *     NVFP4_SF_PLAIN          sfa uint8 [L][M][K/16], sfb uint8 [L][K/16]
 *     NVFP4_SF_PERMUTED_128x4 the pre-permuted tensor [32, 4, rest_m, 4,
 *        rest_k, L] of submission 103289 (`permuted_to_blocked`), stored
 *        L-outermost in 128x4 atoms of 512 bytes: byte (m, kb) of batch l is
 *        at ((l*rest_m + m/128)*rest_k + kb/4)*512 + (m%32)*16
 *        + ((m/32)%4)*4 + kb%4, rest_m = ceil(rows/128), rest_k = ceil(K/64)
 *        (both sized with ceil_div as in submission 69953's
 *        `to_blocked_batch`; padding rows and, when K % 64 != 0, the padding
 *        blocks of the last atom column hold 0x00).
 *        For sfb, rows = 1 (row 0 of each atom is used).
 *        nvfp4_repack_scales() produces this layout from the plain one.
 *
 * Ownership and execution: every pointer is device memory owned by the
 * caller (or memory the device can address, such as mapped pinned host
 * memory).  No call allocates, frees, synchronizes or keeps per-call state
 * (the two wait diagnostics at the end, nvfp4_tensor_wait_timeouts and
 * nvfp4_selftest_bounded_wait, synchronize); all work is enqueued on
 * `stream` (NULL = the legacy default stream), so the compute calls may be
 * captured into CUDA graphs.  Kernels are launched with
 * programmatic stream serialization: they wait for the preceding work on the
 * stream before reading any input, so stream order is preserved.
 *
 * Errors: arguments are validated on the host before anything is launched,
 * and a failing call launches nothing unless it returns NVFP4_ERR_CUDA.
 */
#ifndef NVFP4_GEMV_H
#define NVFP4_GEMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t is a pointer to this opaque driver type. */
struct CUstream_st;

typedef enum {
  NVFP4_SF_PLAIN = 0,
  NVFP4_SF_PERMUTED_128x4 = 1
} nvfp4_sf_layout_t;

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_INVALID_VALUE = 1,     /* NULL pointer with non-empty data, negative size, bad enum */
  NVFP4_ERR_UNSUPPORTED_SHAPE = 2, /* K % 16 != 0, a size beyond the limits below, or a
                                      shape the selected kernel cannot run */
  NVFP4_ERR_MISALIGNED = 3,        /* pointer alignment rule broken (see each call) */
  NVFP4_ERR_CUDA = 4               /* a CUDA runtime call failed; see nvfp4_last_cuda_error() */
} nvfp4_status_t;

/*
 * Batched GEMV, c[m,l] as defined above.
 *
 *   a, b, sfa, sfb : inputs in the layouts above (sf_layout selects the scale layout)
 *   c              : output, fp16 [L][M]
 *   M, K, L        : rows, reduction length (elements), batch count
 *   sf_layout      : NVFP4_SF_PLAIN or NVFP4_SF_PERMUTED_128x4
 *   stream         : CUDA stream (cudaStream_t)
 *
 * Shapes: M, L >= 0 and K >= 0 with K % 16 == 0 (whole 16-element scale
 * blocks; the pages' kernels take K % 64 == 0, their K tile and scale atom
 * `mma_tiler_mnk = (128, 1, 64)`, and K % 64 != 0 runs on the blockwise
 * kernel).  M == 0 or L == 0 is a no-op
 * (pointers may be NULL).  K == 0 writes +0 to every c (a, b, sfa, sfb may be
 * NULL).  Limits: K <= 2^30, M*L < 2^40.
 * Alignment: a and b 16-byte aligned, sfa and sfb 32-byte aligned (the
 * pages' `assumed_align` of 16 and 32), c 2-byte aligned.  (A 16-byte
 * aligned a is never run on the direct kernel, whose 256-bit loads need 32.)
 * Accuracy: on the CUDA-core kernels each 16-element block's dot product is
 * exact and blocks are scaled and summed in FP32; the tensor-core kernel
 * (which nvfp4_gemv runs for large streams in either scale layout, see
 * nvfp4_gemv_plan) sums in FP32 in the MMA's own order.
 * c is rounded to nearest even (overflow gives +-Inf; a NaN scale gives NaN)
 * and stays within 1e-3 * sum|terms| + 1 fp16 ulp of the exact result.
 * Results are bitwise reproducible run to run.  The FP32 summation order
 * follows the launch schedule, which the library picks per shape and scale
 * layout; under one CUDA-core schedule (nvfp4_gemv_explicit) the two layouts
 * give identical bits.
 * Execution detail: before waiting for the preceding work on the stream, the
 * kernel may ask the L2 to prefetch lines of a (a hint that returns no data;
 * every input is read only after that work has completed).
 */
nvfp4_status_t nvfp4_gemv(const void* a, const void* b, const void* sfa, const void* sfb,
                          void* c, int64_t M, int64_t K, int64_t L, int sf_layout,
                          struct CUstream_st* stream);

/*
 * Output activation of nvfp4_gemv_ex and nvfp4_gemm_small_n, applied in fp32
 * to y = alpha * sum + bias before the fp16 rounding: c = fp16(act(y)).  The
 * pages list none; these are the usual MLP activations, with NaN in -> NaN out:
 *   NVFP4_ACT_NONE      act(y) = y
 *   NVFP4_ACT_RELU      act(y) = y > 0 ? y : +0
 *   NVFP4_ACT_SILU      act(y) = y / (1 + exp(-y))
 *   NVFP4_ACT_GELU_TANH act(y) = y/2 * (1 + tanh(sqrt(2/pi) * (y + 0.044715 y^3)))
 *   NVFP4_ACT_GELU_ERF  act(y) = y/2 * (1 + erf(y / sqrt(2)))
 * Accuracy: act is evaluated with CUDA's fp32 expf, tanhf and erff; |act'| <=
 * 1.13 for all five, so c stays within 1.13 * (1e-3 * |alpha| * sum|terms|) + 1
 * fp16 ulp of act applied to the exact value (plus the fp32 evaluation error,
 * a few fp32 ulps).
 */
typedef enum {
  NVFP4_ACT_NONE = 0,
  NVFP4_ACT_RELU = 1,
  NVFP4_ACT_SILU = 2,
  NVFP4_ACT_GELU_TANH = 3,
  NVFP4_ACT_GELU_ERF = 4
} nvfp4_activation_t;

/*
 * Options of nvfp4_gemv_ex.  Zero-initialised fields other than alpha give
 * the plain call; {1.0f, NULL, 0, 0, NVFP4_ACT_NONE} is exactly nvfp4_gemv.
 *
 *   alpha            : fp32 output scale: c = fp16(alpha * sum + bias).  A
 *                      global per-tensor scale of this kind is mentioned in a
 *                      removed docstring line of submission 69575; the pages
 *                      never apply one (alpha = 1).
 *   bias             : NULL, or fp16 [L][M] (row stride M) added after the
 *                      scaling; 2-byte aligned.  With a bias the scaling and the
 *                      addition are one fp32 fused multiply-add before the fp16
 *                      rounding.
 *   b_batch_stride   : bytes from batch l to batch l+1 of b; 0 = K/2 (dense).
 *                      Otherwise >= K/2 and a multiple of 16: b may be row 0 of
 *                      an N-padded [L][N][K/2] buffer such as the one
 *                      submission 103289's host code builds (stride N*K/2).
 *   sfb_batch_stride : bytes from batch l to batch l+1 of sfb; 0 = dense
 *                      (K/16 plain, ceil(K/64)*512 permuted).  Otherwise at least
 *                      that, and a multiple of 4 (plain) or 16 (permuted).
 *   activation       : nvfp4_activation_t, applied last (see above).
 * Violations: a stride below the dense size or an unknown activation ->
 * NVFP4_ERR_INVALID_VALUE; a stride or bias pointer off its alignment ->
 * NVFP4_ERR_MISALIGNED.
 */
typedef struct {
  float alpha;
  const void* bias;
  int64_t b_batch_stride;
  int64_t sfb_batch_stride;
  int32_t activation;
} nvfp4_gemv_options_t;

/*
 * nvfp4_gemv with options (NULL options = nvfp4_gemv).  Same arguments,
 * rules, schedule and accuracy contract; the tolerance scales with |alpha|.
 */
nvfp4_status_t nvfp4_gemv_ex(const void* a, const void* b, const void* sfa, const void* sfb,
                             void* c, int64_t M, int64_t K, int64_t L, int sf_layout,
                             const nvfp4_gemv_options_t* options, struct CUstream_st* stream);

/* The GEMV kernels (CUDA-core kernels 0 and 1 share their arithmetic). */
typedef enum {
  /* Warps load up to 8 rows' 32-byte K chunks straight into registers with
   * 256-bit loads, then compute.  Needs a 32-byte aligned a. */
  NVFP4_KERNEL_DIRECT = 0,
  /* Each lane copies its rows' chunks and scale words into a 3-slot
   * per-warp shared-memory ring with cp.async, so every warp keeps two tasks
   * in flight while it computes one.  The default for every K > 0; needs
   * k_split no larger than the K steps, ceil(K/64 / lanes_per_row). */
  NVFP4_KERNEL_PIPELINED = 1,
  /* The tensor cores' block-scaled MMA (tcgen05 kind::mxf4nvf4, 16-element
   * E4M3 blocks, M = 128 tiles, b padded to N = 16 with zero rows), fed by
   * TMA.  The 128x4 atom of the pre-permuted layout is the MMA's scale
   * layout; plain scales (K % 256 == 0, a sfb batch stride that is a
   * multiple of 16 bytes) arrive as 16 bytes per row and 256-element stage,
   * and the MMA warp writes them out as atoms in shared memory before the
   * MMAs (the same atoms, so the same bits as pre-permuted scales).
   * k_split = CTAs per cluster (1, 2, 4 or 8, at most ceil(K/256))
   * splitting each tile's K range, summed in cluster rank order through
   * distributed shared memory; ctas a multiple of k_split (the clusters are
   * persistent over the L*ceil(M/128) tiles); lanes_per_row = pipeline
   * stages per CTA (2 or 4: 4, 3 or 2 CTAs of 2 stages share an SM, 2 of 4).
   * The MMA sums in fp32 in an order of its own: c meets the same accuracy
   * contract, not the CUDA-core kernels' bits.  The MMA reads scale codes as
   * unsigned magnitudes; the kernel folds every negative sfa or sfb code into
   * the sign bits of the 16 elements it scales before the MMA, so signed,
   * subnormal and NaN codes give the E4M3 result.  nvfp4_gemv runs it with
   * M >= 1024 where it was measured faster than the pipelined kernel: at
   * least 512 MB of A with K <= 8192 (either layout; plain scales with
   * K % 256 == 0 and, through nvfp4_gemv_ex, a sfb batch stride that is a
   * multiple of 16), or, for pre-permuted scales, 128-row tiles
   * (L * ceil(M/128)) filling 80-100% of one wave of 2 CTAs per SM with
   * K >= 6144, or more tiles than that wave holds and at least 128 MB of A
   * (any K); nvfp4_gemm_small_n uses it for N >= 2. */
  NVFP4_KERNEL_TENSOR = 2,
  /* Tensor-core block dots with the scales applied on the CUDA cores: A is
   * streamed by TMA in one box per tile of up to 128 rows (rows handed out to
   * one CTA per SM in units of 8), 512-element K stages (256 when K % 256 !=
   * 0), a ring of lanes_per_row slots (2..32; 0 = the most that fit); the
   * block-scaled MMA runs with unit A scales and constant selector B scales
   * so that it writes each 16-element block's dot to its own accumulator
   * column, and the epilogue adds dot * sfa * sfb in fp32 from the signed
   * E4M3 codes, block by block in K order (bits independent of grid, ring
   * depth and scale layout).  k_split must be 1.  Plain scales need
   * K % 256 == 0.  Selected explicitly only: measured on GB300 it matches the
   * pipelined kernel on the largest streams and is slower on smaller ones. */
  NVFP4_KERNEL_BLOCKDOT = 3,
  /* CUDA cores, any K % 16 == 0: each warp takes a group of 4 rows, each lane
   * whole 16-element blocks (8 bytes of a row of A, one aligned load whatever
   * K % 64 is), b's block decoded once for the 4 rows, then a shuffle sum over
   * the lanes.  Block arithmetic as in kernels 0 and 1; the fp32 sums run in
   * an order fixed by K alone.  lanes_per_row must be 32 and k_split 1.
   * nvfp4_gemv runs it for K % 64 != 0; the other kernels need K % 64 == 0
   * (NVFP4_ERR_UNSUPPORTED_SHAPE otherwise). */
  NVFP4_KERNEL_BLOCKWISE = 4
} nvfp4_kernel_t;

/*
 * nvfp4_gemv with the kernel and launch schedule given instead of chosen
 * (for tuning and for testing every schedule; same arguments, rules and
 * results contract as nvfp4_gemv).  kernel: nvfp4_kernel_t;
 * lanes_per_row in {4, 8, 16, 32}: lanes sharing a row; k_split in
 * {1, 2, 4, 8}: warps splitting a row's K range; ctas in [1, 2^31): grid size.
 * The summation order, and so the last bits of c, depend on (kernel,
 * lanes_per_row, k_split); any valid schedule meets the accuracy contract.
 * Invalid schedule values give NVFP4_ERR_INVALID_VALUE.
 */
nvfp4_status_t nvfp4_gemv_explicit(const void* a, const void* b, const void* sfa,
                                   const void* sfb, void* c, int64_t M, int64_t K, int64_t L,
                                   int sf_layout, int kernel, int lanes_per_row, int k_split,
                                   int64_t ctas, struct CUstream_st* stream);

/*
 * Small-N NVFP4 GEMM (a decode batch of N <= 16 vectors per batch): for each
 * batch l, vector n < N and row m,
 *   c[l][n][m] = fp16(alpha * sum_k E2M1(a[m,k,l]) * E4M3(sfa[m,k/16,l])
 *                                   * E2M1(b[n,k,l]) * E4M3(sfb[n,k/16,l]) + bias[l][n][m]),
 * N GEMVs that share one pass over A.  (Submission 103289's
 * `cute_jit_kernel` gives b a stride of 128 padded columns, made for
 * torch._scaled_mm; here b has the N rows given.)
 * Layouts: a [L][M][K/2] as for nvfp4_gemv; b [L][N][K/2], row n of batch l
 * at b + l*b_batch_stride + n*K/2 (b_batch_stride 0 = N*K/2); scales
 * pre-permuted only: sfa as for nvfp4_gemv, sfb the permuted form of
 * [L][N][K/16] (one 128-row atom block per batch, rows 0..N-1:
 * nvfp4_repack_scales with rows = N), batch stride sfb_batch_stride
 * (0 = (K/64)*512); c fp16 [L][N][M]; bias fp16 [L][N][M] or NULL.
 * N = 1 is nvfp4_gemv_ex with permuted scales (kernel and schedule chosen as
 * nvfp4_gemv chooses them); N >= 2 runs the tensor-core kernel
 * (NVFP4_KERNEL_TENSOR), whose cost does not grow with N.  Shapes: M, L >= 0, 0 <= N <= 16 (N > 16: UNSUPPORTED_SHAPE),
 * K % 64 == 0 (K = 0 gives c = fp16(bias) or zeros).  Alignment: a and b
 * 16 bytes, sfa and sfb 32 bytes; c and bias 2 bytes; batch strides as for
 * nvfp4_gemv_ex.
 * Scales are signed here; nvfp4_gemm (below) reads them as magnitudes, and
 * says which of the two to call for up to 16 rows.
 */
nvfp4_status_t nvfp4_gemm_small_n(const void* a, const void* b, const void* sfa, const void* sfb,
                                  void* c, int64_t M, int64_t N, int64_t K, int64_t L,
                                  const nvfp4_gemv_options_t* options, struct CUstream_st* stream);

/*
 * nvfp4_gemm_small_n (N >= 1, always the tensor-core kernel, default options)
 * with its schedule given: stages (2 or 4) pipeline stages per CTA, k_split
 * (1, 2, 4 or 8, at most ceil(K/256); 1 when K = 0) CTAs per cluster
 * splitting each 128-row tile's K range, ctas in [1, 2^31) a multiple of
 * k_split.  Invalid values give NVFP4_ERR_INVALID_VALUE.
 */
nvfp4_status_t nvfp4_gemm_small_n_explicit(const void* a, const void* b, const void* sfa,
                                           const void* sfb, void* c, int64_t M, int64_t N,
                                           int64_t K, int64_t L, int stages, int k_split,
                                           int64_t ctas, struct CUstream_st* stream);

/*
 * The tensor-core schedule nvfp4_gemm_small_n uses for N >= 2 (computed for
 * any N in 1..16): stages per CTA, CTAs per cluster, grid size, and
 * optionally (resident_ctas non-NULL) the CTAs of that kernel resident at once
 * on the current device.  Queries the device (occupancy; cached per device).
 */
nvfp4_status_t nvfp4_gemm_small_n_plan(int64_t M, int64_t N, int64_t K, int64_t L,
                                       int* stages, int* k_split, int64_t* ctas,
                                       int* resident_ctas);

/*
 * Scale repack: plain [L][rows][K/16] E4M3 -> the 128x4-atom pre-permuted
 * layout above (submission 69953, `to_blocked_batch`; submission 69575,
 * `blocked_transform_kernel`).  A byte permutation, bit-exact; padding rows
 * rows..128*rest_m-1 of the last atom row, and blocks K/16..4*rest_k-1 of the
 * last atom column when K % 64 != 0, are written as 0x00.  dst must hold
 * nvfp4_permuted_scale_bytes(rows, K, L) bytes and must not overlap src.
 * Use rows = M for sfa and rows = 1 for sfb.
 * Shapes: rows, L >= 0, K % 16 == 0 (empty is a no-op).
 * Alignment: src 4-byte aligned; dst 16-byte aligned.  With K % 256 == 0 and a
 * 16-byte aligned src a shared-memory-free kernel runs; the result is the same.
 */
nvfp4_status_t nvfp4_repack_scales(const void* src, void* dst, int64_t rows, int64_t K,
                                   int64_t L, struct CUstream_st* stream);

/* Bytes of a permuted scale tensor: L * ceil(rows/128) * ceil(K/64) * 512.
 * Returns 0 for invalid arguments (negative sizes or K % 16 != 0). */
size_t nvfp4_permuted_scale_bytes(int64_t rows, int64_t K, int64_t L);

/* Static, human-readable name of a status code. */
const char* nvfp4_status_string(int status);

/* The cudaError_t of the most recent NVFP4_ERR_CUDA on the calling thread
 * (0 if none). */
int nvfp4_last_cuda_error(void);

/* Waits of the tensor-core kernels (the GEMV's, the block-dot kernel's, the
 * layer products' and attention's) that gave up: every wait of those kernels on
 * a pipeline barrier is bounded (2 s), and a wait that runs out is counted
 * here and makes its thread skip the rest of its work (the launch's c is
 * then not valid).  Synchronises the device; reset != 0 clears the count
 * after reading it.  Returns the count, or -1 on a CUDA error. */
int nvfp4_tensor_wait_timeouts(int reset);

/* Device self-test of that bounded wait (the one the tensor-core and block-dot
 * kernels use on their pipeline barriers), made so that a wait runs out
 * without hanging anything: one warp initialises two shared-memory barriers
 * for one arrival each, arrives on the first, then waits on phase 0 of each.
 * Expected: *completed = 1 (the first wait returned at once), *gave_up = 1 (the
 * second gave up: nothing arrives on it), *timeouts = 1 (the give-up was
 * counted) and *waited_ns about 2e9 (the wait limit, measured with the global
 * timer).  The self-test has its own counter (nvfp4_tensor_wait_timeouts is
 * not changed) and leaves the context usable.  Synchronises `stream`; takes
 * about 2 s.  NULL outputs give NVFP4_ERR_INVALID_VALUE, a CUDA failure
 * NVFP4_ERR_CUDA. */
nvfp4_status_t nvfp4_selftest_bounded_wait(int* completed, int* gave_up, int* timeouts,
                                           int64_t* waited_ns, struct CUstream_st* stream);

/*
 * Launch plan of nvfp4_gemv, computed on the host only (no GPU needed), for
 * inspection and tests.  kernel = -1 gives the plan nvfp4_gemv uses, an
 * nvfp4_kernel_t value that kernel's plan (NVFP4_ERR_UNSUPPORTED_SHAPE if it
 * cannot run the shape).  num_sms is the device's multiprocessor count and
 * ctas_per_sm the number of the CUDA-core kernel's CTAs resident per SM (pass
 * 0 to use the compiled-in default of 2).  nvfp4_gemv picks: the blockwise
 * kernel for K % 64 != 0; the direct kernel for K = 0 and for plain scales up
 * to 512 KB of A; the tensor-core kernel with M >= 1024 and either at least
 * 512 MB of A with K <= 8192 (plain scales: K % 256 == 0), or, for
 * pre-permuted scales, 80-100% of 2 * num_sms tiles of 128 rows with
 * K >= 6144 or more than 2 * num_sms such tiles with at least 128 MB of A;
 * the pipelined kernel otherwise.
 * For the tensor-core kernel the plan assumes 4 resident 2-stage CTAs (or 2
 * 4-stage ones) per SM (nvfp4_gemm_small_n_plan gives the schedule rule); for the block-dot kernel, one CTA per SM and up to
 * 227 KB of shared memory.
 */
typedef struct {
  int kernel;         /* nvfp4_kernel_t */
  int lanes_per_row;  /* lanes of a warp that share one row (32-byte K chunk
                         each); tensor-core kernel: pipeline stages per CTA;
                         block-dot kernel: ring slots; blockwise: 32 */
  int k_split;        /* warps of a CTA that split one row's K range;
                         tensor-core kernel: CTAs per cluster; block-dot: 1 */
  int rows_per_pass;  /* rows a warp reduces at once; tensor-core and
                         block-dot kernels: 128 (a tile); blockwise: rows a
                         CTA takes at once (8 warps x 4) */
  int threads_per_cta;
  int64_t ctas;       /* grid size */
  int64_t steps;      /* K chunks per lane per row, ceil(K/64 / lanes_per_row);
                         tensor-core kernel: 256-element K stages, ceil(K/256);
                         block-dot kernel: ceil(K/512) (ceil(K/256) when
                         K % 256 != 0); blockwise: ceil(K/16 / 32) */
} nvfp4_gemv_plan_t;

nvfp4_status_t nvfp4_gemv_plan(int64_t M, int64_t K, int64_t L, int sf_layout, int kernel,
                               int num_sms, int ctas_per_sm, nvfp4_gemv_plan_t* out);

/* ------------------------------------------------------------------------
 * Layer operators: what a program that serves a model calls around the
 * product.  Rows of activations are quantised on the GPU, multiplied with
 * quantised weights for any number of rows, and, in layers whose feed-forward
 * part is a set of experts, routed to the experts and summed back.
 *
 * The rules of the calls above hold: device pointers owned by the caller, no
 * allocation, no synchronisation, everything on `stream`, stream-capturable,
 * arguments validated before anything is launched.  Results are bitwise
 * reproducible run to run (no atomics on values).  There are no gradients: the
 * weights are 4-bit codes.
 *
 * Scales: these products read a scale code as an unsigned magnitude (bit 7 is
 * ignored; 0x7F and 0xFF are NaN), unlike the GEMV calls, which take signed
 * codes.  nvfp4_quantize never writes a code with bit 7 set.  Weights whose
 * scales have signs are made unsigned once with nvfp4_fold_scale_signs.
 * ------------------------------------------------------------------------ */

typedef enum {
  NVFP4_DTYPE_FP16 = 0,
  NVFP4_DTYPE_BF16 = 1,
  NVFP4_DTYPE_FP32 = 2
} nvfp4_dtype_t;

/*
 * Quantise rows to NVFP4.  With y = fp32(x * encode_scale), for each block of
 * 16 consecutive elements of a row:
 *   s    = E4M3(max|y| / 6)   to nearest even, at most 448
 *   code = E2M1(y / s)        to nearest even, at most 6 in magnitude
 * s = 0 gives zero codes; a block with an infinity or a NaN in y has the scale
 * code 0x7F (NaN) and zero codes.  x stands for code * s / encode_scale: a
 * product's alpha takes 1 / encode_scale.
 *   x       : [L][rows] rows of K elements of x_dtype (nvfp4_dtype_t), x_row_stride
 *             elements apart (0 = K); element aligned (16-byte aligned rows load faster)
 *   q       : uint8 [L][rows][K/2], 8-byte aligned
 *   sf      : uint8 scales in sf_layout, 4-byte aligned; the permuted layout's padding
 *             is written as 0x00
 *   row_map : NULL, or int32 [rows][copies] (then L = 1, copies <= 32): row r is
 *             written to the rows row_map[r][0..copies-1] of q and sf instead, which
 *             hold q_rows rows; entries outside [0, q_rows) are skipped, rows that no
 *             entry names are left as they are (their scales too), and two
 *             entries must not name one row.  copies and q_rows are ignored without it.
 * Shapes: K % 16 == 0; rows, K or L of 0 is a no-op.  encode_scale is finite and > 0.
 */
nvfp4_status_t nvfp4_quantize(const void* x, int x_dtype, int64_t x_row_stride, int64_t rows, int64_t K,
                              int64_t L, float encode_scale, void* q, void* sf, int sf_layout,
                              const int32_t* row_map, int copies, int64_t q_rows,
                              struct CUstream_st* stream);

/*
 * The values of quantised rows: x = x_dtype(fp32(E2M1 * E4M3) * scale), the product
 * of code and scale exact, signed scale codes accepted.  Arguments as for
 * nvfp4_quantize; q 8-byte aligned.
 */
nvfp4_status_t nvfp4_dequantize(const void* q, const void* sf, int sf_layout, int64_t rows, int64_t K,
                                int64_t L, float scale, void* x, int x_dtype, int64_t x_row_stride,
                                struct CUstream_st* stream);

/*
 * Make the scales of a quantised matrix unsigned, in place: every scale code with
 * bit 7 set has it cleared, and the sign bits of the 16 elements it scales are
 * flipped.  The values stay the same (NaN stays NaN).  a 8-byte aligned.
 */
nvfp4_status_t nvfp4_fold_scale_signs(void* a, void* sf, int sf_layout, int64_t rows, int64_t K, int64_t L,
                                      struct CUstream_st* stream);

/*
 * Options of nvfp4_gemm.  NULL = {1.0f, NULL, NVFP4_ACT_NONE, NVFP4_DTYPE_FP16, 0}.
 *   alpha        : fp32 output scale
 *   bias         : NULL, or fp32 [L][M], added after the scaling
 *   activation   : nvfp4_activation_t, applied last
 *   c_dtype      : nvfp4_dtype_t of c
 *   c_row_stride : elements from row n to n+1 of c; 0 = M
 */
typedef struct {
  float alpha;
  const float* bias;
  int32_t activation;
  int32_t c_dtype;
  int64_t c_row_stride;
} nvfp4_gemm_options_t;

/*
 * NVFP4 product for any number of rows: for each batch l, row n < N of b and row
 * m < M of a,
 *   c[l][n][m] = c_dtype(act(alpha * sum_k a[l][m][k] * b[l][n][k] + bias[l][m])),
 * a and b the values of their codes and (unsigned) scales.
 *   a : uint8 [L][M][K/2]; sfa its scales in the 128x4 layout
 *   b : uint8 [L][N][K/2]; sfb its scales in the 128x4 layout (per batch, ceil(N/128) atom rows)
 *   c : [L][N] rows of M elements, c_row_stride apart
 * Shapes: K % 32 == 0 (rows of 16-byte multiples; K = 0 gives act(bias)), any M and
 * N; an empty c is a no-op.  a, b, sfa, sfb 16-byte aligned; c element aligned.
 * Accuracy: fp32 sums in the tensor cores' order, one rounding to c_dtype.
 * Up to 16 rows, with nvfp4_gemm_small_n: that call for signed scales (this one ignores
 * their signs without a word; nvfp4_fold_scale_signs makes them unsigned), an fp16 bias per
 * row of b, and a single row (1.02 to 1.6 times as fast on five matrices of 7 to 132 MB, read
 * from memory); this one for 2 to 16 rows (1.1 to 1.9 times as fast on four of them, within
 * 4% on the largest), other types of c and bias, c's rows with gaps, and K % 64 == 32.
 */
nvfp4_status_t nvfp4_gemm(const void* a, const void* b, const void* sfa, const void* sfb, void* c,
                          int64_t M, int64_t N, int64_t K, int64_t L,
                          const nvfp4_gemm_options_t* options, struct CUstream_st* stream);

/*
 * The tile and K split that nvfp4_gemm uses (host only, no GPU needed) for a product
 * without an activation (with one, others may be faster), for inspection and tests:
 * tile_rows rows of b per tile (16, 32, 64 or 128 against 128 rows of a on one SM, 256
 * against 256 on a pair of SMs), and k_split CTAs of a cluster that share a tile's K
 * range (1, 2 or 4).  num_sms: the device's multiprocessors (>= 2).
 */
nvfp4_status_t nvfp4_gemm_plan(int64_t M, int64_t N, int64_t K, int64_t L, int num_sms, int* tile_rows,
                               int* k_split);

typedef enum {
  NVFP4_SCORE_SOFTMAX = 0, /* over all E experts */
  NVFP4_SCORE_SIGMOID = 1
} nvfp4_score_t;

/*
 * Options of nvfp4_route.  NULL = {NVFP4_SCORE_SOFTMAX, NULL, 1, 1, 1, 1.0f}.
 *   score        : nvfp4_score_t
 *   bias         : NULL, or fp32 [E]: added to the scores to choose, not to weigh
 *   groups       : the E experts are cut into this many equal runs (<= 32)
 *   top_groups   : runs that stay open, those with the largest sum of their two
 *                  largest score + bias (of one, if only one is not masked)
 *   renormalize  : weights are divided by their sum
 *   weight_scale : and then multiplied by this
 */
typedef struct {
  int32_t score;
  const float* bias;
  int32_t groups;
  int32_t top_groups;
  int32_t renormalize;
  float weight_scale;
} nvfp4_route_options_t;

/*
 * Choose top_k experts for each of T tokens.  logits: [T] rows of E values of dtype,
 * row_stride elements apart (0 = E).  Scores are computed in fp32; experts are
 * ranked by score + bias, or without a bias by the logit (the same order,
 * without the scores' rounding), ties to the lower index.
 *   ids     : int32 [T][top_k], best first
 *   weights : fp32 [T][top_k], the scores of the chosen
 * A logit that is -inf or NaN, or a bias that makes the rank so, masks the expert:
 * it is never chosen.  Where fewer than top_k are left, the remaining ids are -1 and
 * their weights 0.  Logits of +inf share the softmax evenly.
 * Limits: E <= 1024, top_k <= 32 and <= E, E % groups == 0.
 */
nvfp4_status_t nvfp4_route(const void* logits, int dtype, int64_t row_stride, int64_t T, int64_t E,
                           int top_k, const nvfp4_route_options_t* options, int32_t* ids, float* weights,
                           struct CUstream_st* stream);

/*
 * The experts' rows.  T tokens with top_k choices each are sorted by expert into a
 * buffer of row_capacity rows: an expert's choices, in the order of the tokens,
 * fill tiles of tile_rows rows, each tile starting on a row that is a multiple of
 * 128 (a scale atom).  The capacity, the tile and the size of the plan (what the sort
 * tells the products, opaque) follow from T, top_k and E alone.
 * Limits: E <= 1024, top_k <= 32 and <= E, T * top_k <= 2^24.
 */
typedef struct {
  int32_t tile_rows;
  int64_t row_capacity;
  size_t plan_bytes;
} nvfp4_moe_shape_t;
nvfp4_status_t nvfp4_moe_shape(int64_t T, int64_t top_k, int64_t E, nvfp4_moe_shape_t* out);

/*
 * Sort the choices ids int32 [T][top_k]; an id outside [0, E) is no choice.
 *   rows   : int32 [T][top_k], the row of each choice, -1 for none
 *   counts : int32 [E], choices per expert
 *   starts : int32 [E], first row of each expert
 *   plan   : plan_bytes bytes, 16-byte aligned
 */
nvfp4_status_t nvfp4_moe_sort(const int32_t* ids, int64_t T, int64_t top_k, int64_t E, int32_t* rows,
                              int32_t* counts, int32_t* starts, void* plan, struct CUstream_st* stream);

/*
 * Products of the experts' rows, for a plan of the same T, top_k and E.
 *   a, sfa : weights uint8 [E][M][K/2] and their 128x4 scales
 *   b, sfb : rows uint8 [row_capacity][K/2] and their 128x4 scales (nvfp4_quantize with
 *            row_map = rows, or the gated product)
 *   alpha  : fp32 [E] on the device, or NULL (1)
 * nvfp4_moe_gemm: c[row][m] = c_dtype(act(alpha[e] * sum_k a[e][m][k] * b[row][k])).
 * nvfp4_moe_gated_gemm: a has M = 2F rows per expert, row 2f the gate and row 2f+1 the
 * input of output f; h = act(alpha gate) * (alpha input) in fp32 is quantised with
 * encode_scale as nvfp4_quantize does: q uint8 [row_capacity][F/2], sf 128x4 scales
 * (both 16-byte aligned).
 * Rows of the buffers that hold no choice are not read into a result; what the products
 * leave in such rows of c, q and sf is not defined.
 * Shapes: K % 32 == 0, K > 0; F % 32 == 0.  Alignment as for nvfp4_gemm.
 */
nvfp4_status_t nvfp4_moe_gemm(const void* a, const void* sfa, const void* b, const void* sfb,
                              const void* plan, int64_t T, int64_t top_k, int64_t E, int64_t M, int64_t K,
                              const float* alpha, int activation, void* c, int c_dtype,
                              struct CUstream_st* stream);
nvfp4_status_t nvfp4_moe_gated_gemm(const void* a, const void* sfa, const void* b, const void* sfb,
                                    const void* plan, int64_t T, int64_t top_k, int64_t E, int64_t F,
                                    int64_t K, const float* alpha, int activation, float encode_scale,
                                    void* q, void* sf, struct CUstream_st* stream);

/*
 * out[t][m] = dtype(sum_j weights[t][j] * y[rows[t][j]][m]), fp32 sums in the order
 * of j, choices with row -1 left out.  y: [row_capacity][M], of dtype or fp32 (y_dtype);
 * out: [T][M], dtype fp16 or bf16; both 16-byte aligned; M % 8 == 0.
 */
nvfp4_status_t nvfp4_moe_combine(const void* y, int y_dtype, const int32_t* rows, const float* weights,
                                 int64_t T, int64_t top_k, int64_t M, void* out, int dtype,
                                 struct CUstream_st* stream);

/*
 * The whole routed feed-forward layer: sort, quantise, gated product, product, sum.
 *   x       : [T] rows of D fp16 or bf16 elements, x_row_stride apart (0 = D)
 *   ids, weights : [T][top_k], as nvfp4_route writes them
 *   w1, sf1 : [E][2F][D/2], gate and input rows interleaved (see above), 128x4 scales
 *   w2, sf2 : [E][D][F/2], 128x4 scales
 *   out     : [T][D], the type of x, 16-byte aligned
 * Options (NULL = {NULL, NULL, 1, 1, NVFP4_ACT_SILU, 0}): alpha1 and alpha2 scale the two
 * products per expert (fp32 [E] on the device; NULL = 1), encode_x and encode_h the
 * values before they are quantised, activation is the gate's.  An expert's output is
 * fp32 before the weighted sum; with round_outputs 1 (0 and 1 are allowed) it is rounded
 * to the type of x first, which moves fewer bytes in large batches, and costs a second
 * rounding and, in fp16, the range above 65504.
 * workspace: nvfp4_moe_ffn_workspace_bytes bytes (0 for sizes that are not supported),
 * 256-byte aligned; its contents need not be kept.  Shapes: D and F > 0, multiples of 32.
 */
typedef struct {
  const float* alpha1;
  const float* alpha2;
  float encode_x;
  float encode_h;
  int32_t activation;
  int32_t round_outputs;
} nvfp4_moe_options_t;
size_t nvfp4_moe_ffn_workspace_bytes(int64_t T, int64_t top_k, int64_t E, int64_t D, int64_t F);
nvfp4_status_t nvfp4_moe_ffn(const void* x, int dtype, int64_t x_row_stride, const int32_t* ids,
                             const float* weights, const void* w1, const void* sf1, const void* w2,
                             const void* sf2, int64_t T, int64_t top_k, int64_t E, int64_t D, int64_t F,
                             const nvfp4_moe_options_t* options, void* out, void* workspace,
                             size_t workspace_bytes, struct CUstream_st* stream);

/* ------------------------------------------------------------------------
 * Attention on a 4-bit cache: rotary positions, keys and values quantised into pages as
 * they are written, and attention that reads them there.  The rules of the layer operators
 * hold (results bitwise reproducible, nothing allocated, stream-capturable, no gradients but
 * the rotation's own).  examples/attention_layer.py runs them together.
 * ------------------------------------------------------------------------ */

/*
 * Rotary positions.  Pair i of a head, the elements (2i, 2i+1) interleaved or (i, pairs + i)
 * in halves, is turned by positions[t] * f_i:
 *   (a, b) -> factor * (a cos - b sin, b cos + a sin)
 * in fp32, rounded once; the elements past 2 * pairs are copied.
 *   x, y      : [T][H][D] of dtype (nvfp4_dtype_t), element aligned (16-byte aligned rows go
 *               faster).  y may be x with the same strides, and must not overlap it otherwise
 *   positions : int32 [T], of either sign
 *   table     : int64 [pairs], f_i in 2^-64 turns per position (f / (2 pi) * 2^64 modulo 2^64):
 *               the angle is exact modulo a turn at any position
 * Options (NULL = {0, 0, 1, 0, 0, 0, 0}): interleaved 0 or 1; inverse 1 turns the other way
 * (the gradient of the rotation, from y's to x's); factor scales the turned elements (what
 * long contexts multiply their scores by, as its root); strides in elements, 0 = dense.
 * Limits: 1 <= pairs <= 512, 2 * pairs <= D <= 65536, H <= 65536, H * D < 2^31.
 */
typedef struct {
  int32_t interleaved;
  int32_t inverse;
  float factor;
  int64_t x_token_stride;
  int64_t x_head_stride;
  int64_t y_token_stride;
  int64_t y_head_stride;
} nvfp4_rope_options_t;
nvfp4_status_t nvfp4_rope(const void* x, int dtype, int64_t T, int64_t H, int64_t D, const int32_t* positions,
                          const int64_t* table, int64_t pairs, const nvfp4_rope_options_t* options, void* y,
                          struct CUstream_st* stream);

/*
 * The cache: uint8 [pages][heads][page_size/16][2][D/64][576], 16-byte aligned.  A granule of
 * 16 tokens holds K and then V, each as planes of 64 elements: 16 rows of 32 bytes of codes
 * (two a byte, low nibble first), then 16 rows of 4 scale bytes, quantised as nvfp4_quantize
 * does: blocks of 16 elements along the head.  Slot s is token s % page_size of page
 * s / page_size.  page_size is a multiple of 16, D 64, 128 or 256,
 * heads at most 65535, pages * heads * page_size * D at most 2^48 (bytes: 0 for other sizes).
 * Attention reads the scales as signed codes.
 */
size_t nvfp4_kv_cache_bytes(int64_t pages, int64_t heads, int64_t D, int64_t page_size);

/*
 * Rows of keys and values: [T][heads][D] each, strides in elements (0 = dense), and the
 * encode scales (fp32 [heads] on the device, finite and > 0; NULL = 1).
 */
typedef struct {
  void* k;
  void* v;
  const float* encode_k;
  const float* encode_v;
  int64_t k_token_stride;
  int64_t k_head_stride;
  int64_t v_token_stride;
  int64_t v_head_stride;
} nvfp4_kv_rows_t;

/*
 * Write: the rows of token t, times their head's encode scale, are quantised into slot
 * slots[t] (int64 [T]).  Slots outside the cache are skipped (a negative one marks a padding
 * row); other slots' bytes stay as they are.  No slot may be named twice in a call.
 * Rows are element aligned (16- or 32-byte aligned rows load faster).
 */
nvfp4_status_t nvfp4_kv_write(const nvfp4_kv_rows_t* rows, int dtype, int64_t T, int64_t heads, int64_t D,
                              const int64_t* slots, void* cache, int64_t pages, int64_t page_size,
                              struct CUstream_st* stream);

/*
 * Read back: k and v (either may be NULL) get dtype(fp32(code * scale) * fp32(1 / encode)) of
 * slot slots[t], zeros for a slot outside the cache.
 */
nvfp4_status_t nvfp4_kv_read(const nvfp4_kv_rows_t* rows, int dtype, int64_t T, int64_t heads, int64_t D,
                             const int64_t* slots, const void* cache, int64_t pages, int64_t page_size,
                             struct CUstream_st* stream);

/*
 * Attention of query tokens on the cache.  Sequence b has lengths[b] cached tokens, token t in
 * page page_table[b][t / page_size], and its query tokens are its last ones (they are written
 * to the cache before the call).  For the query at position j of the sequence and query head h,
 * which reads key head h / (Hq / Hkv):
 *   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale * q . k_t - max),  over the tokens t <= j,
 *   with a window also t > j - window, or, without causal, over all lengths[b] tokens.
 *   q, out     : [T][Hq][D] fp16 or bf16; out 16-byte aligned, q too (and its strides);
 *                out (and lse, the workspace) must not overlap q or the other arguments
 *   page_table : int32 [B][max_pages], the pages of a sequence's length (room for more costs little, but
 *                where few rows meet a wide table a row tile's tokens are cut by its width)
 *   lengths    : int32 [B]
 * Options (NULL = {0, 1, 0, 0, NULL, NULL, NULL, NULL, 0, 0}):
 *   scale      : > 0; 0 = 1 / sqrt(D)
 *   causal     : 0 or 1
 *   window     : 0 = none (needs causal)
 *   max_q      : with q_starts, the most query tokens of a sequence (0 = T), for the choice of
 *                kernels; the rows of a sequence with more may be left as they are
 *   q_starts   : NULL (T / B query tokens each), or int32 [B + 1]: rows q_starts[b] to
 *                q_starts[b + 1] - 1 of q are sequence b's; rows behind the last stay as they are
 *   encode_k, encode_v : as nvfp4_kv_write had them
 *   lse        : NULL, or fp32 [T][Hq]: log sum_t exp(scale * q . k_t)
 *   q_token_stride, q_head_stride : elements, 0 = dense
 * A query that sees no token has out 0 and lse -inf.  What masked places hold does not matter,
 * infinities and NaN (a NaN scale code) among them.  A page outside [0, pages) makes the
 * queries that see it NaN, a length beyond max_pages * page_size those of the sequence; both
 * read nothing outside the cache.
 * workspace: nvfp4_attention_workspace_bytes bytes, 256-byte aligned; need not be kept, but no
 * two calls that may run at once can share it.
 * Accuracy: scores and sums in fp32; p to fp16 before the product with v (2^-11 of itself, or 2^-32 of the
 * row's largest where that is more); out rounded once.  bf16 queries go over to fp16 in a power of two of
 * their row: elements below 2^-29 of the row's largest lose bits, below 2^-39 they are 0.
 * Limits: Hq % Hkv == 0, T * Hq < 2^31, max_pages * page_size <= 2^31 - 256, B <= 2^20, and
 * B * Hkv * max_pages * page_size < 2^36, less by the passes that more than 8 query tokens x heads of
 * a group take (up to 8).
 */
typedef struct {
  float scale;
  int32_t causal;
  int32_t window;
  int32_t max_q;
  const int32_t* q_starts;
  const float* encode_k;
  const float* encode_v;
  float* lse;
  int64_t q_token_stride;
  int64_t q_head_stride;
} nvfp4_attention_options_t;
size_t nvfp4_attention_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page_size,
                                       int64_t max_pages, int ragged, int64_t max_q);
nvfp4_status_t nvfp4_attention(const void* q, int dtype, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                               const void* cache, int64_t pages, int64_t page_size, const int32_t* page_table,
                               int64_t max_pages, const int32_t* lengths, int64_t B,
                               const nvfp4_attention_options_t* options, void* out, void* workspace,
                               size_t workspace_bytes, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_GEMV_H */
