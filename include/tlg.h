/*
 * tlg.h -- C interface of libtlg, a B200 (sm_100a) fp16 GEMM library.
 *
 * The operation is the block-tiled GEMM of the TileLang pages:
 *
 *   C = A . B      A: M x K fp16, row-major (K contiguous), row stride lda
 *                  B: K x N fp16, row-major (N contiguous), row stride ldb
 *                  C: M x N, row-major, row stride ldc
 *
 * accumulated in fp32 ("tilelang operator-compilation walkthrough",
 * lqnn.cn/news/222844, section 2.1: one fp32 accumulator tile per output block,
 * filled over the K loop; section 4.2: fp16 in, fp32 accumulate, fp16 out;
 * "TileLang Python DSL practice", codechina.net/.../126997, section 3.2: the
 * same product written to an fp32 C).  The fused variant applies a per-column
 * bias and a ReLU before the fp16 store ("domestic-GPU TileLang adoption",
 * xdnf.cn/news/333523, section 4.2); tlg_gemm_fused generalises it to a bias,
 * an activation (ReLU or GELU) and a residual connection (same page, 4.1).
 * Beside it stand operators over 4-bit and 8-bit microscaled matrices, and
 * those of a feed-forward block around its products (their sections below).
 *
 * Conventions shared by every entry point below:
 *
 *  - All matrix pointers are DEVICE pointers (cudaMalloc, a caching
 *    allocator, or managed memory) on the current CUDA device.  A host pointer
 *    is rejected with TLG_ERR_INVALID_ARG instead of silently producing an
 *    empty result (the pitfall named in "tilelang operator-compilation
 *    walkthrough" section 5.2).
 *  - The caller owns every buffer.  C is overwritten (no accumulate-into).
 *    C must not overlap A, B or the bias.
 *  - The call is asynchronous: it enqueues work on `stream` (a cudaStream_t;
 *    NULL means the legacy default stream) and returns.  Calls are
 *    stream-ordered and may be issued from several host threads and on
 *    several streams at once.
 *  - CUDA graphs: a call may be captured into a graph (stream capture) once
 *    a call with the same kernel configuration has run eagerly on the device
 *    (the first call sets the kernel's launch attributes).  The graph keeps
 *    the pointers, sizes and tensor maps of the captured call; each replay
 *    recomputes C from the buffers' current contents.  A split-K workspace
 *    is left ready for the next replay.
 *  - The library allocates no device memory.
 *  - Alignment: every pointer must be aligned to its element (2 bytes for fp16
 *    data, 4 for an fp32 C), else TLG_ERR_ALIGNMENT.  The fast path loads and
 *    stores tiles with the TMA engine, which needs 16-byte aligned bases and
 *    row strides (lda*2, ldb*2, ldc*sizeof(out)) that are multiples of 16
 *    bytes.  Operands that break that rule are copied into an aligned layout
 *    when the call's workspace has room (tlg_gemm_workspace_size_op);
 *    otherwise they are loaded by plain loads (several times slower) and such
 *    a C is written by plain stores.
 *  - Sizes: 0 <= M, N, K <= 2^31 - 257, and ceil(M/128)*ceil(N/64) below 2^31;
 *    leading dimensions at most 2^36 elements and every matrix spanning less
 *    than 2^60 bytes (larger sizes give TLG_ERR_UNSUPPORTED); lda >= K,
 *    ldb >= N, ldc >= N.
 *    M == 0 or N == 0: nothing is written, TLG_OK.  K == 0: the empty sum is
 *    0, so C = 0 (bias variant: C = fp16(max(bias[col], 0)); tlg_gemm_fused:
 *    C = act(bias[col]) + residual).
 *  - The return value is the only error channel; nothing throws or aborts.
 *    Errors found before launch leave C untouched.  An error of the launch
 *    itself is TLG_ERR_CUDA.  Errors the kernel detects on the device (a
 *    pipeline wait that exceeded its time limit) are not visible to the
 *    asynchronous call; read them with tlg_device_error().
 *  - Requires an sm_100 device (B200); other devices give TLG_ERR_UNSUPPORTED.
 */
#ifndef TLG_H
#define TLG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum tlg_status {
    TLG_OK = 0,
    TLG_ERR_INVALID_ARG = 1, /* negative size, null/host pointer, ld too small, overlap */
    TLG_ERR_ALIGNMENT = 2,   /* pointer not aligned to its element; workspace not 256-byte aligned */
    TLG_ERR_UNSUPPORTED = 3, /* not an sm_100 device, size beyond 2^31-1, bad config */
    TLG_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed */
    TLG_ERR_TIMEOUT = 5      /* a kernel reported a pipeline wait past its time limit */
} tlg_status;

/*
 * C (fp32) = A . B with fp32 accumulation.
 * Page: "TileLang Python DSL practice" (codechina.net/.../126997) section 3.2
 * (fp16 A/B, fp32 C, fp32 accumulation).
 */
tlg_status tlg_gemm_f16f32(int64_t M, int64_t N, int64_t K,
                           const void *A, int64_t lda,
                           const void *B, int64_t ldb,
                           float *C, int64_t ldc,
                           void *stream);

/*
 * C (fp16) = round_to_nearest_even(A . B), fp32 accumulation.
 * Page: "tilelang operator-compilation walkthrough" (lqnn.cn/news/222844)
 * sections 2.1 and 4.2 (fp16 in, fp32 accumulator, fp16 C).
 */
tlg_status tlg_gemm_f16f16(int64_t M, int64_t N, int64_t K,
                           const void *A, int64_t lda,
                           const void *B, int64_t ldb,
                           void *C, int64_t ldc,
                           void *stream);

/*
 * C (fp16) = round_to_nearest_even(max(A . B + bias[col], 0)), fp32
 * accumulation; the bias (N fp16 values, device memory, 16-byte aligned) is
 * added in fp32 to the fp32 accumulator before the ReLU.
 * Page: "domestic-GPU TileLang adoption" (xdnf.cn/news/333523) section 4.2
 * (bias looked up at the output column, added, then max with 0).
 */
tlg_status tlg_gemm_bias_relu_f16(int64_t M, int64_t N, int64_t K,
                                  const void *A, int64_t lda,
                                  const void *B, int64_t ldb,
                                  const void *bias,
                                  void *C, int64_t ldc,
                                  void *stream);

/* ---------------------------------------------------------------- extended */

/* Output type / epilogue selectors for tlg_gemm_ex. */
typedef enum tlg_out { TLG_OUT_F32 = 0, TLG_OUT_F16 = 1 } tlg_out;
typedef enum tlg_epilogue { TLG_EPI_NONE = 0, TLG_EPI_BIAS_RELU = 1 } tlg_epilogue;

/*
 * Kernel configuration.  Zero in any field means "choose for me" (the
 * library's per-shape table, the analogue of the pages' cached tuned
 * configurations: "tilelang operator-compilation walkthrough" section 5.3).
 *   block_n     : output tile width, 64, 128 or 256 columns, or 512 for a CTA
 *                 pair whose tile fills TMEM with two 256-column halves
 *   stages      : depth of the shared-memory operand ring (fixed per tile shape)
 *   cta_group   : 1 (one SM per 128-row tile) or 2 (an SM pair per 256-row tile)
 *   raster_group: number of tile rows walked together for L2 reuse, 1..64
 *   max_ctas    : cap on resident CTAs (0 = one per SM, or as many 2-CTA
 *                 clusters as the device can hold); tlg_choose_config
 *                 reports the number of CTAs the launch would use
 *   split_k     : 1 = every tile whole; 2..16 = the tiles left over after
 *                 the last full wave are cut into that many k-slices (needs a
 *                 workspace).  0 = automatic: every tile whole, or, when the
 *                 call supplies a workspace large enough, a split tail of
 *                 2..4 slices behind at least one whole wave where the cost
 *                 model ranks it faster (measured on a B200: +4.5 % at
 *                 4096^3 fp16 with split 2).  Calls without a workspace never
 *                 split.
 *   overlap_prev: 1 = the kernel may begin its set-up (barriers, TMEM, tensor
 *                 maps) while the previous kernel in the stream is still
 *                 finishing (programmatic dependent launch); it reads and
 *                 writes global memory only after that kernel has completed.
 *                 0 (default) = ordinary stream order.
 *   k_split     : 1 = each tile's whole K range is summed by one CTA (or CTA
 *                 pair); 2 or 4 = a cluster of that many one-CTA tiles'
 *                 CTAs shares every tile, each summing a slice of its
 *                 k-blocks, and the partial sums are added in slice order
 *                 through distributed shared memory (no workspace, so the
 *                 plain entry points use it too).  Built for block_n 128
 *                 (k_split 2) and 256 (k_split 2 or 4), untransposed operands
 *                 that TMA can describe, at least k_split k-blocks of 64, and
 *                 no split_k tail.  0 = automatic: chosen where few tiles
 *                 would leave most SMs idle (small or short-K shapes).
 * A combination the library does not provide gives TLG_ERR_UNSUPPORTED.
 */
typedef struct tlg_config {
    int32_t block_n;
    int32_t stages;
    int32_t cta_group;
    int32_t raster_group;
    int32_t max_ctas;
    int32_t split_k;
    int32_t overlap_prev;
    int32_t k_split;
} tlg_config;

/*
 * The three entry points above in one call, with an explicit configuration
 * (NULL = automatic) and an optional workspace.  bias must be NULL unless
 * epilogue is TLG_EPI_BIAS_RELU, and the bias epilogue needs
 * out == TLG_OUT_F16.  Same arguments, ownership and errors as above.
 *
 * Workspace (split-K tail): when the tile count leaves the last wave of SMs
 * partly idle, the leftover tiles can be cut along K into slices that run
 * concurrently; each slice writes an fp32 partial sum to the workspace and the
 * last slice to finish adds all partials in slice order (so the result does
 * not depend on timing) and writes C.  `workspace` is caller-owned device
 * memory, 256-byte aligned, not overlapping A, B, C or the bias;
 * tlg_gemm_workspace_size() gives the bytes a configuration needs (at most
 * about 20 MB on a B200 for any shape: the tail holds fewer slices than
 * there are SMs).  Its first 4 KB hold counters
 * that must be ZERO before the first call (e.g. cudaMemsetAsync once); every
 * completed call leaves them zero again.  Calls that overlap in time (other
 * streams) must not share a workspace.  After a TLG_ERR_TIMEOUT report the
 * counters may be non-zero: clear them again.  NULL or too small a workspace
 * with split_k >= 2 is TLG_ERR_INVALID_ARG; without a split the workspace is
 * not touched.
 */
tlg_status tlg_gemm_ex(int64_t M, int64_t N, int64_t K,
                       const void *A, int64_t lda,
                       const void *B, int64_t ldb,
                       const void *bias,
                       void *C, int64_t ldc,
                       tlg_out out, tlg_epilogue epilogue,
                       const tlg_config *config,
                       void *workspace, size_t workspace_bytes,
                       void *stream);

/*
 * tlg_gemm_ex for callers that cannot allocate device memory.  (This entry
 * point has no counterpart on the pages; it exists for library users.)
 *
 * Some callers cannot call cudaMalloc where they run a GEMM: a plugin inside
 * a framework that owns all device memory through its own allocator, code
 * with a fixed memory budget set at start-up, or a latency-critical path
 * that must not risk the device-wide synchronisation an allocation can
 * cause.  For them this call runs the split-K tail (config->split_k >= 2)
 * with the library's own scratch: a static device array of 16 MiB that every
 * GPU loading this library holds until the process exits.  Without
 * config->split_k >= 2 no scratch is needed and the call is tlg_gemm_ex with
 * no workspace.
 *
 * - Nothing is allocated: no cudaMalloc, cudaFree or allocating library call.
 * - Every call, split or not, first looks up the array's device address on
 *   the current device (once per device; later calls reuse it).  The first
 *   call on a device may also load the library's device code: make it before
 *   any stream capture.
 * - A schedule needing more than 16 MiB of scratch gives TLG_ERR_UNSUPPORTED
 *   before anything is launched (tlg_gemm_workspace_size reports the need).
 * - With split_k >= 2 and an A, B or C that TMA cannot describe (see
 *   tlg_gemm_workspace_size_op), the aligned copies also go into the array,
 *   after the split scratch, when they fit; otherwise the plain-load path
 *   runs, as for tlg_gemm_ex with too small a workspace.
 * - Every call on a device shares the one array, which keeps what the last
 *   call left; each call clears the counters it needs on its stream first.
 *   Calls that overlap on the GPU (different streams, or different host
 *   threads without ordering) race on the array and give wrong results:
 *   order them on one stream.
 * - Arguments, layout, ownership and the other errors are as tlg_gemm_ex.
 */
tlg_status tlg_gemm_ex_noalloc(int64_t M, int64_t N, int64_t K,
                               const void *A, int64_t lda,
                               const void *B, int64_t ldb,
                               const void *bias,
                               void *C, int64_t ldc,
                               tlg_out out, tlg_epilogue epilogue,
                               const tlg_config *config,
                               void *stream);

/* Whether an operand is used as stored (N) or transposed (T). */
typedef enum tlg_op { TLG_OP_N = 0, TLG_OP_T = 1 } tlg_op;

/*
 * C = op(A) . op(B) with the same epilogues, configuration and workspace as
 * tlg_gemm_ex, for operands stored transposed: the products of the pages'
 * autograd wrapper, grad_A = grad_C . B^T and grad_B = A^T . grad_C ("TileLang
 * Python DSL practice", codechina.net/.../126997, section 5.1).
 *   op_a == TLG_OP_N: A is M x K row-major, lda >= K (as tlg_gemm_ex).
 *   op_a == TLG_OP_T: A is stored K x M row-major, lda >= M; op(A) = A^T.
 *   op_b == TLG_OP_N: B is K x N row-major, ldb >= N (as tlg_gemm_ex).
 *   op_b == TLG_OP_T: B is stored N x K row-major, ldb >= K; op(B) = B^T.
 * C is always M x N row-major.  The 16-byte alignment rules apply to the
 * stored matrices (lda*2, ldb*2 multiples of 16).  Other arguments and errors
 * as tlg_gemm_ex; an op other than N or T is TLG_ERR_INVALID_ARG.
 */
tlg_status tlg_gemm_op(int64_t M, int64_t N, int64_t K,
                       tlg_op op_a, const void *A, int64_t lda,
                       tlg_op op_b, const void *B, int64_t ldb,
                       const void *bias,
                       void *C, int64_t ldc,
                       tlg_out out, tlg_epilogue epilogue,
                       const tlg_config *config,
                       void *workspace, size_t workspace_bytes,
                       void *stream);

/* Activations of the fused epilogue. */
typedef enum tlg_activation {
    TLG_ACT_NONE = 0,
    TLG_ACT_RELU = 1,      /* max(x, 0) */
    TLG_ACT_GELU = 2,      /* x * Phi(x) = x/2 * (1 + erf(x / sqrt 2)), the exact (erf) form */
    TLG_ACT_SILU = 3,      /* x * sigmoid(x) = x / (1 + exp(-x)) */
    TLG_ACT_GELU_TANH = 4  /* x/2 * (1 + tanh(sqrt(2/pi) * (x + 0.044715 x^3))) */
} tlg_activation;

/*
 * The general fused epilogue of tlg_gemm_fused:
 *
 *   C[i][j] = act(acc[i][j] + bias[j]) + residual[i][j]
 *
 * acc is the fp32 accumulator of op(A) . op(B); everything is computed in
 * fp32 and rounded once to C's type at the store.  Activation accuracy:
 * GELU is within 3e-7 of the exact form for an fp32 C; for an fp16 C its
 * fp32 value is within 0.15 fp16 units in the last place, so the stored
 * result is within 0.65 units.  SiLU and the tanh form use the hardware
 * exp2 and reciprocal approximations: on [-12, 12] their error stays below
 * 2e-6 times (1 + the largest |value|).
 *   bias       : N fp16 values (device memory), or NULL for none
 *   activation : a tlg_activation
 *   residual   : M x N row-major in C's type (fp16 for TLG_OUT_F16, fp32 for
 *                TLG_OUT_F32), row stride ldr >= N elements, device memory;
 *                or NULL for none.  It may be C itself (residual == C and
 *                ldr == ldc: an in-place residual connection); any other
 *                overlap with C is TLG_ERR_INVALID_ARG.
 * Page: "domestic-GPU TileLang adoption" (xdnf.cn/news/333523) section 4.1
 * names fusing an activation and a residual connection into the GEMM;
 * section 4.2 gives the bias-by-column-then-ReLU form (bias, TLG_ACT_RELU,
 * no residual, fp16 C is exactly tlg_gemm_bias_relu_f16).  The pages print
 * no activation formulas; each activation is its standard definition.
 */
typedef struct tlg_fused_epilogue {
    const void *bias;
    int32_t activation;
    const void *residual;
    int64_t ldr;
} tlg_fused_epilogue;

/*
 * C = act(op(A) . op(B) + bias) + residual, with either output type.
 * Operands, op_a / op_b, configuration, workspace and errors as tlg_gemm_op.
 * epilogue == NULL, or one with no bias, TLG_ACT_NONE and no residual, is
 * the plain product.  An activation outside tlg_activation is
 * TLG_ERR_INVALID_ARG; a residual pointer not aligned to its element is
 * TLG_ERR_ALIGNMENT (a 16-byte aligned base and row stride let it be read
 * 16 bytes at a time).  K == 0 gives C = act(bias) + residual.
 */
tlg_status tlg_gemm_fused(int64_t M, int64_t N, int64_t K,
                          tlg_op op_a, const void *A, int64_t lda,
                          tlg_op op_b, const void *B, int64_t ldb,
                          const tlg_fused_epilogue *epilogue,
                          void *C, int64_t ldc, tlg_out out,
                          const tlg_config *config,
                          void *workspace, size_t workspace_bytes,
                          void *stream);

/*
 * Workspace bytes tlg_gemm_ex would use for this shape and configuration
 * (NULL = automatic) when given enough; 0 when every tile runs whole.
 * The answer does not depend on the epilogue, so it also holds for
 * tlg_gemm_op and tlg_gemm_fused.
 * No kernel is launched; the only CUDA calls read device attributes.
 */
tlg_status tlg_gemm_workspace_size(int64_t M, int64_t N, int64_t K, tlg_out out,
                                   tlg_epilogue epilogue, const tlg_config *config,
                                   size_t *bytes);

/*
 * Workspace bytes for a call with these operands (tlg_gemm_ex, tlg_gemm_op or
 * tlg_gemm_fused with the same sizes, layouts, pointers and strides):
 * the split-K scratch of the configuration (NULL = automatic), plus room for
 * aligned copies of the matrices TMA cannot describe (a base address or row
 * stride not a multiple of 16 bytes).
 *
 * Given that much workspace, a call copies each such A or B into an aligned
 * layout in the workspace first and runs the TMA path on the copies; such a
 * C is produced in the workspace and copied out at the end.  Each copy moves
 * every byte once, so a call with odd strides then runs near the speed of
 * an aligned one instead of on the plain-load path.  Such a call enqueues up
 * to three kernels: one copying A and B, the GEMM, and the copy of C; the
 * GEMM and the copy of C start as programmatic dependents of the kernel
 * before them (their set-up overlaps its end; each waits for it before
 * touching memory).  With less workspace the
 * call still succeeds on the plain-load path (A and B copies are made only
 * when both fit; a C copy when it fits after them).  The copies never touch
 * the workspace's first 4 KB (the split-K counters).  0 when every matrix is
 * aligned and no split is chosen.  Only host-side checks and device-attribute
 * queries run; nothing is launched.
 */
tlg_status tlg_gemm_workspace_size_op(int64_t M, int64_t N, int64_t K,
                                      tlg_op op_a, const void *A, int64_t lda,
                                      tlg_op op_b, const void *B, int64_t ldb,
                                      const void *C, int64_t ldc, tlg_out out,
                                      const tlg_config *config, size_t *bytes);

/* ---------------------------------------------------------------- microscaled formats
 *
 * Matrices in 4 or 8 bits with one power-of-two scale for every 32 elements
 * along a row (the microscaling, MX, formats of the Open Compute Project), for
 * 4-bit products and 8-bit activation checkpoints.  (These entry points have
 * no counterpart on the pages; they exist for users who train and serve the
 * layers tlg_gemm_fused and tlg_gemm_op compute.)
 *
 * An MX matrix of rows x cols is two buffers:
 *
 *  - Q, the elements, row-major with a row stride of ldq BYTES.  A row holds
 *    ceil(cols / 32) whole blocks (16 bytes each for E2M1, 32 for E4M3); the
 *    elements past cols are 0.  E2M1: element 2i in the low half of byte i,
 *    2i + 1 in the high half.  Q must be 16-byte aligned and ldq a multiple
 *    of 16, at least the row bytes tlg_mx_size gives.
 *  - S, one E8M0 byte b per block, which stands for 2^(b - 127), 0xFF for
 *    NaN.  The bytes lie in tiles of 128 rows x 4 blocks, 512 bytes each: with
 *    tiles_x = ceil(ceil(cols / 32) / 4), the scale of (row, block) is byte
 *      ((row / 128) * tiles_x + block / 4) * 512
 *        + (row % 32) * 16 + ((row % 128) / 32) * 4 + block % 4.
 *    S must be 16-byte aligned and hold the bytes tlg_mx_size gives.  The
 *    bytes of blocks past the last one (up to a multiple of 4) are written as
 *    0 and must not be 0xFF in a matrix built elsewhere; the bytes of rows
 *    past the last one (up to a multiple of 128) are neither written nor used.
 *
 * An element's value is its E2M1 or E4M3 value times its block's scale.
 * Quantising a block whose largest magnitude is amax:
 *  - E2M1: scale 2^(floor(log2 amax) - 2); magnitudes above 6 scales saturate;
 *  - E4M3: the smallest power of two with amax <= 448 scales; nothing
 *    saturates;
 * with exponents held to [-127, 127] (-127 for an all-zero block), and each
 * element the nearest representable value, ties to even.  A block that holds
 * a NaN or an infinity gets the scale 0xFF: all of it reads back as NaN.
 *
 * Sizes: 0 <= rows, cols <= 2^31 - 257, strides at most 2^36, every matrix
 * below 2^60 bytes (TLG_ERR_UNSUPPORTED beyond).  Rows or cols of 0: nothing
 * is written, TLG_OK (tlg_act_backward_mx still writes dbias = 0 for rows of
 * 0).  Other matrices need only element alignment; those whose base and row
 * stride are multiples of 16 bytes are accessed 16 bytes at a time.  Inputs
 * must not overlap outputs except where an entry point says so, which is judged
 * by the bytes from a buffer's first element to its last (so two column ranges
 * of one matrix overlap), and every buffer is device memory of the current
 * device.  These calls launch as programmatic dependents of the kernel before
 * them in the stream: only their launch overlaps it; they touch memory after
 * it has completed.  All may be captured into CUDA graphs.
 */

/* Element types of ordinary matrices (f32 and f16 as in tlg_out). */
typedef enum tlg_type { TLG_TYPE_F32 = 0, TLG_TYPE_F16 = 1, TLG_TYPE_BF16 = 2 } tlg_type;

/* Element formats of MX matrices: 4 bits (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
 * negatives) and 8 bits (4 exponent and 3 mantissa bits, up to 448). */
typedef enum tlg_mx_format { TLG_MX_E2M1 = 0, TLG_MX_E4M3 = 1 } tlg_mx_format;

/* Bytes of one row of Q, and of S, for a rows x cols MX matrix.  Host only. */
tlg_status tlg_mx_size(tlg_mx_format format, int64_t rows, int64_t cols,
                       int64_t *q_row_bytes, size_t *s_bytes);

/*
 * Quantises a matrix.  op == TLG_OP_N: X is rows x cols, row-major, ldx >= cols.
 * op == TLG_OP_T: X is stored cols x rows, ldx >= rows, and its transpose is
 * quantised, the blocks running down X's columns: what the backward products
 * of a 4-bit layer need of its weights, activations and gradients.
 */
tlg_status tlg_mx_quantize(tlg_mx_format format, int64_t rows, int64_t cols,
                           tlg_op op, tlg_type type, const void *X, int64_t ldx,
                           void *Q, int64_t ldq, void *S, void *stream);

/* X (rows x cols) = the values of an MX matrix, rounded once to X's type. */
tlg_status tlg_mx_dequantize(tlg_mx_format format, int64_t rows, int64_t cols,
                             const void *Q, int64_t ldq, const void *S,
                             tlg_type type, void *X, int64_t ldx, void *stream);

/*
 * C = act(A . B^T + bias) + residual over 4-bit operands: A is an M x K and B
 * an N x K E2M1 MX matrix (K runs along the rows of both, as weights are
 * stored), C is M x N row-major of type out.  Every product of two elements
 * and their scales is exact, sums are fp32, and the result is rounded once.
 * M may be 1: a single token against a layer's weights.
 *
 * The backward products are the same call on transposed quantisations: with
 * C = A . B^T, dA = dC . B takes dC and B^T (tlg_mx_quantize with TLG_OP_T on
 * B), and dB = dC^T . A takes dC^T and A^T.
 *
 * epilogue as for tlg_gemm_fused, NULL for none: the bias holds N fp16 values
 * (bf16 when C is bf16), the residual has C's type and may be C itself.
 * config: NULL or zero fields choose automatically; block_n, cta_group,
 * stages, raster_group and max_ctas as for tlg_gemm_ex, split_k 0 or 1,
 * overlap_prev is always on.  M <= 32 has a kernel of its own (block_n 16 up
 * to 16 rows, else 32; it runs when cta_group, stages and max_ctas are 0, or
 * when block_n names it and they are 0 or what it runs with), where k_split 1,
 * 2, 4 or 8 CTAs share the K range (at most one per 256 k); elsewhere k_split
 * is 0 or 1.  No workspace.  K == 0 gives C = act(bias)
 * + residual.  Sizes and errors as tlg_gemm_fused's; lda and ldb are in BYTES
 * (ldq above).  A pipeline wait past its time limit is reported by
 * tlg_device_error().
 */
tlg_status tlg_gemm_mxfp4(int64_t M, int64_t N, int64_t K,
                          const void *A, int64_t lda, const void *SA,
                          const void *B, int64_t ldb, const void *SB,
                          const tlg_fused_epilogue *epilogue,
                          void *C, int64_t ldc, tlg_type out,
                          const tlg_config *config, void *stream);

/*
 * The configuration tlg_gemm_mxfp4 runs for this shape and type of C, as
 * tlg_choose_config: the request in *config (zero fields: automatic) is
 * replaced by the answer, which passed back as a request gives itself.  The
 * choice depends on whether there is an epilogue: the first function answers
 * for the plain product (epilogue NULL, or none of its parts), the second for
 * a call with `epilogue` (only which parts are set matters; its pointers are
 * not followed).
 */
tlg_status tlg_choose_config_mxfp4(int64_t M, int64_t N, int64_t K, tlg_type out,
                                   tlg_config *config);
tlg_status tlg_choose_config_mxfp4_fused(int64_t M, int64_t N, int64_t K,
                                         const tlg_fused_epilogue *epilogue,
                                         tlg_type out, tlg_config *config);

/*
 * Y = act(Z), and Z saved for the backward pass as an E4M3 MX matrix, in one
 * pass over Z.  Y may be Z itself (same base and row stride).  Computed in
 * fp32 and rounded once; the activations and their accuracy are
 * tlg_gemm_fused's (a bf16 Y takes the 16-bit form of GELU).
 */
tlg_status tlg_act_forward_mx(int64_t rows, int64_t cols, tlg_activation activation,
                              tlg_type type, const void *Z, int64_t ldz,
                              void *Y, int64_t ldy, void *Q, int64_t ldq, void *S,
                              void *stream);

/*
 * The backward pass of act on a saved input: dZ = dY * act'(Z), with Z the
 * values of the E4M3 MX matrix (Q, S), and, when dbias is not NULL, dbias[c] =
 * the sum over the rows of dZ[., c] (cols fp32 values), summed in fp32 before
 * dZ is rounded, in an order that does not depend on timing.  dZ may be dY
 * itself.  act' is computed in fp32 with an error below 1e-6, and GELU's on
 * [-12, -2], where it is small, within 2e-5 of its value.  ReLU's is 0 at 0,
 * and where it is 0 dZ is 0 whatever dY holds.  A NaN in Z makes dZ NaN, except
 * with TLG_ACT_NONE, whose derivative is 1 for every Z: dZ = dY.
 * workspace: tlg_act_backward_mx_workspace_size() bytes of device memory,
 * 256-byte aligned, needed when dbias is not NULL (TLG_ERR_INVALID_ARG when too
 * small; the size may be 0).  Its contents on entry do not matter; calls that
 * overlap in time must not share one.
 */
tlg_status tlg_act_backward_mx(int64_t rows, int64_t cols, tlg_activation activation,
                               tlg_type type, const void *dY, int64_t lddy,
                               const void *Q, int64_t ldq, const void *S,
                               void *dZ, int64_t lddz, float *dbias,
                               void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of tlg_act_backward_mx with a dbias, for the current device. */
tlg_status tlg_act_backward_mx_workspace_size(int64_t rows, int64_t cols, tlg_type type,
                                              size_t *bytes);

/* ---------------------------------------------------------------- around the linear layers
 *
 * Operators of a feed-forward block beside its linear layers: products grouped by expert with their
 * gradients, the root-mean-square norm with the residual's addition and its backward pass, and
 * products of a few rows with integer 4-bit weights.  (These entry points have no counterpart on the
 * pages; they exist for users who train and serve whole blocks with the products above.)  Pointers,
 * ownership, streams, graphs and errors are as for the microscaled operators: matrices need element
 * alignment only, those with a base and row stride that are multiples of 16 bytes are accessed faster,
 * inputs must not overlap outputs except where an entry point says so, and calls launch as programmatic
 * dependents of the kernel before them.
 */

/*
 * Products grouped by expert.  The rows of A and C are sorted by group: those of group g are
 * offsets[g] <= r < offsets[g + 1], and
 *
 *   C[r] = act(A[r] . op(B_g))     A: rows x K, C: rows x N
 *
 * with B_g the matrix at B + g * stride_b elements, K x N (TLG_OP_N, ldb >= N) or N x K (TLG_OP_T,
 * ldb >= K), as tlg_gemm_op.  stride_b may be 0: every group has the same B.  type is the type of A and
 * B (TLG_TYPE_F16 or TLG_TYPE_BF16), out that of C: the same, or TLG_TYPE_F32.  Sums are fp32, rounded
 * once after the activation, whose accuracy is tlg_gemm_fused's: at most 1024 terms (512 for an fp32 C) at a
 * time by the tensor core, whose adder truncates, and those parts added with rounding to nearest, so that
 * a long sum loses no more of its size than a short one.
 *
 * offsets: groups + 1 int32 values in device memory, read by the kernel (0 <= groups <= 1024).  They
 * should not decrease: values outside [0, rows] are held to it, and one that is less than an earlier one
 * counts as that one.  Rows of C before offsets[0] and from offsets[groups] on are left as they were, and
 * may hold anything in A.  K == 0
 * gives C = act(0) in the groups' rows.  The input gradient is the same call: dA_g = dC_g . op(B_g)^T
 * takes dC for A and the other op.  A pipeline wait past its time limit is reported by
 * tlg_device_error().
 */
tlg_status tlg_gemm_grouped(int64_t rows, int64_t N, int64_t K, int32_t groups, const int32_t *offsets,
                            tlg_type type, const void *A, int64_t lda,
                            tlg_op op_b, const void *B, int64_t ldb, int64_t stride_b,
                            tlg_activation activation,
                            void *C, int64_t ldc, tlg_type out, void *stream);

/*
 * Its weight gradient: dB_g = A_g^T . dC_g (K x N) or, for TLG_OP_T, its transpose (N x K), in the
 * layout of B: lddb and stride_db (not 0 for more than one group; the matrices must not overlap) in
 * elements.  dC has A's type; out is that type or TLG_TYPE_F32.  A group without rows gets dB_g = 0, and
 * every dB_g is overwritten.  Sums run over a group's rows in order, in fp32 as above, rounded once; what other
 * rows hold (NaN, infinities) does not matter.
 */
tlg_status tlg_gemm_grouped_dw(int64_t rows, int64_t N, int64_t K, int32_t groups, const int32_t *offsets,
                               tlg_type type, const void *A, int64_t lda, const void *dC, int64_t lddc,
                               tlg_op op_b, void *dB, int64_t lddb, int64_t stride_db,
                               tlg_type out, void *stream);

/*
 * The root-mean-square norm of every row, with the residual's addition in front of it:
 *
 *   H = X + R,   rstd[r] = 1 / sqrt(mean of H[r]^2 + eps),   Y = H * rstd * weight
 *
 * X, R, H and Y are rows x cols matrices of one type (any tlg_type), weight a vector of cols elements of
 * that type, rstd rows fp32 values.  R may be NULL (H = X); H and rstd may be NULL where they are not
 * needed.  H and Y may each be X or R itself (same base and row stride).  Computed in fp32 from the
 * unrounded H and rounded once; the sum of a row does not depend on timing.  eps >= 0 and finite.
 * cols <= 16384 (TLG_ERR_UNSUPPORTED beyond).  A row that holds a NaN has rstd and Y NaN.  Of a row whose
 * sum of squares is infinite in fp32 (it holds an infinity, or squares that add up to one) rstd is 0, and Y is
 * 0 but for NaN where H is infinite.
 */
tlg_status tlg_rmsnorm_forward(int64_t rows, int64_t cols, tlg_type type,
                               const void *X, int64_t ldx, const void *R, int64_t ldr,
                               const void *weight, float eps, void *H, int64_t ldh,
                               void *Y, int64_t ldy, float *rstd, void *stream);

/*
 * The same with Y written as an MX matrix, quantised from the fp32 values as tlg_mx_quantize does:
 * TLG_MX_E2M1 for the A operand of tlg_gemm_mxfp4, TLG_MX_E4M3 in 8 bits.  So a row that holds a
 * NaN reads back as NaN, and of a row with an infinity its blocks of 32 with one do, the others as 0.
 */
tlg_status tlg_rmsnorm_forward_mx(int64_t rows, int64_t cols, tlg_type type,
                                  const void *X, int64_t ldx, const void *R, int64_t ldr,
                                  const void *weight, float eps, void *H, int64_t ldh,
                                  tlg_mx_format format, void *Q, int64_t ldq, void *S,
                                  float *rstd, void *stream);

/*
 * Its backward pass, from the H and rstd of the forward pass: with x = H * rstd and g = dY * weight,
 *
 *   dX = rstd * (g - x * mean over the row of (g * x)) + dH,   dweight[c] = sum over the rows of dY * x
 *
 * dX is the gradient of X and of R alike.  dH, what arrives on the residual stream behind the norm, may
 * be NULL, and so may dweight (cols fp32 values).  dX may be dY or dH itself (same base and row stride).
 * Sums are fp32, in an order that does not depend on timing; dweight's parts, sums of some rows each, are
 * added in 64 bits.  rows of 0: dweight = 0.  cols <= 16384.
 * workspace: tlg_rmsnorm_backward_workspace_size() bytes of device memory, 256-byte aligned, needed when
 * dweight is not NULL (TLG_ERR_INVALID_ARG when too small; the size may be 0).  Its contents on entry do
 * not matter; calls that overlap in time must not share one.
 */
tlg_status tlg_rmsnorm_backward(int64_t rows, int64_t cols, tlg_type type,
                                const void *dY, int64_t lddy, const void *H, int64_t ldh,
                                const void *weight, const float *rstd, const void *dH, int64_t lddh,
                                void *dX, int64_t lddx, float *dweight,
                                void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of tlg_rmsnorm_backward with a dweight, for the current device. */
tlg_status tlg_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols, tlg_type type, size_t *bytes);

/*
 * A product of few rows (tokens) with integer 4-bit weights that have a scale for each group of k:
 *
 *   C = act(X . W^T + bias) + residual,   W[n, k] = (q[n, k] - z[n, k / group]) * s[n, k / group]
 *
 *  - X is M x K of type TLG_TYPE_F16 or TLG_TYPE_BF16; C is M x N of that type or TLG_TYPE_F32.
 *  - Q holds q (0 .. 15), row-major with a row stride of ldq BYTES, two elements to a byte, 2i in the low
 *    half of byte i.  A row holds ceil(K / 32) * 16 bytes, whose elements past K do not matter.  Q must be
 *    16-byte aligned and ldq a multiple of 16.
 *  - S holds s, N x ceil(K / group) contiguous values of X's type, Z the zero points z, as many bytes of
 *    0 .. 15 (their low four bits count), or NULL for z = 8 everywhere.
 *  - group is a power of two from 32 on.
 *
 * Products and sums are fp32 and no weight is rounded: a group's sum of (q - z) * X is multiplied by its
 * scale.  epilogue as for tlg_gemm_fused, NULL for none: the bias holds N elements of X's type, the residual
 * has C's type and may be C itself.  M may be any: rows of X are taken 16 at a time, which read the
 * weights again each time, so the call is made for the few rows of a decoding step.  K == 0 gives C =
 * act(bias) + residual.  No workspace.
 */
tlg_status tlg_gemv_q4(int64_t M, int64_t N, int64_t K, tlg_type type, const void *X, int64_t ldx,
                       const void *Q, int64_t ldq, const void *S, const uint8_t *Z, int64_t group,
                       const tlg_fused_epilogue *epilogue, void *C, int64_t ldc, tlg_type out, void *stream);

/*
 * Resolve a configuration for this shape.  On input *config (never NULL)
 * holds the requested fields, zero meaning "choose for me" (all zero: the
 * automatic choice); on output it holds the configuration tlg_gemm_ex would
 * run given a workspace of tlg_gemm_workspace_size() bytes, every field
 * filled in.  TLG_ERR_UNSUPPORTED if the request names a
 * combination the library does not provide.  No kernel is launched; the only
 * CUDA calls read the current device's attributes.
 */
tlg_status tlg_choose_config(int64_t M, int64_t N, int64_t K, tlg_out out,
                             tlg_epilogue epilogue, tlg_config *config);

/*
 * Device-side error report for the current device.  Synchronizes the device,
 * reads the library's device error word and, if clear != 0, resets it.
 * *code_out (may be NULL) receives the raw word: 0 when no kernel has
 * reported an error; otherwise bit 0 = a pipeline wait ran past its limit,
 * and one bit per role that gave up: bit 8 the TMA producer, bit 9 the MMA
 * issuer, bit 10 the epilogue, bit 11 tlg_selftest_timeout.
 * Returns TLG_ERR_TIMEOUT when the word is non-zero, TLG_ERR_CUDA when the
 * synchronization fails, TLG_OK otherwise.
 */
tlg_status tlg_device_error(int clear, uint32_t *code_out);

/*
 * Self-test of the error path: launches one tiny kernel that waits on a
 * pipeline barrier nothing will ever signal, with a limit of `limit_us`
 * microseconds (1..1000000), on `stream`.  The wait gives up, the kernel
 * records the timeout in the device error word and returns normally; no
 * fault, trap or hang.  Read the result with tlg_device_error().
 */
tlg_status tlg_selftest_timeout(uint32_t limit_us, void *stream);

/* Static string for a status code; never NULL. */
const char *tlg_status_string(tlg_status status);

/* Library version, major*10000 + minor*100 + patch. */
int32_t tlg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TLG_H */
