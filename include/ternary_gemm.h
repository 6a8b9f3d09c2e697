/*
 * ternary_gemm.h -- C ABI of the MI355X (gfx950) ternary x int8 GEMM library
 * (libternary_gemm.so).
 *
 * Sources (cited by page title and section):
 *   [P10425] t27 pull request #10425, "t27c PTX backend: ternary x int8 GEMM
 *            kernel emitted by a .t27 spec (int8 mma.sync), ptx-run glue".
 *   [P10855] t27 pull request #10855, "spec(igla): hslm_bwd_ptx -- HSLM
 *            backward dX and dW as int8 tensor-core PTX written by t27".
 *
 * Stored ternary weights ("Wpacked").  W is a K x N matrix of weights in
 * {-1, 0, +1} kept as 2-bit codes, four per byte, one row of K/4 bytes per
 * output column n (N-major, the code index of (k, n) being n*K + k) [P10425
 * "What this adds"; P10855 PR body].  The code of (k, n) sits in byte
 * n*(K/4) + k/4 at bits 2*(k%4) and 2*(k%4)+1, the first code of a byte in the
 * least significant bits (the pages do not state the order inside a byte;
 * this is the reading taken).  A code c stands for the weight
 * (c & 1) - ((c >> 1) & 1): codes 0, 1, 2, 3 are 0, +1, -1, 0 [P10425 "What
 * this adds"; the same table appears as the byte-permute word 0x00FF0100 in
 * P10855 PR body].
 *
 * Conventions shared by every call:
 *   - All matrix arguments are DEVICE pointers to dense row-major storage with
 *     no padding between rows; the caller owns them.  The library allocates,
 *     frees, copies and retains nothing (the dX calls that take a workspace
 *     borrow the caller's device memory for the duration of the call).
 *   - No alignment beyond the element size is required; aligned bases and
 *     row lengths that are multiples of 16 take the fast load path.
 *   - Each call validates its arguments on the host first.  On any error it
 *     returns a negative status, launches nothing and leaves every output
 *     untouched.
 *   - On success the work is enqueued on `stream` (NULL: the default stream)
 *     and the call returns without waiting.  Faults that only show while the
 *     kernel runs surface at the caller's next synchronisation.
 *   - Results are exact: integer sums in int32, each output reduced over the
 *     whole contraction in a fixed order with no atomics: inside one
 *     workgroup, or, on the workspace path of dX, as per-workgroup partial
 *     sums added in split order by a second kernel.  Integer addition is
 *     exact, so every path and every repeated call gives identical bits.
 *   - Calls are thread-safe; concurrent calls on different streams may run at
 *     the same time as long as their outputs do not overlap.
 */
#ifndef TERNARY_GEMM_H
#define TERNARY_GEMM_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
typedef enum tgemm_status {
    TGEMM_OK = 0,
    TGEMM_ERR_NULL = -1,   /* a required pointer is NULL                        */
    TGEMM_ERR_DIM = -2,    /* a dimension is < 1, or a size does not fit        */
    TGEMM_ERR_PACK = -3,   /* the packed dimension K is not a multiple of 4     */
    TGEMM_ERR_BOUND = -4,  /* the contraction is longer than the exact-int32 bound */
    TGEMM_ERR_ALIAS = -5,  /* the output overlaps an input                       */
    TGEMM_ERR_HIP = -6,    /* the HIP runtime reported an error at launch        */
    TGEMM_ERR_KIND = -7,   /* the output kind of a scaled call is not one of
                              TGEMM_OUT_F32, TGEMM_OUT_BF16, or the input kind
                              of a quantizer call not TGEMM_IN_F32,
                              TGEMM_IN_BF16                                   */
    TGEMM_ERR_SCRATCH = -8, /* ternary_gemm_s8_dx_noalloc: the split needs more
                              than TGEMM_STATIC_SCRATCH_BYTES of scratch      */
    TGEMM_ERR_VALUE = -9,  /* a scalar argument (eps, max_norm, act) is out of
                              its range                                       */
    TGEMM_ERR_WORKSPACE = -10 /* a required workspace is NULL, too small or not
                              16-byte aligned                                 */
} tgemm_status;

/* Longest contraction for which every int32 result is exact whatever the
 * inputs.  Ternary x int8 (forward, dX): |sum| <= 128 * L must fit int32,
 * L <= floor((2^31 - 1) / 128) [P10425 "What this adds", invariant "i32
 * overflow bound"].  int8 x int8 (dW): L <= floor((2^31 - 1) / 128^2) = 131071
 * [P10855 PR body, kernel 2, "k <= 131071"]. */
#define TGEMM_TERNARY_MAX_CONTRACTION 16777215LL
#define TGEMM_INT8_MAX_CONTRACTION 131071LL

/*
 * Forward product [P10425 "What this adds"]:
 *     C[m][n] = sum_{k<K} A[m][k] * w(k, n)
 *   A        int8    [M][K]
 *   Wpacked  uint8   [N][K/4]   (stored ternary weights, layout above)
 *   C        int32   [M][N]     (written, never read)
 * Requires M, N, K >= 1, K % 4 == 0 (TGEMM_ERR_PACK otherwise) and
 * K <= TGEMM_TERNARY_MAX_CONTRACTION (TGEMM_ERR_BOUND).
 */
int ternary_gemm_s8(const int8_t *A, const uint8_t *Wpacked, int32_t *C,
                    int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * dX = dC x W^T with the same stored ternary W as the forward product
 * [P10855 PR body, kernel 1 "hslm_dx_s8"]:
 *     dX[m][k] = sum_{n<N} dC[m][n] * w(k, n)
 *   dC       int8    [M][N]
 *   Wpacked  uint8   [N][K/4]   (the forward call's buffer, unchanged)
 *   dX       int32   [M][K]     (written, never read)
 * Requires M, N, K >= 1, K % 4 == 0 (TGEMM_ERR_PACK) and
 * N <= TGEMM_TERNARY_MAX_CONTRACTION (TGEMM_ERR_BOUND).
 */
int ternary_gemm_s8_dx(const int8_t *dC, const uint8_t *Wpacked, int32_t *dX,
                       int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * dW = A^T x dC, int8 x int8 -> int32, summed over the M rows
 * [P10855 PR body, kernel 2 "hslm_dw_s8"]:
 *     dW[k][n] = sum_{m<M} A[m][k] * dC[m][n]
 *   A        int8    [M][K]
 *   dC       int8    [M][N]
 *   dW       int32   [K][N]     (written, never read)
 * Requires M, N, K >= 1 and M <= TGEMM_INT8_MAX_CONTRACTION (TGEMM_ERR_BOUND).
 * K need not be a multiple of 4 (no packed operand).
 */
int ternary_gemm_s8_dw(const int8_t *A, const int8_t *dC, int32_t *dW,
                       int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * Scaled outputs: the integer product followed by its dequantization, fused
 * into the kernels' stores.  The pages leave the scales to the host: the
 * activations are quantized per row for dX and X and dY per column for dW
 * [P10855 PR body]; the forward takes the same per-row activation scale, and
 * the ternary weights one scale for the whole matrix (the reading taken).
 * Each output element is
 *     y = (float(acc) * row_scale[row]) * col_scale
 * where acc is the exact int32 result of the plain call, the int32 -> float
 * conversion and each product are IEEE single precision rounded to nearest
 * even, in that order, and col_scale is the weight scale (forward, dX) or
 * dc_col_scale[n] (dW).  TGEMM_OUT_F32 stores y as float; TGEMM_OUT_BF16
 * stores y rounded to the nearest bfloat16, ties to even (a NaN stays a
 * quiet NaN), as uint16 bit patterns, which halves the bytes written.
 * Scale vectors are DEVICE float arrays; output element counts and layouts
 * are those of the plain calls.  Besides the plain calls' checks, a NULL
 * scale vector returns TGEMM_ERR_NULL, an output kind other than the two
 * below TGEMM_ERR_KIND, and an output overlapping a scale vector
 * TGEMM_ERR_ALIAS.
 */
#define TGEMM_OUT_F32 1
#define TGEMM_OUT_BF16 2

/* forward: Y[m][n] = (float(C[m][n]) * a_row_scale[m]) * w_scale;
 * a_row_scale float [M]. */
int ternary_gemm_s8_scaled(const int8_t *A, const uint8_t *Wpacked, const float *a_row_scale,
                           float w_scale, void *Y, int out_kind,
                           int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* dX: Y[m][k] = (float(dX[m][k]) * dc_row_scale[m]) * w_scale;
 * dc_row_scale float [M]. */
int ternary_gemm_s8_dx_scaled(const int8_t *dC, const uint8_t *Wpacked, const float *dc_row_scale,
                              float w_scale, void *dX, int out_kind,
                              int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * dX with a workspace, for few rows and long rows of Wpacked (the backward
 * of a decode-sized batch, [P10855 "Measured"]: 27 rows).  Same products,
 * arguments, checks and results as ternary_gemm_s8_dx and
 * ternary_gemm_s8_dx_scaled; in addition the caller lends `workspace`, a
 * DEVICE buffer of `workspace_bytes` bytes.  When M <= 32, N % 64 == 0,
 * K % 256 == 0, dC and Wpacked are 16-byte aligned and K / 256 column
 * blocks are too few to fill the chip, the contraction is split across
 * workgroups: each writes its int32 partial sums to the workspace and a
 * second kernel adds them in split order, which is faster when each W row is
 * long (27 x 16384 x 16384: about 32 against 46 us).  The workspace must then hold
 * ternary_gemm_dx_workspace() bytes and be 16-byte aligned; a NULL, smaller
 * or unaligned workspace runs the one-pass kernels instead, with the same
 * results.  The workspace's contents on entry do not matter and are garbage
 * afterwards; it is in use until the call completes on `stream`, so calls
 * that may overlap need workspaces of their own.  A workspace overlapping an
 * input, the output or the scale vector returns TGEMM_ERR_ALIAS, a negative
 * workspace_bytes TGEMM_ERR_DIM.
 */
int ternary_gemm_s8_dx_ws(const int8_t *dC, const uint8_t *Wpacked, int32_t *dX,
                          int64_t M, int64_t N, int64_t K, void *workspace,
                          int64_t workspace_bytes, hipStream_t stream);
int ternary_gemm_s8_dx_scaled_ws(const int8_t *dC, const uint8_t *Wpacked, const float *dc_row_scale,
                                 float w_scale, void *dX, int out_kind,
                                 int64_t M, int64_t N, int64_t K, void *workspace,
                                 int64_t workspace_bytes, hipStream_t stream);

/*
 * dX that allocates nothing, for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same product, arguments, checks and results as
 * ternary_gemm_s8_dx_ws, with the workspace taken from a static device
 * buffer of TGEMM_STATIC_SCRATCH_BYTES that the library holds on each device
 * it runs on until the process ends (its address is looked up once per
 * device, on the device's first call).  When the contraction split applies
 * and needs more than that buffer (ternary_gemm_dx_workspace() bytes), the
 * call returns TGEMM_ERR_SCRATCH and launches nothing; without a split it
 * runs the one-pass kernels.  The call itself allocates nothing: no
 * hipMalloc, hipFree or allocating library routine.  Every call on a device
 * shares that device's buffer, whose contents on entry do not matter: calls
 * that may overlap on one device (two streams, two threads) race on it and
 * must be serialized by the caller.
 */
#define TGEMM_STATIC_SCRATCH_BYTES (8 << 20)
int ternary_gemm_s8_dx_noalloc(const int8_t *dC, const uint8_t *Wpacked, int32_t *dX,
                               int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* Workspace bytes the dX calls above use for these dimensions when the
 * inputs' base alignment is `align` bytes (the smallest power-of-two
 * alignment of dC and Wpacked; <= 0 counts as 1): written to *bytes, 0 when
 * the one-pass kernels run anyway.  Returns TGEMM_OK, TGEMM_ERR_NULL for a
 * NULL `bytes`, or the status a dX call would return for the dimensions. */
int ternary_gemm_dx_workspace(int64_t M, int64_t N, int64_t K, int64_t align, int64_t *bytes);

/* dW: Y[k][n] = (float(dW[k][n]) * a_col_scale[k]) * dc_col_scale[n];
 * a_col_scale float [K], dc_col_scale float [N]. */
int ternary_gemm_s8_dw_scaled(const int8_t *A, const int8_t *dC, const float *a_col_scale,
                              const float *dc_col_scale, void *dW, int out_kind,
                              int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * The steps before the product (the pages give the stored format and where
 * the activation scales go; the rules below are the readings taken).
 *
 * Packing the trainer's ternary weights [P10425 "What this adds": code
 * table; P10855 PR body: wiring the trainer is left for later]:
 *     Wpacked[n][k/4] bits 2(k%4), 2(k%4)+1  <-  code of Wt[n][k]
 * with code 1 for w > 0, 2 for w < 0, 0 for w == 0 (so {-1, 0, +1} map to
 * their codes and code 3 is never written).
 *   Wt       int8   [N][K]     (row n: the weights of output column n, the
 *                               layout of a linear layer's weight; device)
 *   Wpacked  uint8  [N][K/4]   (written, never read; device)
 * Requires N, K >= 1 and K % 4 == 0 (TGEMM_ERR_PACK); an output overlapping
 * the input returns TGEMM_ERR_ALIAS.
 */
int ternary_pack_weights(const int8_t *Wt, uint8_t *Wpacked, int64_t N, int64_t K, hipStream_t stream);

/*
 * Symmetric int8 quantization of activations, with one scale per row
 * (ternary_quantize_rows: the forward's A and dX's dC) or per column
 * (ternary_quantize_cols: dW's A and dC) [P10855 PR body, the host's
 * scales: per row for dX, per column of X and dY for dW]:
 *     s = max |x| / 127                       over the row or column
 *     q = clamp(rint(x / s), -127, 127)       (q = 0 where s == 0)
 * each step in IEEE single precision rounded to nearest even (rint: ties to
 * even).  The scale is the one the scaled calls above take, so that
 * q * s approximates x to within half a step.
 *   X      [R][C] float32 (TGEMM_IN_F32) or bfloat16 bit patterns
 *          (TGEMM_IN_BF16), finite values (device)
 *   Q      int8  [R][C] (written; device)
 *   scale  float [R] (rows) or [C] (cols) (written; device; the column
 *          variant also uses it as its running maximum, so it must not be
 *          read by other work until the call completes)
 * A NULL pointer returns TGEMM_ERR_NULL, another input kind TGEMM_ERR_KIND,
 * R or C < 1 TGEMM_ERR_DIM, overlapping buffers TGEMM_ERR_ALIAS.
 */
#define TGEMM_IN_F32 1
#define TGEMM_IN_BF16 2
int ternary_quantize_rows(const void *X, int in_kind, int8_t *Q, float *scale, int64_t R, int64_t C,
                          hipStream_t stream);
int ternary_quantize_cols(const void *X, int in_kind, int8_t *Q, float *scale, int64_t R, int64_t C,
                          hipStream_t stream);

/*
 * The operators around the product, for a block of a network whose linear
 * layers are ternary products: the norm that makes a product's int8 rows, the
 * product with its bias, activation and residual addition in one pass, their
 * backward passes, and the clipping of all gradients by their global norm.
 * In all of them
 *   - matrices are dense and row-major, their elements float32 or bfloat16
 *     bit patterns by the call's kind (TGEMM_IN_*, TGEMM_OUT_*), any width,
 *     any alignment from the element's own;
 *   - sums and statistics are float32 (the global norm's double), summed in
 *     a fixed order without atomics: repeated calls give identical bits.  The
 *     order goes by the sizes, so a row's rstd may differ in its last bits
 *     between calls with other numbers of rows (the product's outputs do not);
 *   - int8 rows and their scales are what ternary_quantize_rows would make of
 *     the float32 values before they are rounded to the kind: s = max|y| / 127,
 *     q = clamp(rint(y / s), -127, 127), q = 0 where s is 0 or not finite.  The
 *     scale of a row that holds an infinity or a NaN is not finite;
 *   - a call that needs a workspace takes caller-owned DEVICE memory, 16-byte
 *     aligned, of at least the bytes that the query beside it gives
 *     (TGEMM_ERR_WORKSPACE otherwise; where that is 0, NULL will do).  Its
 *     contents on entry do not matter; it is in use until the call completes
 *     on `stream`;
 *   - outputs overlap neither inputs nor each other nor the workspace
 *     (TGEMM_ERR_ALIAS), but for the in-place forms named below, where the
 *     two pointers are equal.
 */

/*
 * Root-mean-square norm with the residual's addition, into int8 rows:
 *     h = x + residual       rounded to the kind (h = x without a residual)
 *     rstd = 1 / sqrt(sum_c h^2 / C + eps)
 *     y = (h * rstd) * gain[c]
 * and Q, scale from y as above.
 *   X         [R][C] of in_kind
 *   residual  [R][C] of in_kind, or NULL
 *   gain      float [C]
 *   H         [R][C] of in_kind, the sum that the residual stream goes on
 *             with; needed with a residual (may be X or residual itself),
 *             NULL without
 *   Y         [R][C] of in_kind, y rounded to the kind, or NULL
 *   rstd      float [R], or NULL (the backward pass takes it)
 *   Q, scale  int8 [R][C], float [R]
 * Requires R, C >= 1 (TGEMM_ERR_DIM), a finite eps >= 0 (TGEMM_ERR_VALUE).
 * With eps = 0 a row of zeros has rstd = inf and y = NaN, as the formula does.
 */
int ternary_rmsnorm_quantize(const void *X, int in_kind, const void *residual, const float *gain, float eps,
                             void *H, void *Y, float *rstd, int8_t *Q, float *scale, int64_t R, int64_t C,
                             hipStream_t stream);

/*
 * Its backward pass, from the gradient of y (straight through the rounding
 * to int8) and, with a residual stream, the gradient dH that reaches h past
 * the norm.  With xhat = h * rstd and t = dy * gain,
 *     dX[r][c]  = rstd (t - xhat * sum_c(t xhat) / C) + dH[r][c]
 *     dgain[c]  = sum_r dy * xhat
 * dX is the gradient of x and of the residual alike.
 *   dY, H, dX  [R][C] of in_kind; rstd float [R]; gain float [C]
 *   dH         [R][C] of in_kind, or NULL; dX may be dH itself
 *   dgain      float [C] (written)
 */
int ternary_rmsnorm_backward(const void *dY, const void *H, int in_kind, const float *gain, const float *rstd,
                             const void *dH, void *dX, float *dgain, int64_t R, int64_t C, void *workspace,
                             int64_t workspace_bytes, hipStream_t stream);
int ternary_rmsnorm_backward_workspace(int64_t R, int64_t C, int64_t *bytes);

/*
 * Forward product with its epilogue, fused into the kernels' stores:
 *     z = (float(acc) * a_row_scale[m]) * w_scale + bias[n]
 *     Y[m][n] = act(z) + residual[m][n]
 * in float32 (acc the exact int32 product), each stored matrix rounded once.
 *   bias      float [N], or NULL
 *   act       TGEMM_ACT_*: relu2 is max(z, 0)^2, silu z sigmoid(z), gelu_tanh
 *             0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
 *   residual  [M][N] of out_kind, or NULL; may be Y itself
 *   Y         [M][N] of out_kind
 *   Z         [M][N] of out_kind, z for the backward pass, or NULL
 * The checks of ternary_gemm_s8_scaled, and TGEMM_ERR_VALUE for another act.
 */
#define TGEMM_ACT_NONE 0
#define TGEMM_ACT_RELU 1
#define TGEMM_ACT_RELU2 2
#define TGEMM_ACT_SILU 3
#define TGEMM_ACT_GELU_TANH 4
int ternary_gemm_s8_epilogue(const int8_t *A, const uint8_t *Wpacked, const float *a_row_scale, float w_scale,
                             const float *bias, int act, const void *residual, void *Y, void *Z, int out_kind,
                             int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * The epilogue's backward pass: from Y's gradient (which is the residual's
 * too), in one pass over dY and Z,
 *     dZ = dY * act'(Z)        rounded to the kind: ternary_quantize_cols and
 *                              ternary_gemm_s8_dw take it on to dW
 *     dbias[c] = sum_r dZ      of the unrounded values
 *     Q, scale                 the int8 rows of the unrounded dZ: the dC of
 *                              the dX calls
 * relu's slope at 0 is 0.
 *   dY, Z, dZ  [R][C] of in_kind; dbias float [C], or NULL (then no workspace
 *   is needed); Q int8 [R][C], scale float [R]
 */
int ternary_epilogue_backward(const void *dY, const void *Z, int in_kind, int act, void *dZ, float *dbias,
                              int8_t *Q, float *scale, int64_t R, int64_t C, void *workspace,
                              int64_t workspace_bytes, hipStream_t stream);
int ternary_epilogue_backward_workspace(int64_t R, int64_t C, int64_t *bytes);

/*
 * Layer norm with the residual's addition, into int8 rows, as the RMS norm:
 *     h = x + residual       rounded to the kind (h = x without a residual)
 *     mean = sum_c h / C,  rstd = 1 / sqrt(sum_c (h - mean)^2 / C + eps)
 *     y = ((h - mean) * rstd) * gain[c] + beta[c]
 * and Q, scale from y.  With eps = 0 a row of one value has rstd = inf and
 * y = NaN, as the formula does.  Arguments, checks and in-place forms are those of
 * ternary_rmsnorm_quantize, and
 *   beta        float [C], or NULL for 0
 *   mean, rstd  float [R] each, or both NULL (the backward pass takes them)
 * In float32 the mean that y and rstd are taken with is held to more than 32 bits;
 * mean[r] is its nearest float, and the backward pass takes it as given: its xhat is
 * off by up to half a step of mean[r] times rstd[r].
 */
int ternary_layernorm_quantize(const void *X, int in_kind, const void *residual, const float *gain, const float *beta,
                               float eps, void *H, void *Y, float *mean, float *rstd, int8_t *Q, float *scale,
                               int64_t R, int64_t C, hipStream_t stream);

/*
 * Its backward pass, as ternary_rmsnorm_backward.  With xhat = (h - mean) *
 * rstd and t = dy * gain,
 *     dX[r][c]  = rstd (t - sum_c(t) / C - xhat * sum_c(t xhat) / C) + dH[r][c]
 *     dgain[c]  = sum_r dy * xhat,  dbeta[c] = sum_r dy
 *   dbeta  float [C], or NULL
 */
int ternary_layernorm_backward(const void *dY, const void *H, int in_kind, const float *gain, const float *mean,
                               const float *rstd, const void *dH, void *dX, float *dgain, float *dbeta, int64_t R,
                               int64_t C, void *workspace, int64_t workspace_bytes, hipStream_t stream);
int ternary_layernorm_backward_workspace(int64_t R, int64_t C, int64_t *bytes);

/*
 * Product of int8 rows with int8 weights, a scale for each row (token) and one
 * for each column (channel), with the epilogue of ternary_gemm_s8_epilogue:
 *     z = (float(acc) * a_row_scale[m]) * w_col_scale[n] + bias[n]
 *     Y[m][n] = act(z) + residual[m][n]
 * in float32, acc[m][n] = sum_k A[m][k] * W[n][k] exact, each stored matrix
 * rounded once.  For layers that stay at 8 bits beside ternary ones (the first,
 * the head); ternary_quantize_rows makes A, W and both scales.
 *   A            int8 [M][K]
 *   W            int8 [N][K]  (row n: the weights of output column n)
 *   a_row_scale  float [M]
 *   w_col_scale  float [N], or NULL for 1
 *   bias, act, residual, Y, Z  as in ternary_gemm_s8_epilogue
 * Any K up to TGEMM_INT8_MAX_CONTRACTION (TGEMM_ERR_BOUND).  Its gradients: dX is
 * this call on dZ's int8 rows and the transposed weights, quantized row by row
 * like the weights; dW is ternary_gemm_s8_dw_scaled on both operands' columns.
 * N is at most 2^27 (TGEMM_ERR_DIM).
 * Workspace: where K is not a multiple of 16 or an operand's base not 16-byte
 * aligned, more than 64 rows need it (operands are copied into aligned rows).
 * The query takes the smallest alignment of A and W, in bytes.
 */
int ternary_gemm_s8s8_epilogue(const int8_t *A, const int8_t *W, const float *a_row_scale, const float *w_col_scale,
                               const float *bias, int act, const void *residual, void *Y, void *Z, int out_kind,
                               int64_t M, int64_t N, int64_t K, void *workspace, int64_t workspace_bytes,
                               hipStream_t stream);
int ternary_gemm_s8s8_workspace(int64_t M, int64_t N, int64_t K, int64_t align, int64_t *bytes);

/*
 * Gated product: the two projections of a gated feed-forward layer, the
 * activation and the product in one pass,
 *     g = (float(acc_g) * a_row_scale[m]) * gate_scale + bias[n]
 *     u = (float(acc_u) * a_row_scale[m]) * up_scale + bias[N + n]
 *     Y[m][n] = act(g) * u
 * in float32, acc_g and acc_u the exact ternary products with the gate's and the
 * up projection's weights, each stored matrix rounded once.
 *   A        int8 [M][K]
 *   Wpacked  uint8 [2N][K/4], stored ternary weights: the gate's N rows, then the
 *            up projection's (one matrix for the dX and dW calls)
 *   bias     float [2N], or NULL
 *   Y        [M][N] of out_kind
 *   Z        [M][2N] of out_kind, (g | u) for ternary_gated_backward, or NULL
 * The checks of ternary_gemm_s8_epilogue; N is at most 2^27 (TGEMM_ERR_DIM).
 * Workspace: more than 128 to 192 rows need one (the weights' codes are decoded
 * into it, 2 N K bytes), and so do fewer where K is not a multiple of 64 or A or
 * Wpacked not 16-byte aligned.  The query takes their smallest alignment, in bytes.
 */
int ternary_gemm_s8_gated(const int8_t *A, const uint8_t *Wpacked, const float *a_row_scale, float gate_scale,
                          float up_scale, const float *bias, int act, void *Y, void *Z, int out_kind, int64_t M,
                          int64_t N, int64_t K, void *workspace, int64_t workspace_bytes, hipStream_t stream);
int ternary_gemm_s8_gated_workspace(int64_t M, int64_t N, int64_t K, int64_t align, int64_t *bytes);

/*
 * Backward pass of the gated product (ternary_gemm_s8_gated), from Y's gradient
 * and the Z = (g | u) that it saved, in one pass over both:
 *     dg = dY * u * act'(g),  du = dY * act(g)
 *     dZ = (dg | du)           rounded to the kind, for dW of the two matrices
 *     dbias[c] = sum_r (dg | du)   of the unrounded values
 *     Q, scale                 the int8 rows of (gate_scale dg | up_scale du):
 *                              the dC of one dX call with the stored weights
 *                              of both and a weight scale of 1
 *   dY [R][C], Z and dZ [R][2C] of in_kind; dbias float [2C], or NULL (then no
 *   workspace is needed); Q int8 [R][2C], scale float [R]
 */
int ternary_gated_backward(const void *dY, const void *Z, int in_kind, int act, float gate_scale, float up_scale,
                           void *dZ, float *dbias, int8_t *Q, float *scale, int64_t R, int64_t C, void *workspace,
                           int64_t workspace_bytes, hipStream_t stream);
int ternary_gated_backward_workspace(int64_t R, int64_t C, int64_t *bytes);

/*
 * Clipping of `count` gradients by their global norm:
 *     norm = sqrt(sum over all elements of g^2)      (the sum in double)
 *     out = g * min(1, max_norm / (norm + eps))
 * The four arrays are HOST arrays, read before the call returns; the pointers
 * in them are DEVICE pointers.  Gradient i has sizes[i] >= 0 elements
 * (pointers of an empty one are not used) of kinds[i] (TGEMM_IN_*), and
 * outs[i], of the same kind, may be grads[i] itself.  `norm` is a DEVICE
 * float, and the factor is computed from it as it is stored: a norm past the
 * largest float32 is an infinity.  A norm that is not finite makes the factor 0
 * or NaN, as the formula does.
 * Requires count >= 1 and every size >= 0 (TGEMM_ERR_DIM), max_norm >= 0 and
 * eps >= 0, neither a NaN (TGEMM_ERR_VALUE).
 */
int ternary_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *sizes,
                           const int32_t *kinds, int64_t count, float max_norm, float eps, float *norm,
                           void *workspace, int64_t workspace_bytes, hipStream_t stream);
int ternary_clip_grad_norm_workspace(const int64_t *sizes, int64_t count, int64_t *bytes);

/* Static description of a status code (never NULL). */
const char *ternary_gemm_status_str(int status);

/*
 * Launch plan the library would use for a call, computed on the host without
 * touching the device (for tests and tooling).  op: 0 forward, 1 dX, 2 dW.
 * Fills the output tile (rows x cols of the row-major output computed at a
 * time by one workgroup), the number of tiles, the number of workgroups
 * launched and the most tiles any one of them computes (1 for the one-tile
 * kernels; persistent kernels loop over several), the tile columns per band
 * of the one-tile kernels' workgroup -> tile order, whether the fast
 * (vector-load) path applies given the base alignments passed in `align`
 * (the smallest power-of-two alignment of the input pointers, in bytes),
 * which kernel runs (TGEMM_KERNEL_*), and that kernel's threads and LDS bytes
 * per workgroup.  The plan is that of the calls without a workspace and
 * without an epilogue, which has ternary_gemm_epilogue_plan below.
 * Returns TGEMM_OK, or the status the real call would return for these
 * dimensions (pointer checks excepted).
 */
#define TGEMM_KERNEL_TILED 0   /* one 4-wave workgroup per output tile          */
#define TGEMM_KERNEL_SPLIT 2   /* dW, and dX with at most 256 tiles, on 128 x 144
                                  tiles: the tile's contraction split between
                                  two 4-wave halves of one workgroup          */
#define TGEMM_KERNEL_STREAM 3  /* forward (K % 64 == 0) and dX (N % 64 == 0,
                                  K % 16 == 0) on 16-byte aligned A or dC and
                                  4-byte aligned Wpacked, 32-bit offsets, at
                                  least 256 tiles of 512 x 144 (forward) or
                                  512 x 160 (dX): one persistent 8-wave
                                  workgroup per CU, operands loaded straight
                                  into LDS                                    */
#define TGEMM_KERNEL_SKINNY 4  /* forward with M <= 32, K % 64 == 0, 16-byte
                                  aligned A and Wpacked; dX with M <= 32,
                                  N % 64 == 0, K % 16 == 0, 16-byte aligned dC
                                  and Wpacked aligned for its row loads: one
                                  8-wave workgroup per 16, 32 or 64 output
                                  columns and all M rows, its waves splitting
                                  the contraction                             */
#define TGEMM_KERNEL_RING 5    /* the forward with its epilogue on mid-size
                                  outputs (K % 64 == 0, 16-byte aligned A,
                                  4-byte aligned Wpacked, 32-bit offsets): one
                                  8-wave workgroup per 128 x 128 output tile,
                                  operands loaded straight into LDS          */

#define TGEMM_KERNEL_INT8 6    /* the gated product and the product with int8
                                  weights: persistent workgroups over output
                                  tiles of one of six sizes, operands loaded
                                  straight into LDS                           */
#define TGEMM_KERNEL_INT8_FEW 7 /* the product with int8 weights of few rows:
                                  one 8- or 16-wave workgroup per 16, 32 or 64
                                  output columns and 16 or 32 rows, its waves
                                  splitting the contraction                   */

typedef struct tgemm_plan {
    int64_t out_rows, out_cols, contraction;
    int32_t tile_rows, tile_cols;
    int64_t tiles;
    int64_t workgroups;
    int64_t tiles_per_workgroup;
    int32_t band_cols;
    int32_t threads_per_workgroup;
    int32_t lds_bytes;
    int32_t fast_path;
    int32_t kernel;
    int32_t xcds;              /* XCDs of the machine planned for            */
} tgemm_plan;

int ternary_gemm_plan(int op, int64_t M, int64_t N, int64_t K, int64_t align,
                      tgemm_plan *plan);

/*
 * The same plan for a machine with `cus` compute units in `xcds` XCDs (cus a
 * multiple of xcds; TGEMM_ERR_DIM otherwise).  ternary_gemm_plan plans for
 * MI355X (256 CUs, 8 XCDs); the calls plan for the device they run on, whose
 * counts ternary_gemm_machine reports (it queries the current HIP device
 * once and keeps the answer; TGEMM_ERR_HIP if there is none).
 */
int ternary_gemm_plan_on(int op, int64_t M, int64_t N, int64_t K, int64_t align,
                         int32_t cus, int32_t xcds, tgemm_plan *plan);
int ternary_gemm_machine(int32_t *cus, int32_t *xcds);

/*
 * The plan of ternary_gemm_s8_epilogue, for a machine of cus compute units in
 * xcds XCDs (256 and 8 on MI355X): the forward's kernels, and
 * TGEMM_KERNEL_RING.
 */
int ternary_gemm_epilogue_plan(int64_t M, int64_t N, int64_t K, int64_t align, int32_t cus, int32_t xcds,
                               tgemm_plan *plan);

/*
 * The plans of ternary_gemm_s8s8_epilogue and ternary_gemm_s8_gated with these
 * arguments (align: the smallest alignment of the operands, in bytes; residual and
 * save: whether there is a residual and a Z): TGEMM_KERNEL_INT8_FEW or
 * TGEMM_KERNEL_INT8, and TGEMM_KERNEL_SKINNY (blocks of up to 32 rows) or
 * TGEMM_KERNEL_INT8.  The gated product's plan counts the product's columns, 2 N of
 * them.  fast_path: the operands' rows are read where they are (the gated product's
 * weights are decoded into the workspace by every call with TGEMM_KERNEL_INT8).
 */
int ternary_gemm_s8s8_plan(int64_t M, int64_t N, int64_t K, int64_t align, int act, int residual, int save, int out_kind,
                           int32_t cus, int32_t xcds, tgemm_plan *plan);
int ternary_gemm_s8_gated_plan(int64_t M, int64_t N, int64_t K, int64_t align, int act, int save, int out_kind, int32_t cus,
                               int32_t xcds, tgemm_plan *plan);

/*
 * Output tile that workgroup `workgroup` computes in its iteration
 * `iteration` (0 .. tiles_per_workgroup - 1) under a plan: a host mirror of
 * the kernels' own workgroup -> tile order.  That order gives each of the
 * chip's eight L2 slices (XCDs; workgroup b runs on XCD b % 8) a contiguous
 * run of tiles, row by row (inside bands of band_cols tile columns for the
 * one-tile kernels), so tiles in flight together on one XCD share input rows
 * and columns in its L2.  Writes the tile's first output row and column.
 * Returns TGEMM_OK, or TGEMM_ERR_DIM if the workgroup is out of range or
 * computes no tile in that iteration.
 */
int ternary_gemm_tile_of(const tgemm_plan *plan, int64_t workgroup, int64_t iteration,
                         int64_t *row0, int64_t *col0);

#ifdef __cplusplus
}
#endif

#endif /* TERNARY_GEMM_H */
