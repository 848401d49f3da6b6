/*
 * hlq.h - C ABI of the HLQ/HOT linear-layer backward on AMD Instinct MI355X
 * (gfx950).
 *
 * The method: "HLQ: Fast and Efficient Backpropagation via Hadamard Low-rank
 * Quantization" (Kim, Park; arXiv 2406.15102), TL;DR, and "HOT:
 * Hadamard-based Optimized Training" (HF paper page abstract; scime.ai summary,
 * section "Approach").  For y = x . w^T the backward needs
 *     g_x = g_y . w            (T x I)
 *     g_w = g_y^T . x          (O x I)
 * g_x runs through 4-bit Hadamard quantization along O; g_w through a
 * Hadamard low-rank approximation along the token dimension T followed by
 * INT8 quantization; x is kept as INT4 from the forward pass (activation
 * buffer compression, ACBP); per-token or per-tensor scales are chosen per
 * path (layer-wise quantizer selection).
 *
 * Conventions for every entry point
 *  - Data pointers are DEVICE pointers owned by the caller; the library never
 *    allocates, frees or keeps them.  Matrices are row-major and densely
 *    packed.  Every data pointer must be 16-byte aligned.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Calls only
 *    enqueue work on it and return; nothing is synchronised.  A kernel fault
 *    surfaces at the caller's next synchronisation.
 *  - Arguments are validated on the host before anything is enqueued; on an
 *    error no work is enqueued and outputs are untouched.
 *  - Thread-safe for distinct (stream, workspace) pairs.  Outputs must not
 *    alias inputs or the workspace.
 *  - Hadamard blocks are aligned and non-overlapping; the transform is the
 *    unnormalised Sylvester matrix H[i][j] = (-1)^popcount(i&j), applied with
 *    fp32 radix-2 butterflies in ascending stage order; the normalising 1/n is
 *    applied once in the GEMM epilogue.
 *  - Quantizer: symmetric absmax; for a scale group with maximum magnitude a,
 *    scale s = fl(a/qmax), code q = clamp(rne(fl(v * fl(qmax/a))), +-qmax);
 *    a == 0 gives s = 0 and all codes 0.  qmax = 7 (INT4) or 127 (INT8).
 */
#ifndef HLQ_H
#define HLQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum hlq_status {
  HLQ_OK = 0,
  HLQ_ERR_NULL = 1,      /* a required pointer is NULL                        */
  HLQ_ERR_SHAPE = 2,     /* T, I or O non-positive or not a required multiple */
  HLQ_ERR_BLOCK = 3,     /* block not in {16, 32, 64, 128}                    */
  HLQ_ERR_RANK = 4,      /* rank not a power of two in [1, block]             */
  HLQ_ERR_MODE = 5,      /* quantizer mode or reduction out of range          */
  HLQ_ERR_DTYPE = 6,     /* dtype code out of range                           */
  HLQ_ERR_ALIGN = 7,     /* a data pointer is not 16-byte aligned             */
  HLQ_ERR_OVERFLOW = 8,  /* an INT32 accumulator could overflow              */
  HLQ_ERR_WORKSPACE = 9, /* workspace NULL or smaller than required           */
  HLQ_ERR_HIP = 10,      /* the HIP runtime refused a launch                  */
  HLQ_ERR_VALUE = 11     /* a scalar argument is out of its range             */
} hlq_status;

/* Element type of g_y, w and of the forward activation x. */
enum { HLQ_F32 = 0, HLQ_BF16 = 1 };
/* Scale granularity per path (layer-wise quantizer selection, HOT). */
enum { HLQ_PER_TOKEN = 0, HLQ_PER_TENSOR = 1 };
/* Reduction of g_w: MEAN multiplies g_w by 1/T (the "1/B" of the HLQ TL;DR
   identity for g_w, read as a mean over tokens). */
enum { HLQ_SUM = 0, HLQ_MEAN = 1 };

/*
 * ACBP - activation buffer compression (HLQ TL;DR: int4 activation
 * compression; HOT summary, "Approach": stored activations compressed at
 * forward time).
 *   x        [T][I] f32 or bf16 (x_dtype), the layer input.
 *   x_codes  [T][I/2] bytes out: two's-complement INT4 codes, element 2k in
 *            bits 3:0 and element 2k+1 in bits 7:4 of byte k.
 *   x_scales [T] f32 out: one scale per token (qmax 7).
 * Requires T >= 1, I >= 8, I % 8 == 0.
 */
hlq_status hlq_compress_act(const void* x, int x_dtype, int64_t T, int64_t I,
                            uint8_t* x_codes, float* x_scales, void* stream);

/*
 * Forward product of a bf16 linear layer, y = x . w^T, with ACBP fused in
 * (HOT summary, "Approach": stored activations compressed at forward time;
 * HOT abstract: activation buffer compression): the same launch writes the
 * INT4 codes and per-token scales of x that hlq_compress_act would, without a
 * separate read of x from HBM (the first column of output tiles tracks each
 * token row's maximum |x| from the operand fragments of its MFMAs, then
 * re-reads its rows from cache for the codes).
 *   x        [T][I] bf16;  w [O][I] bf16;  I % 32 == 0.
 *   y        [T][O] out, y_dtype HLQ_F32 (fp32 sums) or HLQ_BF16 (rounded to
 *            nearest even).
 *   x_codes  [T][I/2], x_scales [T] out (both NULL: the product only);
 *            bit-identical to hlq_compress_act of x.
 */
hlq_status hlq_linear_forward(const void* x, const void* w, int64_t T, int64_t I, int64_t O,
                              void* y, int y_dtype, uint8_t* x_codes, float* x_scales,
                              void* stream);

/*
 * Bytes of device workspace hlq_linear_backward needs for this shape
 * (0 if the shape or block/rank is invalid).  Independent of modes/dtypes.
 */
size_t hlq_linear_backward_workspace_size(int64_t T, int64_t I, int64_t O,
                                          int block, int rank);

/*
 * The HLQ/HOT backward of one linear layer (HLQ TL;DR; HOT summary,
 * "Approach").
 *   g_y      [T][O] f32 or bf16 (gy_dtype), upstream gradient.
 *   x_codes  [T][I/2], x_scales [T]: the ACBP buffer of hlq_compress_act.
 *   w        [O][I] f32 or bf16 (w_dtype).
 *   block    Hadamard block n in {16, 32, 64, 128}; T % n == 0, O % n == 0.
 *   rank     r, power of two, 1 <= r <= n: rows kept per block of n tokens
 *            on the g_w path (the r lowest-sequency rows, j*n/r).
 *   gx_mode  HLQ_PER_TOKEN: one scale per token of H.g_y and per input channel
 *            of H.w; HLQ_PER_TENSOR: one scale per operand.
 *   gw_mode  HLQ_PER_TOKEN: one scale per output channel of the low-rank g_y
 *            and per input channel of the low-rank x; HLQ_PER_TENSOR: one each.
 *   reduction HLQ_SUM or HLQ_MEAN (g_w only).
 *   g_x      [T][I] f32 out = acc_x * s_gy * s_w / n.
 *   g_w      [O][I] f32 out = acc_w * s_gyl * s_xl / n  (/ T for MEAN).
 *   workspace device buffer of at least hlq_linear_backward_workspace_size()
 *            bytes; holds the quantized operands and scales afterwards (layout
 *            from hlq_workspace_layout).
 * Also requires I % 8 == 0 (stricter than the even I that nibble packing
 * alone needs: every kernel moves a row's codes in whole 32-bit words of 8
 * codes, so rows never split a word; HLQ_ERR_SHAPE otherwise) and that no
 * accumulator can lose exactness: O <= 342391 (49 * O < 2^24, the fp32 sums of
 * the FP6 g_x product) and T*rank/block <= 133143 (127^2 * T' < 2^31, INT32).
 */
hlq_status hlq_linear_backward(const void* g_y, int gy_dtype,
                               const uint8_t* x_codes, const float* x_scales,
                               const void* w, int w_dtype,
                               int64_t T, int64_t I, int64_t O,
                               int block, int rank,
                               int gx_mode, int gw_mode, int reduction,
                               float* g_x, float* g_w,
                               void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * hlq_linear_backward for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, no workspace.  The intermediates go to a static
 * device array owned by the library, HLQ_NOALLOC_SCRATCH_BYTES on each GPU the
 * library runs on, held until the process ends; the call allocates and frees
 * nothing.  Its first call on a device resolves that device's copy of the
 * array (hipGetSymbolAddress, a runtime query; make one call before any graph
 * capture).  A shape whose intermediates do not fit (the workspace of
 * hlq_linear_backward_workspace_size less its split-K partial region, which
 * this call never uses) returns HLQ_ERR_WORKSPACE before anything is
 * enqueued.  All calls on one GPU share its array: calls that can overlap on
 * one GPU (other streams, other host threads) race and must be serialised by
 * the caller.  Each call writes every intermediate before reading it, so the
 * array needs no clearing between calls.
 */
#define HLQ_NOALLOC_SCRATCH_BYTES (64u << 20)
hlq_status hlq_linear_backward_noalloc(const void* g_y, int gy_dtype,
                                       const uint8_t* x_codes, const float* x_scales,
                                       const void* w, int w_dtype,
                                       int64_t T, int64_t I, int64_t O,
                                       int block, int rank,
                                       int gx_mode, int gw_mode, int reduction,
                                       float* g_x, float* g_w, void* stream);

/*
 * The launches hlq_linear_backward enqueues, in order.  Bit k of a step mask
 * selects HLQ_STEP k.
 */
enum {
  HLQ_STEP_TR_MAX = 0,     /* partial maxima of H.g_y (along O), the low-rank
                              g_y and x (along T) and H.w (along O)          */
  HLQ_STEP_TR_REDUCE = 1,  /* fold partials: per-token maxima, scales,
                              tensor maxima                                  */
  HLQ_STEP_TR_QUANT = 2,   /* transforms again -> INT4 / INT8 GEMM operands  */
  HLQ_STEP_GEMM_GX = 3,    /* INT4 GEMM + dequantizing epilogue -> g_x       */
  HLQ_STEP_GEMM_GW = 4,    /* INT8 GEMM + dequantizing epilogue -> g_w       */
  HLQ_STEP_COUNT = 5
};
#define HLQ_STEPS_ALL 0x1Fu

/*
 * hlq_linear_backward restricted to the steps whose bit is set in step_mask
 * (same arguments, same validation).  All steps in one call equal
 * hlq_linear_backward.  A subset re-runs those launches on a workspace that
 * the earlier steps have filled (every step is idempotent given its inputs),
 * which lets a caller time or inspect one kernel of the sequence in place.
 * The GEMM steps read what the QUANT step last wrote to the workspace,
 * including the arrival counters of the K-split g_w tiles it clears.
 */
hlq_status hlq_linear_backward_steps(const void* g_y, int gy_dtype,
                                     const uint8_t* x_codes, const float* x_scales,
                                     const void* w, int w_dtype,
                                     int64_t T, int64_t I, int64_t O,
                                     int block, int rank,
                                     int gx_mode, int gw_mode, int reduction,
                                     float* g_x, float* g_w,
                                     void* workspace, size_t workspace_bytes,
                                     uint32_t step_mask, void* stream);

/*
 * Where hlq_linear_backward leaves its intermediates inside the workspace
 * (byte offsets), for tests and diagnostics.
 * The four code operands are matrices of `rows` rows whose K run is pitch
 * bytes per row, stored in K planes of U bytes: plane p (p = 0 ..
 * pitch/U - 1) holds bytes [p*U, (p+1)*U) of every row's run, row after row,
 * so byte k of row m is at (k / U) * rows * U + m * U + k % U.  U = 96 for
 * q_gy and q_w, 64 for q_gyl and q_xl.
 *   q_gy   T rows, kx_pitch bytes: INT4 codes of H.g_y (along O), stored as
 *          FP6 E2M3 fields (exact for -7..7: sign bit 5, exponent bits 4-3
 *          with bias 1, mantissa bits 2-0) in groups of 128 codes (96 bytes,
 *          one plane): quarter Q of a group (codes 32Q .. 32Q+31) is a
 *          24-byte stream, code j at bits 6j .. 6j+5, and the quarters are
 *          stored in the order 0, 2, 1, 3.  Codes past O are zero fields
 *          (kx_pitch = 96 * ceil(O / 128)).
 *   s_gy   [T] (PER_TOKEN) or [1] f32.
 *   q_w    I rows, kx_pitch bytes: INT4 codes of H.w, transposed (K = O), in
 *          the same FP6 groups.
 *   s_w    [I] or [1] f32.
 *   q_gyl  O rows, kw_pitch bytes: INT8 codes of the low-rank g_y, transposed
 *          (K = T'), zero past T' = T*rank/block.
 *   s_gyl  [O] or [1] f32.
 *   q_xl   I rows, kw_pitch bytes: INT8 codes of the low-rank x, transposed.
 *   s_xl   [I] or [1] f32.
 *   partial  scratch of the split-K GEMMs (contents unspecified).
 * The workspace also holds, after these, the INT32 partial sums and arrival
 * counters of the K-split g_w tiles of the pair launch (contents unspecified).
 */
typedef struct hlq_workspace_layout {
  size_t q_gy, s_gy, q_w, s_w, q_gyl, s_gyl, q_xl, s_xl;
  int64_t kx_pitch;  /* K bytes per row of q_gy and q_w (96-byte planes)  */
  int64_t kw_pitch;  /* K bytes per row of q_gyl and q_xl (64-byte planes) */
  int64_t t_low;     /* T' = T * rank / block           */
  size_t total;      /* == hlq_linear_backward_workspace_size() */
  size_t partial;    /* INT32 split-K partial sums shared by both GEMMs */
  size_t partial_bytes;
  int32_t gx_splits; /* split-K factor of the g_x GEMM (1 = none) */
  int32_t gw_splits; /* split-K factor of the g_w GEMM            */
} hlq_workspace_layout;

hlq_status hlq_workspace_layout_query(int64_t T, int64_t I, int64_t O, int block,
                                      int rank, hlq_workspace_layout* out);

/*
 * INT32 accumulators of the two integer GEMMs, recomputed from a workspace
 * that hlq_linear_backward has filled (tests and diagnostics; HLQ TL;DR:
 * "int8-accelerated" products).  acc_x [T][I] = sum_o q_gy[t,o] q_w[o,i];
 * acc_w [O][I] = sum_t' q_gyl[t',o] q_xl[t',i].
 *   hlq_gemm_pair_acc: the one launch hlq_linear_backward runs for both
 *     GEMMs (same tile grids, K splits and schedule), its epilogue storing
 *     the INT32 sums instead of the fp32 gradients.  It writes the
 *     workspace's split-K partial sums and arrival counters (the codes and
 *     scales are only read), hence the non-const workspace.
 *   hlq_gemm_gx_acc / hlq_gemm_gw_acc: the single-GEMM launches that
 *     hlq_linear_backward_steps runs when only one GEMM step is selected.
 * workspace_bytes is checked against hlq_linear_backward_workspace_size
 * (HLQ_ERR_WORKSPACE); acc_* are device buffers of the sizes above.
 */
hlq_status hlq_gemm_pair_acc(void* workspace, size_t workspace_bytes, int64_t T, int64_t I,
                             int64_t O, int block, int rank, int32_t* acc_x, int32_t* acc_w,
                             void* stream);
hlq_status hlq_gemm_gx_acc(const void* workspace, size_t workspace_bytes, int64_t T,
                           int64_t I, int64_t O, int block, int rank, int32_t* acc_x,
                           void* stream);
hlq_status hlq_gemm_gw_acc(const void* workspace, size_t workspace_bytes, int64_t T,
                           int64_t I, int64_t O, int block, int rank, int32_t* acc_w,
                           void* stream);

/*
 * The HLQ/HOT backward of one 2-D convolution (HLQ abstract: backpropagation
 * of convolutional and linear layers; HOT summary, "Key results": ResNet-50
 * at batch 256), as implicit GEMMs: no im2col or col2im buffer.
 *   y[n,p,q,o] = sum_{r,s,c} x[n, p*stride - pad + r, q*stride - pad + s, c]
 *                * w[o,r,s,c]   (zero padding; P = (H + 2 pad - R)/stride + 1,
 *                                Q = (W + 2 pad - S)/stride + 1)
 * is the linear layer y = im2col(x) . w^T with tokens t = (n, p, q) and
 * features i = (r*S + s)*C + c; the backward is that layer's (same
 * transforms, quantizers, codes and g_w), with the g_w path's low-rank x
 * gathered from the ACBP codes of x itself and g_x the sum over the taps
 * that read each input pixel (col2im).
 *   g_y      [N][P][Q][O] f32 or bf16.
 *   x_codes, x_scales: hlq_compress_act of x viewed as [N*H*W][C] (one scale
 *            per pixel).
 *   w        [O][R][S][C] f32 or bf16.
 *   g_x      [N][H][W][C] f32 out = s_gy * s_w / n * sum over taps and O of
 *            the INT4 code products (an implicit GEMM over the taps).
 *   g_w      [O][R][S][C] f32 out, as hlq_linear_backward's g_w.
 * Requires C % 8 == 0, N*P*Q and O multiples of block, gx_mode ==
 * HLQ_PER_TENSOR (HLQ_ERR_MODE otherwise: per-token scales of H.g_y and H.w
 * do not factor out of the sum over the taps), O*R*S <= 342391 and
 * T' = N*P*Q*rank/block <= 133143 (HLQ_ERR_OVERFLOW), pixel and position
 * counts below 2^31.  workspace: hlq_conv_backward_workspace_size bytes.
 * Launches: the transform MAX, reduce and QUANT passes, the INT8 g_w GEMM
 * (with split-K partials when its grid is small), the INT4 input-gradient GEMM.
 */
size_t hlq_conv_backward_workspace_size(int64_t N, int64_t H, int64_t W, int64_t C, int64_t O,
                                        int R, int S, int stride, int pad, int block,
                                        int rank);
hlq_status hlq_conv_backward(const void* g_y, int gy_dtype, const uint8_t* x_codes,
                             const float* x_scales, const void* w, int w_dtype, int64_t N,
                             int64_t H, int64_t W, int64_t C, int64_t O, int R, int S,
                             int stride, int pad, int block, int rank, int gx_mode,
                             int gw_mode, int reduction, float* g_x, float* g_w,
                             void* workspace, size_t workspace_bytes, void* stream);
/*
 * INT32 accumulators of the convolution backward's two GEMMs from a workspace
 * hlq_conv_backward has filled (tests): acc_x [N*H*W][C] (sums over taps and
 * O, before the per-tensor scales), acc_w [O][R*S*C].
 */
hlq_status hlq_conv_gemm_acc(const void* workspace, size_t workspace_bytes, int64_t N,
                             int64_t H, int64_t W, int64_t C, int64_t O, int R, int S,
                             int stride, int pad, int block, int rank, int32_t* acc_x,
                             int32_t* acc_w, void* stream);

/*
 * Ablation variants: the backward with another transform / quantizer on
 * either path, for synthetic error studies (HOT summary, "Measured effects":
 * the ResNet50 ablation rows; "Surprising findings": internal and external
 * Hadamard low-rank approximation on the activation-gradient path,
 * quantization sensitivity of the weight-gradient path).  Each path is one
 * integer GEMM over its contracted dimension K (O for g_x, T for g_w):
 *   HLQ_VAR_HQ4       block Hadamard along K on both operands, INT4 (the
 *                     method's g_x path);
 *   HLQ_VAR_Q4        no transform, INT4;
 *   HLQ_VAR_HLA8_INT  low-rank rows j*n/r of the block Hadamard along K on
 *                     both operands ("internal" HLA), INT8 (the method's g_w
 *                     path);
 *   HLQ_VAR_HLA8_EXT  low-rank Hadamard along the left operand's output
 *                     dimension (T for g_x, O for g_w: "external" HLA), none
 *                     on the right operand, INT8; the r rows per block of the
 *                     product are expanded back to n by H_low^T / n.
 * The pages list HLA without a quantizer; HOT pairs it with INT8, as here.
 * Scale groups and modes as hlq_linear_backward.  Plain kernels, one thread
 * per block of n source values, then the library's INT8 GEMM (INT4 codes are
 * stored one per byte): not the hot path.  acc_x [T or T*r/n][I] and acc_w
 * [O or O*r/n][I] (device, may be NULL) receive the GEMMs' INT32 sums.
 * Errors as hlq_linear_backward; HLQ_ERR_MODE for an unknown variant.
 */
enum { HLQ_VAR_HQ4 = 0, HLQ_VAR_Q4 = 1, HLQ_VAR_HLA8_INT = 2, HLQ_VAR_HLA8_EXT = 3 };
size_t hlq_ablation_workspace_size(int64_t T, int64_t I, int64_t O, int block, int rank,
                                   int gx_variant, int gw_variant);
hlq_status hlq_linear_backward_ablation(const void* g_y, int gy_dtype, const uint8_t* x_codes,
                                        const float* x_scales, const void* w, int w_dtype,
                                        int64_t T, int64_t I, int64_t O, int block, int rank,
                                        int gx_variant, int gw_variant, int gx_mode,
                                        int gw_mode, int reduction, float* g_x, float* g_w,
                                        int32_t* acc_x, int32_t* acc_w, void* workspace,
                                        size_t workspace_bytes, void* stream);

/*
 * Layer-wise quantizer selection (LQS).  "HOT: Hadamard-based Optimized
 * Training": HF page abstract (layer-wise quantizer selection), scime.ai
 * summary "Approach" (per-token vs per-tensor chosen per layer) and
 * "Limitations" (chosen from a calibration set with a 50% MSE-difference
 * threshold).  The pages name the threshold, not the error measure; the
 * reading taken here: the squared reconstruction error of each quantized
 * GEMM operand under each mode.
 *
 * hlq_lqs_accumulate adds one calibration batch (the same inputs as
 * hlq_linear_backward) to `stats`, a DEVICE array of 16 doubles the caller
 * zeroes once and keeps across batches.  For operand k = 0 (H.g_y along O,
 * INT4), 1 (H.w along O, INT4), 2 (low-rank g_y along T, INT8), 3 (low-rank
 * x along T, INT8), with v the fp32 transformed values of the backward:
 *   stats[4k]   += sum v^2
 *   stats[4k+1] += sum e^2 with PER_TOKEN scales (one per group of reading R6)
 *   stats[4k+2] += sum e^2 with a PER_TENSOR scale
 *   stats[4k+3] += number of elements
 * where e = fl32(v - fl32(s * q)) with the code q and scale s the backward's
 * quantizer gives v; e^2 and the sums are fp64 (fixed summation order, so a
 * call is reproducible).  Five launches on `stream`: the backward's MAX and
 * reduce launches with both paths per token (group and tensor maxima,
 * scales), two error passes (row and column operands) and a fixed-order
 * fold.  The workspace (at least
 * hlq_lqs_workspace_size bytes) holds the backward's workspace regions
 * followed by per-workgroup partial sums.  Shape
 * rules and errors as for hlq_linear_backward; `stats` must be 16-byte
 * aligned; HLQ_ERR_OVERFLOW also when g_y, w or the ACBP codes hold 4 GiB or
 * more (the statistics kernels use 32-bit byte offsets).
 *
 * hlq_lqs_select is a host function on a HOST copy of the 16 statistics.
 * A path's error in a mode is the sum over its two operands of
 * SSE / sum v^2 (0 for an all-zero operand).  The path takes HLQ_PER_TOKEN
 * when its per-tensor error exceeds (1 + threshold) times its per-token
 * error, else HLQ_PER_TENSOR (the single-scale quantizer).  The pages'
 * threshold is 0.5.  Errors: HLQ_ERR_NULL, HLQ_ERR_MODE (threshold negative
 * or NaN).
 */
size_t hlq_lqs_workspace_size(int64_t T, int64_t I, int64_t O, int block, int rank);
hlq_status hlq_lqs_accumulate(const void* g_y, int gy_dtype, const uint8_t* x_codes,
                              const float* x_scales, const void* w, int w_dtype,
                              int64_t T, int64_t I, int64_t O, int block, int rank,
                              double* stats, void* workspace, size_t workspace_bytes,
                              void* stream);
hlq_status hlq_lqs_select(const double* stats, double threshold, int* gx_mode,
                          int* gw_mode);

/* ------------------------------------------------------------------------
 * Operators of a training step around the linear layer: layer norm, token log
 * probabilities with the policy and preference losses on them, and gradient
 * clipping by the global norm.
 *
 * They follow the conventions above with two differences.  Data pointers need
 * the alignment of their elements only (rows of odd length, and views into a
 * packed buffer, start anywhere); the workspace still needs 16 bytes.  A
 * count of rows, tokens or tensors may be zero, and the pointers of the
 * operands that are then empty may be NULL.  Every sum is kept in fp32 or
 * fp64 in an order fixed by the sizes and, for rows of logits, by where in 16
 * bytes a row starts, so results are reproducible; an output in bf16 is rounded
 * once, to nearest even.
 * ------------------------------------------------------------------------ */

/*
 * Layer norm over the last dimension, with the residual addition in front.
 *   h = x + residual, rounded to the type of x   (h = x without residual)
 *   mean = 1/C sum_c h_c,   rstd = (1/C sum_c (h_c - mean)^2 + eps)^(-1/2)
 *   y = (h - mean) * rstd * weight + bias
 *   x, residual  [T][C] f32 or bf16 (dtype); residual NULL: none.
 *   weight, bias [C] f32 or bf16 (param_dtype); bias NULL: none.
 *   y            [T][C] out, dtype.
 *   h            [T][C] out, dtype: the sum, for the residual stream and the
 *                backward pass; NULL exactly when residual is.
 *   mean, rstd   [T] f32 out, for the backward pass.
 * Statistics are fp32, the squares of the differences to the mean included: they
 * pass its range where a row's values lie more than 2^63 apart.
 * One launch.  Errors: HLQ_ERR_NULL, HLQ_ERR_DTYPE, HLQ_ERR_SHAPE (T < 0,
 * C < 1, T or C >= 2^31), HLQ_ERR_VALUE (eps negative or not finite),
 * HLQ_ERR_ALIGN.
 */
hlq_status hlq_layer_norm_forward(const void* x, const void* residual, int dtype,
                                  const void* weight, const void* bias, int param_dtype,
                                  int64_t T, int64_t C, double eps, void* y, void* h,
                                  float* mean, float* rstd, void* stream);

/*
 * Backward of the layer norm.  With n = (h - mean) * rstd and u = g_y * weight,
 *   g_x      = rstd * (u - 1/C sum_c u - n * 1/C sum_c u n) + g_h
 *   g_weight = sum_t g_y * n,   g_bias = sum_t g_y
 * g_x is the gradient of x and of residual alike.
 *   g_y      [T][C] dtype, the gradient of y.
 *   h        [T][C] dtype, the normalised input (x itself without residual).
 *   g_h      [T][C] dtype, the gradient that reaches h along the residual
 *            stream; NULL: none.
 *   mean, rstd [T] f32, from the forward call.
 *   g_x      [T][C] out, dtype.
 *   g_weight, g_bias [C] out, param_dtype; g_bias NULL: not computed.
 *   workspace at least hlq_layer_norm_backward_workspace_size(T, C, dtype)
 *            bytes: per-workgroup column sums (0 for an invalid shape).
 * Two launches, one for a few rows.  Errors as above and HLQ_ERR_WORKSPACE.
 */
size_t hlq_layer_norm_backward_workspace_size(int64_t T, int64_t C, int dtype);
hlq_status hlq_layer_norm_backward(const void* g_y, const void* h, const void* g_h, int dtype,
                                   const float* mean, const float* rstd, const void* weight,
                                   int param_dtype, int64_t T, int64_t C, void* g_x,
                                   void* g_weight, void* g_bias, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * Log probability of one target per row of logits.  With z = scale * logits,
 *   logprob[t] = z[t][target] - log sum_v exp(z[t][v])
 *   stats[t]   = (max_v logits[t][v], sum_v exp(z[t][v] - max_v z[t][v]))
 *   logits   T rows of V elements, dtype, row t at element t * ld (ld >= V).
 *   targets  [T] int64; one outside [0, V) is ignored: its row is not read,
 *            logprob is 0 and stats (0, 1).  The losses on log probabilities do
 *            not see targets: to them such a token is one of probability 1 until
 *            its weight is 0.
 *   scale    the inverse temperature, 2^-64 to 2^64.
 *   logprob  [T] f32 out;  stats [T][2] f32 out, for the backward pass.
 * Logits of -inf have probability zero; a row of nothing else has logprob
 * -inf and stats (-inf, 0).  A NaN or +inf in a row makes its logprob NaN.
 * Errors: HLQ_ERR_NULL, HLQ_ERR_DTYPE, HLQ_ERR_SHAPE (T < 0, V < 1, ld < V,
 * T >= 2^31, V >= 2^30), HLQ_ERR_VALUE (scale), HLQ_ERR_ALIGN.
 */
hlq_status hlq_token_logprob_forward(const void* logits, int dtype, int64_t ld,
                                     const int64_t* targets, int64_t T, int64_t V, double scale,
                                     float* logprob, float* stats, void* stream);

/*
 * Gradient of the logits from that of the log probabilities,
 *   g_x[t][v] = g_logprob[t] * scale * ([v == target] - softmax(z[t])[v]),
 * the softmax taken from stats.
 *   g_logprob [T] f32.  Rows whose g_logprob is zero, whose target is ignored
 *            or which hold nothing but -inf get zeros, and are not read.  An
 *            infinite one gives zero where the factor in brackets is zero.
 *   g_x      T rows of V elements out, dtype, row t at element t * g_ld; may be
 *            logits itself (g_ld = ld), no other overlap.
 * One launch.  Errors as above (HLQ_ERR_SHAPE also for g_ld < V).
 */
hlq_status hlq_token_logprob_backward(const float* g_logprob, const void* logits, int dtype,
                                      int64_t ld, const int64_t* targets, const float* stats,
                                      int64_t T, int64_t V, double scale, void* g_x,
                                      int64_t g_ld, void* stream);

/*
 * Clipped policy loss with a KL term, from log probabilities:
 *   r_t = exp(logprob - old),   d_t = ref - logprob
 *   loss = sum_t w_t (kl_coef * (exp(d_t) - d_t - 1)
 *                     - min(r_t A_t, clamp(r_t, 1 - clip_low, 1 + clip_high) A_t))
 *   logprob, old_logprob, advantage [T] f32.
 *   weight   [T] f32: 0 takes a token out, whatever its other values are (1/n
 *            for a mean over n tokens); NULL: every token has weight 1.
 *   ref_logprob [T] f32 of the reference policy; NULL exactly when kl_coef is
 *            0.  Only logprob has a gradient.
 *   sums     [3] f32 out: the loss, sum_t w_t (exp(d_t) - d_t - 1), and the
 *            weight of the tokens whose clamped term was the smaller one.
 *   g_logprob [T] f32 out, the gradient of the loss.
 *   workspace at least hlq_policy_loss_workspace_size(T) bytes.
 * A logprob of -inf (a banned target) has the ratio 0; with a KL term the loss
 * and its estimate are then +inf and the gradient -inf, as the formula's limits
 * are.  A reference of -inf makes the loss +inf and leaves the gradient finite.
 * An advantage of 0 adds nothing, however large the ratio.  NaN where logprob and
 * old_logprob, or logprob and a reference that counts, are both -inf: such
 * tokens are taken out by their weight.
 * clip_low in [0, 1], clip_high >= 0, kl_coef >= 0, all finite
 * (HLQ_ERR_VALUE).  Two launches.
 */
size_t hlq_policy_loss_workspace_size(int64_t T);
hlq_status hlq_policy_loss(const float* logprob, const float* old_logprob,
                           const float* advantage, const float* weight,
                           const float* ref_logprob, int64_t T, double clip_low,
                           double clip_high, double kl_coef, float* sums, float* g_logprob,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * hlq_token_logprob_forward, hlq_policy_loss and hlq_token_logprob_backward
 * in one pass over the logits, with one difference: a token whose target is
 * ignored does not count, as if its weight were 0 (the three calls need the
 * weight for that).
 *   logprob  [T] f32 out; 0 where the weight is 0 or the target is ignored
 *            (such a token does not count in the loss, its row is not read).
 *   g_x      T rows of V elements out: the gradient of the loss; may be logits
 *            itself (g_ld = ld), no other overlap.
 * The other arguments, the workspace and the errors as there.
 */
hlq_status hlq_policy_loss_logits(const void* logits, int dtype, int64_t ld,
                                  const int64_t* targets, const float* old_logprob,
                                  const float* advantage, const float* weight,
                                  const float* ref_logprob, int64_t T, int64_t V, double scale,
                                  double clip_low, double clip_high, double kl_coef,
                                  float* sums, float* logprob, void* g_x, int64_t g_ld,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Preference loss over P pairs of sequences, from log probabilities:
 *   s_q      = sum over the tokens of sequence q of w_t (logprob_t - ref_t)
 *              (HLQ_MEAN: divided by sum w_t, 0 where that is not positive)
 *   margin_p = beta (s_p - s_{P+p})
 *   loss     = 1/P sum_p -(1 - e) log sigmoid(margin_p) - e log sigmoid(-margin_p)
 * with e = label_smoothing.
 *   logprob  [T] f32; ref_logprob [T] f32 or NULL (no reference policy).
 *   weight   [T] f32 or NULL (ones); 0 takes a token out, whatever its values.
 *            Ignored targets (log probability 0) have to be taken out that way:
 *            they count in a sequence's length under HLQ_MEAN, and their
 *            reference in its score.
 *            A token of logprob -inf (a banned target) makes the score of its
 *            sequence -inf and the margin -inf or +inf: the loss then has the
 *            limit's value (0 for a margin of +inf without smoothing), the
 *            gradient is finite.  Where the reference gives it -inf too, or both
 *            sequences of a pair hold one, the margin is NaN.
 *   start    [2P + 1] int64, non-decreasing within 0 to T: sequence q is tokens
 *            start[q] .. start[q+1] - 1; the chosen ones are 0 .. P-1, the
 *            rejected ones P .. 2P-1 in the same order.  Read on the device
 *            and limited to [0, T] there; tokens before start[0] or from
 *            start[2P] on belong to no sequence, and their gradient is zero.
 *   loss     [1] f32, margin [P] f32, g_logprob [T] f32 out.
 *   workspace at least hlq_preference_loss_workspace_size(P) bytes.
 * beta > 0 and finite, 0 <= label_smoothing <= 1 (HLQ_ERR_VALUE), reduction
 * HLQ_SUM or HLQ_MEAN (HLQ_ERR_MODE), 1 <= P < 2^24 and T < 2^31
 * (HLQ_ERR_SHAPE).
 */
size_t hlq_preference_loss_workspace_size(int64_t P);
hlq_status hlq_preference_loss(const float* logprob, const float* ref_logprob,
                               const float* weight, const int64_t* start, int64_t P, int64_t T,
                               double beta, double label_smoothing, int reduction, float* loss,
                               float* margin, float* g_logprob, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Clipping of gradients by their global norm:
 *   norm = (sum of v^2)^(1/2)   (HLQ_NORM_L2)   or   max |v|   (HLQ_NORM_INF)
 *   out  = grad * min(1, max_norm / (norm + 1e-6))
 * over all elements v of all tensors.  Nothing is read back by the host.
 *   grads, outs [count] host arrays of device pointers; outs NULL: in place.
 *            outs[i] may equal grads[i]; no other overlap.  Read during the
 *            call only.
 *   sizes    [count] elements of each tensor (0 allowed).
 *   dtypes   [count] HLQ_F32 or HLQ_BF16, of grads[i] and outs[i].
 *   max_norm >= 0 (HLQ_ERR_VALUE); +inf leaves gradients of finite norm alone.
 *   norm     [1] f64 out (device).
 *   workspace at least hlq_clip_grad_norm_workspace_size(sizes, count) bytes.
 * An infinite norm gives the factor 0 (NaN where the gradient is infinite), a
 * NaN in a gradient makes the norm and every output NaN.  One launch for the
 * norm and one for the scaling per 160 tensors (a tensor of more than 2^30
 * elements counts once per 2^30).
 */
enum { HLQ_NORM_L2 = 0, HLQ_NORM_INF = 1 };
size_t hlq_clip_grad_norm_workspace_size(const int64_t* sizes, int64_t count);
hlq_status hlq_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes,
                              const int* dtypes, int64_t count, double max_norm, int norm_kind,
                              double* norm, void* workspace, size_t workspace_bytes,
                              void* stream);

/* ------------------------------------------------------------------------
 * Operators of an attention block between its linear layers: attention over
 * packed sequences with a learned relative position bias, and dropout in front
 * of the residual addition.  Conventions as for the operators above: data
 * pointers need the alignment of their elements, counts of tokens may be zero,
 * results are reproducible.
 * ------------------------------------------------------------------------ */

/* A tensor [tokens][heads][head_dim], head_dim elements dense, strides in
   elements and not negative: a slice of what the qkv layer wrote, or of the
   gradient it will read.  Tokens are less than 2^22 elements apart, heads less than
   2^40 (a single token's or head's stride may be anything).  An input's strides may
   be 0; outputs must not overlap themselves, each other or what the call reads (slices
   that lie between each other are fine).  One that starts where another operand does, in
   whose place it would give wrong results, is refused (HLQ_ERR_VALUE). */
typedef struct hlq_tokens {
  void* data;
  int64_t token_stride, head_stride;
} hlq_tokens;

/*
 * What one attention call deals with.  Sequence s has the queries start_q[s] ..
 * start_q[s+1] - 1 and the keys start_k[s] .. start_k[s+1] - 1 of the packed
 * tensors (the bounds [sequences + 1] int64, non-decreasing, read on the device and
 * limited there to the tokens there are; tokens before the first and behind the
 * last sequence get zeros).  start_q NULL: one sequence of all tokens; start_k
 * NULL: start_q, for as many keys as queries.  Query i of Lq stands at position
 * i + Lk - Lq of its sequence's Lk keys, so that new tokens follow those of a
 * cache.  Lengths may be zero.
 *   max_len   the longest sequence's queries, for the launch alone (0: unknown);
 *             longer ones are dealt with all the same.  Not looked at without bounds.
 *             A launch has that many queries' tiles in every sequence, up to 16 times
 *             what the tokens can need, and a bias's gradient [buckets] f32 of workspace
 *             for each tile and head.
 *   heads     query heads; head h reads key head h / (heads / kv_heads).
 *   head_dim  1 to 128.
 *   causal    a query sees the keys up to its own position.
 *   scale     2^-64 to 2^64.
 *   bias      [buckets][heads] of bias_dtype or NULL: added to scale * q k, by the
 *             bucket of d = key position - query position (hlq_relative_bucket).
 *             Entries below -2^127 * 1.4 (the types' lowest values among them) hide
 *             their bucket as -inf does.
 * Fewer than 2^30 queries times heads and keys times heads, 2^16 heads.
 */
typedef struct hlq_attention {
  int64_t queries, keys, sequences, max_len;
  const int64_t *start_q, *start_k;
  const void* bias;
  double scale;
  int32_t dtype, heads, kv_heads, head_dim, causal;
  int32_t bias_dtype, buckets, max_distance, bidirectional;
} hlq_attention;

/*
 * Bucket of a distance d (a host function; -1 for sizes out of range).  A side has
 * n = buckets distances (bidirectional: buckets / 2, and those of d > 0 come after
 * the others), e = n / 2 of them by themselves:
 *   a = |d| (one side: max(-d, 0));   bucket = a for a < e, else
 *   min(n - 1, e + floor((n - e) log(a / e) / log(max_distance / e)))
 * 2 <= n, buckets <= 128 and even if bidirectional, e < max_distance <= 1024.
 */
int hlq_relative_bucket(int distance, int buckets, int max_distance, int bidirectional);

/*
 * Attention:  S_ij = scale q_i k_j + bias,  lse_i = log sum_j exp(S_ij),
 *   o_i = sum_j exp(S_ij - lse_i) v_j      over the keys j that query i sees.
 *   q, o     [queries][heads][head_dim], k, v [keys][kv_heads][head_dim], dtype.
 *   lse      [heads][queries] f32 out, for the backward pass.
 *   workspace at least hlq_attention_forward_workspace_size(a) bytes (0 unless
 *            there are too few queries to fill the GPU: then the keys are shared out).
 * A query that sees no key, or none with a score above -inf, gets o = 0 and lse =
 * -inf.  Keys and values that a query does not see do not reach it, infinities and
 * NaN among them included; one that it does see makes its row infinite or NaN,
 * in elements that are not specified (none of them, if only scores of -inf come of
 * it).  Scores, sums and statistics are fp32; for bf16 the
 * probabilities are rounded to bf16 in the product with v.
 * One launch, two with a workspace.  Errors: HLQ_ERR_NULL, HLQ_ERR_DTYPE,
 * HLQ_ERR_SHAPE, HLQ_ERR_VALUE (scale, buckets, places), HLQ_ERR_ALIGN,
 * HLQ_ERR_WORKSPACE.
 */
size_t hlq_attention_forward_workspace_size(const hlq_attention* a);
hlq_status hlq_attention_forward(const hlq_attention* a, const hlq_tokens* q, const hlq_tokens* k,
                                 const hlq_tokens* v, const hlq_tokens* o, float* lse,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * Its backward pass.  The probabilities P_ij = exp(S_ij - lse_i) are computed
 * again:  D_i = sum_d g_o o (o as stored),  G_ij = P_ij (g_o_i v_j - D_i),
 *   g_q_i = scale sum_j G_ij k_j,  g_k_j = scale sum_i G_ij q_i,
 *   g_v_j = sum_i P_ij g_o_i (the last two over the query heads that share a key
 *   head),  g_bias[b][h] = sum of G over the pairs of head h in bucket b.
 *   g_o      [queries][heads][head_dim]; q, k, v, o, lse of the forward call.
 *   g_q, g_k, g_v  out, dtype;  g_bias [buckets][heads] out, bias_dtype, NULL
 *            exactly when there is no bias.
 * For bf16 P and G are rounded to bf16 in the products for g_k and g_v; that for g_q
 * takes G as two bf16 numbers, and g_bias sums G unrounded.  D_i differs from that of
 * the o before its rounding by up to 2^-8 sum_d |g_o o|, and then the sum of a row's G is
 * not zero: a part c that all keys share leaves up to scale |c| times that in g_q.
 * Infinities and NaN reach the gradients of what they meet in a pair that is seen,
 * in elements that are not specified, and no others.
 * Two launches, three with a bias.  No atomics: a call repeats bit for bit.
 * Errors as above.
 */
size_t hlq_attention_backward_workspace_size(const hlq_attention* a);
hlq_status hlq_attention_backward(const hlq_attention* a, const hlq_tokens* g_o,
                                  const hlq_tokens* q, const hlq_tokens* k, const hlq_tokens* v,
                                  const hlq_tokens* o, const float* lse, const hlq_tokens* g_q,
                                  const hlq_tokens* g_k, const hlq_tokens* g_v, void* g_bias,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Dropout with the residual addition:
 *   y_i = residual_i + (r_i >= t ? x_i * 65536 / (65536 - t) : 0)
 * with t = p * 65536 rounded to nearest (ties to even) and r_i 16 random bits of element i; p = 1
 * leaves the residual.  The mask is not stored: r_i is half i % 2 (the lower
 * first) of word i % 8 / 2 of Philox 4x32 with seven rounds (Salmon, Moraes,
 * Dror, Shaw 2011) for the counter (i / 8, site, seed[1] low, seed[1] high)
 * and the key seed[0] (low, high), so that the backward pass draws it again.
 *   x, residual, y [n] dtype, n < 2^35; residual NULL: none.  y may be x or residual.
 *   seed     [2] int64 on the device: a key and a step, which the caller moves on
 *            between training steps (in a captured graph too).
 *   site     tells the places of a model apart that share a seed.
 *   p        0 to 1 (HLQ_ERR_VALUE).
 * An element that is dropped contributes zero whatever it is.  One launch.
 */
hlq_status hlq_dropout_forward(const void* x, const void* residual, int dtype, int64_t n, double p,
                               const int64_t* seed, uint32_t site, void* y, void* stream);
/* The gradient of x: g_x_i = (r_i >= t ? g_y_i * 65536 / (65536 - t) : 0).  g_x may
   be g_y.  The residual's gradient is g_y itself. */
hlq_status hlq_dropout_backward(const void* g_y, int dtype, int64_t n, double p,
                                const int64_t* seed, uint32_t site, void* g_x, void* stream);

/* Static text for a status code (never NULL). */
const char* hlq_status_string(int status);

/* Library ABI version (major*100 + minor). */
int hlq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HLQ_H */
