/*
 * w4a16q_block.h -- C ABI of what lies around the linears of w4a16q.h and w4a16q_layer.h in a decoder's
 * block and its training step: the norms before and after a block with its gate and residual scale, the
 * product in 8-bit floating point for linears that are not held in INT4, and the clipping of the gradients
 * before the optimiser's step.
 *
 * The chain of one training step of a block:
 *   block_norm_fwd -> lsq_linear_fwd or fp8_quant + fp8_gemm -> block_norm_fwd -> (loss)
 *   -> block_norm_bwd -> lsq_linear_bwd or fp8_quant + two fp8_gemm -> grad_clip -> muon_step or lsq_adam_step
 * and of one decoded token:  block_norm_fwd -> w4a16_linear -> block_norm_fwd -> ... -> fp8_gemm (the head).
 *
 * The conventions of w4a16q.h hold (device memory, row-major and contiguous, work enqueued on `stream`,
 * nothing allocated or synchronised, argument errors reported before anything is enqueued, every call can be
 * captured in a HIP graph).  Outputs must not overlap inputs or each other except where named.  Calls that
 * may overlap in time need distinct workspaces.  All results are run-to-run deterministic.
 * dtype arguments: 0 fp32, 1 bf16.  A bf16 output is rounded once, to nearest even, from fp32.
 */
#ifndef W4A16Q_BLOCK_H
#define W4A16Q_BLOCK_H

#include "w4a16q_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Constants of both norms of a block.  eps >= 0; all finite.  weight_offset is added to the norms' weights (1
 * where they are stored as their distance from one). */
typedef struct w4q_norm_params {
  float eps, weight_offset, skip_scale, branch_scale;
} w4q_norm_params;

/*
 * block_norm_fwd -- what lies between two blocks of a decoder: the norm after a block, its gate, the scaled
 * addition to the residual stream, and the norm before the next block, in one pass.  For each row, with
 * rms(v) = sqrt(mean(v^2) + eps):
 *   u = y / rms(y) * (w_post + weight_offset)            (w_post NULL: u = y)
 *   r = skip_scale * h + branch_scale * gate * u         (gate NULL: 1)
 *   n = r / rms(r) * (w_pre + weight_offset)             (of the unrounded r)
 *   h       [m][d] fp32 or bf16 (h_dtype).
 *   y       [m][d] (y_dtype) or NULL: no block's output; then n is h's norm, w_pre and n are needed, w_post,
 *           gate and r must be NULL and the scales are not used (here and in the backward call).
 *   w_post, w_pre   fp32 [d] or NULL; w_pre and n are given together, or neither (r alone).
 *   gate    [gate_rows][d] (gate_dtype) or NULL; m a multiple of gate_rows, row i of m takes gate row
 *           i / (m / gate_rows): one gate for all rows (gate_rows 1), one for each sequence, or one for each row.
 *   r       [m][d] of h's type, out; may be h itself.
 *   n       [m][d] (n_dtype), out.
 * All arithmetic in fp32 (the mean of squares must stay inside fp32's range).  eps 0 gives NaN on rows of zeros.
 * Any d up to 16384, m up to 2^30 (else W4Q_EUNSUPPORTED).  Element-aligned.
 */
int block_norm_fwd(const void* h, int h_dtype, const void* y, int y_dtype, int64_t m, int64_t d, const float* w_post,
                   const float* w_pre, const void* gate, int gate_dtype, int64_t gate_rows, const w4q_norm_params* hp,
                   void* r, void* n, int n_dtype, hipStream_t stream);

/*
 * block_norm_bwd -- its gradients, from the values that a training step keeps (r as it was stored, and y).  With
 * a = 1 / rms(r), g = grad_n * (w_pre + weight_offset), b = 1 / rms(y), q = du * (w_post + weight_offset):
 *   dr = grad_r + a g - a^3 r mean(g r)                   grad_w_pre  = sum_rows grad_n r a
 *   grad_h = skip_scale * dr                              du          = branch_scale * gate * dr
 *   grad_y = b q - b^3 y mean(q y)   (no w_post: du)      grad_w_post = sum_rows du y b
 *   grad_gate = branch_scale * sum over the gate row's rows of u * dr
 *   grad_n  [m][d] (n_dtype) or NULL (then w_pre must be NULL too).
 *   grad_r  [m][d] of r's type or NULL: what reaches r from further on.  Not both NULL.
 *   r       [m][d] (r_dtype); may be NULL without grad_n.  (Without y: r is h.)
 *   y       [m][d] (y_dtype) or NULL as in the forward; may also be NULL where neither w_post nor a gate's
 *           gradient needs it; with y, grad_y or a gate the branch exists.  Without all three the forward had no y:
 *           the scales are not used there, and not here (grad_h = dr).
 *   grad_h  [m][d] of r's type, or NULL; may be grad_r itself.  grad_y [m][d] (y_dtype) or NULL.
 *   grad_w_post, grad_w_pre   fp32 [d] or NULL.  grad_gate [gate_rows][d] of the gate's type or NULL.
 *           At least one output.  Each needs its inputs: grad_w_pre grad_n, grad_w_post w_post, grad_gate gate.
 *   Sums over rows: fp32 within a workgroup's rows, then fp64, in a fixed order.  Sums of a row are fp32's, of products of
 *           branch_scale, gate, weight, y and r (or a gradient) among them: these must stay inside fp32's range.
 *   workspace  block_norm_bwd_workspace_size bytes, 256-B aligned (W4Q_EINVAL if smaller or NULL).
 */
int block_norm_bwd(const void* grad_n, int n_dtype, const void* grad_r, const void* r, int r_dtype, const void* y,
                   int y_dtype, int64_t m, int64_t d, const float* w_post, const float* w_pre, const void* gate,
                   int gate_dtype, int64_t gate_rows, const w4q_norm_params* hp, void* grad_h, void* grad_y,
                   float* grad_w_post, float* grad_w_pre, void* grad_gate, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

int block_norm_bwd_workspace_size(int64_t m, int64_t d, size_t* bytes);

/* 8-bit floating point, a scale for each block of 128 */
#define W4Q_FP8_BLOCK 128
enum w4q_fp8_format { W4Q_FP8_E4M3 = 0 /* largest 448, no infinities */, W4Q_FP8_E5M2 = 1 /* largest 57344 */ };

/*
 * fp8_quant -- a matrix in 8-bit floating point.  A block is 128 consecutive values of a row (square 0) or 128
 * rows by 128 columns (square 1):
 *   scale = fl32(max|x| / largest),  code = the format's value nearest to the exact quotient x / scale, ties to the
 *           even code
 *   codes   [rows][kp], kp = cols rounded up to a multiple of 128, zeros behind the columns; or NULL.
 *   scale   fp32 [rows][kp / 128], or with square [ceil(rows / 128)][kp / 128]; with codes.
 *   codes_t, scale_t   the same of the transpose of x ([cols][rp], rp = rows rounded up; its own blocks run along
 *           the rows of x), or NULL.  At least one of the two forms; both take one pass over x.
 * A block of zeros, or of values whose largest gives a quotient that rounds to zero (at most 2^-150), has scale 0 and
 * codes 0; one with a NaN or an infinity has scale NaN (and codes 0), so that what is made of it is NaN.
 *   x [rows][cols] fp32 or bf16, element-aligned; codes 16-B aligned.  rows, cols <= 2^22 (else W4Q_EUNSUPPORTED).
 */
int fp8_quant(const void* x, int x_dtype, int64_t rows, int64_t cols, int fmt, int square, uint8_t* codes, float* scale,
              uint8_t* codes_t, float* scale_t, hipStream_t stream);

/*
 * fp8_gemm -- the product of two matrices so held, with the layer's epilogue:
 *   z[i][j] = sum_t a_scale[i][t] * b_scale[j'][t] * sum_{k in block t} a[i][k] * b[j][k] + bias[j]
 *   y[i][j] = act(z[i][j]) + residual[i][j]
 * j' = j, or j / 128 with b_square.  a holds activations or gradients (blocks along its rows), b weights (square) or,
 * for a weight gradient, the transposed activations.
 *   a, b    codes [m][k], [n][k] in their formats, 16-B aligned; k a multiple of 128 (as fp8_quant pads it).
 *   a_scale fp32 [m][k / 128], b_scale fp32 [n][k / 128] or [ceil(n / 128)][k / 128].
 *   bias fp32 [n] or NULL; residual [m][n] of y's type or NULL (may be y itself); act as w4q_act.
 *   y_dtype  0 fp32, 1 bf16, or 1 | W4Q_FP8_SHORT: bf16 from the 8-bit matrix cores' own sums, at up to twice the rate.
 * Every product is exact and every sum fp32's.  With W4Q_FP8_SHORT the matrix cores cut each of 8 consecutive k's products
 * off below 2^-13 of the largest of them (7 2^-13 of that at most in all); the sums of eights, and of the blocks, are
 * fp32's there too.  a_scale * b_scale is rounded to fp32 and must stay in its range: below 2^-126 it keeps fewer digits,
 * and from 2^128 on it is infinite: so is what the block adds then, or no number where its sum of codes is zero.
 *   workspace  fp8_gemm_workspace_size bytes, 256-B aligned (W4Q_EINVAL if smaller, or NULL where it is not 0).
 *   Limits: m, n < 2^30, k <= 2^22, at most 2^30 halves of blocks of k over all 64 x 64 output tiles and at most
 *   2^24 - 16 of the tiles (W4Q_EUNSUPPORTED).
 */
#define W4Q_FP8_SHORT 256 /* with y_dtype 1, in fp8_gemm and its workspace's size */
int fp8_gemm(const uint8_t* a, int a_fmt, const float* a_scale, int64_t m, const uint8_t* b, int b_fmt, const float* b_scale,
             int b_square, int64_t n, int64_t k, const float* bias, int act, const void* residual, void* y, int y_dtype,
             void* workspace, size_t workspace_bytes, hipStream_t stream);

int fp8_gemm_workspace_size(int64_t m, int64_t n, int64_t k, int y_dtype, size_t* bytes);

/* One gradient of grad_norm and grad_clip. */
typedef struct w4q_grad {
  const void* g;  /* device, element-aligned */
  void* out;      /* grad_clip: where the clipped gradient goes, element-aligned; may be g where the types are equal */
  int64_t numel;  /* > 0 */
  int g_dtype, out_dtype;
} w4q_grad;

/*
 * grad_norm -- norm = sqrt(sum over the tensors and their elements of g^2), squares and sums in fp64, rounded to
 * fp32 once.  grads: HOST array of n_grads, read before the call returns; out and out_dtype are not used.
 * grad_clip -- with that norm in fp64, out = g * c, c = fl32(1 where norm + eps <= max_norm, else
 * max_norm / (norm + eps)); a norm that is NaN makes every output NaN, an infinite one zeros (and NaN where g is
 * infinite).
 *   max_norm, eps   finite, >= 0; taken in fp64 up to the factor's one rounding.
 *   norm       fp32 [1], device: the norm before clipping.
 *   workspace  grad_norm_workspace_size bytes, 256-B aligned (W4Q_EINVAL if smaller or NULL).
 * 1 <= n_grads <= 65536, at most 2^40 elements in all.  The tensors must not overlap one another.
 */
int grad_norm(const w4q_grad* grads, int64_t n_grads, float* norm, void* workspace, size_t workspace_bytes,
              hipStream_t stream);
int grad_clip(const w4q_grad* grads, int64_t n_grads, double max_norm, double eps, float* norm, void* workspace,
              size_t workspace_bytes, hipStream_t stream);
int grad_norm_workspace_size(int64_t n_grads, size_t* bytes);

#ifdef __cplusplus
}
#endif
#endif /* W4A16Q_BLOCK_H */
