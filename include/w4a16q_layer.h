/*
 * w4a16q_layer.h -- C ABI of the quantization-aware layer around the core in w4a16q.h: the layer's
 * product with bias, activation and residual in its epilogue, its gradients, its deployed form on
 * packed codes, and the Muon optimiser step (orthogonalised update) for its weights.
 *
 * The chain of one training step of a linear:
 *   lsq_linear_fwd -> (loss) -> lsq_linear_bwd -> lsq_bwd -> muon_step (or lsq_adam_step)
 * (muon_step steps the weights alone: the step of Delta from lsq_bwd's gradient is the caller's, where
 * lsq_adam_step steps both) and after training: quant_pack -> w4a16_linear.
 *
 * The conventions of w4a16q.h hold (device memory, row-major and contiguous, work enqueued on
 * `stream`, nothing allocated or synchronised, argument errors reported before anything is
 * enqueued, every call can be captured in a HIP graph).  Outputs must not overlap inputs or each
 * other except where named.  Calls that may overlap in time need distinct workspaces.  All results
 * are run-to-run deterministic.
 */
#ifndef W4A16Q_LAYER_H
#define W4A16Q_LAYER_H

#include "w4a16q.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations, for finite z:
 *   NONE z    RELU max(z, 0)    GELU z Phi(z), Phi the normal distribution function
 *   SILU z / (1 + exp(-z))
 * Derivatives: RELU' (z > 0), GELU' Phi(z) + z phi(z), SILU' s (1 + z (1 - s)), s = 1 / (1 + exp(-z)). */
enum w4q_act { W4Q_ACT_NONE = 0, W4Q_ACT_RELU = 1, W4Q_ACT_GELU = 2, W4Q_ACT_SILU = 3 };

/*
 * lsq_linear_fwd -- the layer in the training forward ([blog] section 3: the forward emulates the
 * deployment grid), with the weights in the 16-bit activation format as w4a16_gemm_dq takes them:
 *   w_hat[n][k] = bf16_RNE(fl32(Delta * code(w[n][k], Delta))),  Delta = scale[n][k/32]
 *   z[m][n]     = sum_k x[m][k] * w_hat[n][k] + bias[n]           (fp32 accumulation)
 *   y[m][n]     = act(z[m][n]) + residual[m][n]                   (act on the unrounded z)
 *   x         bf16 [m][d_in], 16-B aligned.
 *   w, scale  fp32 [d_out][d_in] (16-B aligned) and [d_out][d_in/32]: w_hat is written from them and
 *             used; or both NULL: w_hat is read as it is (further micro-batches on the same weights).
 *   w_hat     bf16 [d_out][d_in], 16-B aligned, out (or in).
 *   bias      fp32 [d_out] or NULL.
 *   residual  [m][d_out] of y's type or NULL; may be y itself.
 *   z         bf16 [m][d_out] out or NULL: RNE of z, what lsq_linear_bwd takes.
 *   y         [m][d_out], fp32 (y_dtype 0) or bf16 RNE (y_dtype 1).
 *   workspace NULL with 0 bytes, or 256-B aligned scratch; with less than the query's size no
 *             output tile is split over workgroups (same arithmetic up to the summation order).
 *   Limits: m, d_out < 2^30, d_in <= 2^21, at most 2^30 steps of 32 k over all 64 x 64 output
 *   tiles, and at most 2^24 - 16 of the tiles; with w, d_out * d_in <= 2^35 - 2^11 (W4Q_EUNSUPPORTED).
 */
int lsq_linear_fwd(const uint16_t* x, int64_t m, const float* w, const float* scale, int64_t d_out,
                   int64_t d_in, const float* bias, int act, const void* residual, uint16_t* w_hat,
                   uint16_t* z, void* y, int y_dtype, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

/* Scratch bytes of lsq_linear_fwd's fastest schedule (0: none), in *bytes (host). */
int lsq_linear_fwd_workspace_size(int64_t m, int64_t d_out, int64_t d_in, size_t* bytes);

/*
 * lsq_linear_bwd -- the gradients of lsq_linear_fwd.  With dz = grad_y * act'(z), z the saved bf16
 * pre-activation:
 *   grad_x[m][k]     = sum_n dz[m][n] * w_hat[n][k]     bf16 RNE of the fp32 sum
 *   grad_w_hat[n][k] = sum_m dz[m][n] * x[m][k]         fp32: what lsq_bwd and lsq_adam_step take
 *   grad_bias[n]     = sum_m dz[m][n]                   fp32
 * (the residual's gradient is grad_y itself).
 *   x, w_hat   bf16 as in the forward, 16-B aligned.
 *   grad_y     [m][d_out] fp32 (grad_y_dtype 0) or bf16 (1), 16-B aligned.
 *   z          bf16 [m][d_out]; NULL only with W4Q_ACT_NONE.
 *   grad_x, grad_w_hat, grad_bias   outputs; each may be NULL, not all three.
 *   dz enters both products in 22 bits (with bf16 grad_y and W4Q_ACT_NONE or W4Q_ACT_RELU: as it
 *   is) down to 2^-16 of the largest |grad_y|, and off by at most 2^-38 of that largest below; x and w_hat
 *   then enter as they are down to 2^-30 of their largest, and off by at most 2^-38 of it below.
 *   workspace  lsq_linear_bwd_workspace_size bytes, 256-B aligned (W4Q_EINVAL if smaller or NULL).
 *   Limits: as for the forward, with m <= 4194240, d_out <= 2^20 and at most 2^24 - 2^13 blocks of
 *   64 x 64 in dz (W4Q_EUNSUPPORTED).
 */
int lsq_linear_bwd(const uint16_t* x, int64_t m, const uint16_t* w_hat, int64_t d_out, int64_t d_in,
                   const void* grad_y, int grad_y_dtype, int act, const uint16_t* z, uint16_t* grad_x,
                   float* grad_w_hat, float* grad_bias, void* workspace, size_t workspace_bytes,
                   hipStream_t stream);

int lsq_linear_bwd_workspace_size(int64_t m, int64_t d_out, int64_t d_in, int grad_y_dtype, int act,
                                  size_t* bytes);

/*
 * w4a16_linear -- the deployed layer: w4a16_gemm (w_mode 0: exact weights) or w4a16_gemm_dq (w_mode
 * 1: weights rounded to bf16) with the forward's epilogue applied to the fp32 sums:
 *   y[m][n] = act(sum_k x[m][k] * w_hat[n][k] + bias[n]) + residual[m][n]
 *   bias fp32 [d_out] or NULL; residual [m][d_out] of y's type or NULL (may be y itself); the other
 *   arguments and limits as for those calls, and with one row d_out < 2^31 and d_in <= 2^24
 *   (W4Q_EUNSUPPORTED).
 *   workspace  NULL with 0 bytes, or 256-B aligned scratch.  With the size the query returns the fastest
 *   schedule runs (for many rows with w_mode 1 that holds the weights dequantised once); with
 *   less, one whose scratch fits, with the same arithmetic up to the order of the sums.
 */
int w4a16_linear(const uint16_t* x, int64_t m, const uint8_t* packed, const uint16_t* scale_f16,
                 int64_t d_out, int64_t d_in, const float* bias, int act, const void* residual, void* y,
                 int y_dtype, int w_mode, void* workspace, size_t workspace_bytes, hipStream_t stream);

int w4a16_linear_workspace_size(int64_t m, int64_t d_out, int64_t d_in, int w_mode, size_t* bytes);

/*
 * newton_schulz -- an update orthogonalised by Newton-Schulz products (the published Muon
 * iteration), each matrix of the batch for itself:
 *   X = G / (||G||_F + eps), transposed where rows > cols
 *   steps times:  A = X X^T;  X = a X + (b A + c A A) X
 * which applies s -> a s + b s^3 + c s^5 to every singular value `steps` times.
 *   g, out   [batch][rows][cols], fp32 (dtype 0) or bf16 (1), element-aligned; out may be g where the
 *            types are equal.
 *   coeffs   HOST array {a, b, c}.  Refused (W4Q_EINVAL) if singular values in [0, 1] can grow so
 *            far that A or b A + c A^2 exceeds 7.9 in norm (the operands' fixed-point range).
 *   steps 1 .. 64, eps >= 0 and finite.  (A zero matrix gives zeros; with eps = 0, NaN.)
 *   Operands of the products are held in 22 bits and summed in fp32: the error is that of fp32
 *   products, also where ||G||_F is far below eps (a not 0: small singular values go by a s).
 *   workspace  newton_schulz_workspace_size bytes, 256-B aligned (W4Q_EINVAL if smaller or NULL).
 *   Limits: 1 <= rows, cols <= 131072, batch <= 65535, at most 2^30 steps of 32 k over all
 *   output tiles of a product and at most 2^24 - 16 tiles (W4Q_EUNSUPPORTED).
 */
int newton_schulz(const void* g, int g_dtype, int64_t batch, int64_t rows, int64_t cols, int steps,
                  const float* coeffs, double eps, void* out, int out_dtype, void* workspace,
                  size_t workspace_bytes, hipStream_t stream);

int newton_schulz_workspace_size(int64_t batch, int64_t rows, int64_t cols, size_t* bytes);

/*
 * muon_step -- one Muon step on fp32 weights, in place:
 *   m = momentum * m + grad;  u = nesterov ? grad + momentum * m : m
 *   w = w - lr * (update_scale * newton_schulz(u) + weight_decay * w)
 *   w, grad, m  fp32 [batch][rows][cols], 4-B aligned, not overlapping.
 *   hp          HOST pointer; 0 <= momentum < 1, lr, weight_decay >= 0, update_scale finite,
 *               nesterov 0 or 1, the rest as for newton_schulz (else W4Q_EINVAL).
 *   workspace and limits as for newton_schulz.
 */
typedef struct w4q_muon_params {
  float lr, momentum, weight_decay, update_scale;
  float coeffs[3];
  int nesterov, steps;
  double eps;
} w4q_muon_params;

int muon_step(float* w, const float* grad, float* m, int64_t batch, int64_t rows, int64_t cols,
              const w4q_muon_params* hp, void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* W4A16Q_LAYER_H */
