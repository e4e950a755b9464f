// api_block.hip -- the extern "C" entry points of w4a16q_block.h: argument checks on the host, then one
// launcher per call.  As in api.hip: no allocation, no synchronisation, no mutable state.
#include "common.hpp"
#include "w4a16q_block.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool dtype_ok(int t) { return t == 0 || t == 1; }
inline bool flag_ok(int t) { return t == 0 || t == 1; }
inline uintptr_t width(int dtype) { return dtype == 0 ? 4 : 2; }
inline bool gemm_dtype_ok(int t) { return dtype_ok(t) || t == (1 | W4Q_FP8_SHORT); }
inline bool finite_value(double v) { return __builtin_isfinite(v); }

// scratch of exactly or more than `need` bytes (0: none is needed)
int check_ws(const void* ws, size_t have, size_t need) {
  if (ws == nullptr && (have != 0 || need != 0)) return W4Q_EINVAL;
  if (ws != nullptr && !aligned(ws, 256)) return W4Q_EALIGN;
  return have < need ? W4Q_EINVAL : W4Q_OK;
}

int check_rows(int64_t m, int64_t d) {
  if (m <= 0 || d <= 0) return W4Q_ESHAPE;
  return w4q_norm_fits(m, d) ? W4Q_OK : W4Q_EUNSUPPORTED;
}
bool params_ok(const w4q_norm_params* hp) {
  return hp != nullptr && finite_value(hp->eps) && hp->eps >= 0.0f && finite_value(hp->weight_offset) &&
         finite_value(hp->skip_scale) && finite_value(hp->branch_scale);
}
int check_gate(const void* gate, int64_t gate_rows, int64_t m) {
  return gate != nullptr && (gate_rows <= 0 || gate_rows > m || m % gate_rows != 0) ? W4Q_ESHAPE : W4Q_OK;
}

int check_gemm(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || k <= 0 || k % W4Q_FP8_BLOCK != 0) return W4Q_ESHAPE;
  if (m >= (int64_t(1) << 30) || n >= (int64_t(1) << 30) || k > (int64_t(1) << 22)) return W4Q_EUNSUPPORTED;
  return w4q_fp8_fits(m, n, k) ? W4Q_OK : W4Q_EUNSUPPORTED;
}

int check_grads(const w4q_grad* grads, int64_t n, bool clip) {
  if (!grads) return W4Q_EINVAL;
  if (n <= 0) return W4Q_ESHAPE;
  if (n > 65536) return W4Q_EUNSUPPORTED;
  int64_t total = 0;
  for (int64_t i = 0; i < n; ++i) {
    const w4q_grad& g = grads[i];
    if (!g.g || !dtype_ok(g.g_dtype) || (clip && (!g.out || !dtype_ok(g.out_dtype)))) return W4Q_EINVAL;
    if (clip && g.out == g.g && g.out_dtype != g.g_dtype) return W4Q_EINVAL;
    if (g.numel <= 0) return W4Q_ESHAPE;
    if (g.numel > (int64_t(1) << 40)) return W4Q_EUNSUPPORTED;
    total += g.numel;
    if (total > (int64_t(1) << 40)) return W4Q_EUNSUPPORTED;
    if (!aligned(g.g, width(g.g_dtype)) || (clip && !aligned(g.out, width(g.out_dtype)))) return W4Q_EALIGN;
  }
  return W4Q_OK;
}

}  // namespace

extern "C" {

int block_norm_fwd(const void* h, int h_dtype, const void* y, int y_dtype, int64_t m, int64_t d, const float* w_post,
                   const float* w_pre, const void* gate, int gate_dtype, int64_t gate_rows, const w4q_norm_params* hp,
                   void* r, void* n, int n_dtype, hipStream_t stream) {
  if (!h || !params_ok(hp) || !dtype_ok(h_dtype) || (y && !dtype_ok(y_dtype)) || (gate && !dtype_ok(gate_dtype)) ||
      (n && !dtype_ok(n_dtype)) || (w_pre == nullptr) != (n == nullptr) || (!r && !n))
    return W4Q_EINVAL;
  if (y ? !r : (w_post || gate || r)) return W4Q_EINVAL;
  int rc = check_rows(m, d);
  if (rc != W4Q_OK || (rc = check_gate(gate, gate_rows, m)) != W4Q_OK) return rc;
  if (!aligned(h, width(h_dtype)) || (y && !aligned(y, width(y_dtype))) || !aligned(w_post, 4) || !aligned(w_pre, 4) ||
      (gate && !aligned(gate, width(gate_dtype))) || !aligned(r, width(h_dtype)) || (n && !aligned(n, width(n_dtype))))
    return W4Q_EALIGN;
  return w4q_launch_norm_fwd(h, h_dtype, y, y_dtype, m, d, w_post, w_pre, gate, gate_dtype, gate_rows, *hp, r, n, n_dtype,
                             stream);
}

int block_norm_bwd_workspace_size(int64_t m, int64_t d, size_t* bytes) {
  if (!bytes) return W4Q_EINVAL;
  const int rc = check_rows(m, d);
  if (rc != W4Q_OK) return rc;
  *bytes = w4q_norm_bwd_workspace(m, d);
  return W4Q_OK;
}

int block_norm_bwd(const void* grad_n, int n_dtype, const void* grad_r, const void* r, int r_dtype, const void* y,
                   int y_dtype, int64_t m, int64_t d, const float* w_post, const float* w_pre, const void* gate,
                   int gate_dtype, int64_t gate_rows, const w4q_norm_params* hp, void* grad_h, void* grad_y,
                   float* grad_w_post, float* grad_w_pre, void* grad_gate, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
  if ((!grad_n && !grad_r) || (!grad_h && !grad_y && !grad_w_post && !grad_w_pre && !grad_gate)) return W4Q_EINVAL;
  if (!params_ok(hp) || !dtype_ok(r_dtype) || (grad_n && !dtype_ok(n_dtype)) || ((y || grad_y) && !dtype_ok(y_dtype)) ||
      (gate && !dtype_ok(gate_dtype)))
    return W4Q_EINVAL;
  if ((grad_n == nullptr) != (w_pre == nullptr) || (grad_n && !r) || (grad_w_pre && !grad_n) || (grad_w_post && !w_post) ||
      (grad_gate && !gate) || ((w_post || grad_gate) && !y))
    return W4Q_EINVAL;
  int rc = check_rows(m, d);
  if (rc != W4Q_OK || (rc = check_gate(gate, gate_rows, m)) != W4Q_OK) return rc;
  const uintptr_t rw = width(r_dtype), yw = y || grad_y ? width(y_dtype) : 1, gw = gate ? width(gate_dtype) : 1;
  if ((grad_n && !aligned(grad_n, width(n_dtype))) || !aligned(grad_r, rw) || !aligned(r, rw) || !aligned(y, yw) ||
      !aligned(w_post, 4) || !aligned(w_pre, 4) || !aligned(gate, gw) || !aligned(grad_h, rw) || !aligned(grad_y, yw) ||
      !aligned(grad_w_post, 4) || !aligned(grad_w_pre, 4) || !aligned(grad_gate, gw))
    return W4Q_EALIGN;
  if ((rc = check_ws(workspace, workspace_bytes, w4q_norm_bwd_workspace(m, d))) != W4Q_OK) return rc;
  w4q_norm_params p = *hp;
  if (!y && !grad_y && !gate) p.skip_scale = 1.0f;  // no branch: the forward used h as it was
  return w4q_launch_norm_bwd(grad_n, n_dtype, grad_r, r, r_dtype, y, y_dtype, m, d, w_post, w_pre, gate, gate_dtype, gate_rows,
                             p, grad_h, grad_y, grad_w_post, grad_w_pre, grad_gate, workspace, stream);
}

int fp8_quant(const void* x, int x_dtype, int64_t rows, int64_t cols, int fmt, int square, uint8_t* codes, float* scale,
              uint8_t* codes_t, float* scale_t, hipStream_t stream) {
  if (!x || !dtype_ok(x_dtype) || !flag_ok(fmt) || !flag_ok(square) || (codes == nullptr) != (scale == nullptr) ||
      (codes_t == nullptr) != (scale_t == nullptr) || (!codes && !codes_t))
    return W4Q_EINVAL;
  if (rows <= 0 || cols <= 0) return W4Q_ESHAPE;
  if (rows > (int64_t(1) << 22) || cols > (int64_t(1) << 22)) return W4Q_EUNSUPPORTED;
  if (!aligned(x, width(x_dtype)) || !aligned(codes, 16) || !aligned(codes_t, 16) || !aligned(scale, 4) || !aligned(scale_t, 4))
    return W4Q_EALIGN;
  return w4q_launch_fp8_quant(x, x_dtype, rows, cols, fmt, square, codes, scale, codes_t, scale_t, stream);
}

int fp8_gemm_workspace_size(int64_t m, int64_t n, int64_t k, int y_dtype, size_t* bytes) {
  if (!bytes || !gemm_dtype_ok(y_dtype)) return W4Q_EINVAL;
  const int rc = check_gemm(m, n, k);
  if (rc != W4Q_OK) return rc;
  *bytes = w4q_fp8_gemm_workspace(m, n, k, y_dtype);
  return W4Q_OK;
}

int fp8_gemm(const uint8_t* a, int a_fmt, const float* a_scale, int64_t m, const uint8_t* b, int b_fmt, const float* b_scale,
             int b_square, int64_t n, int64_t k, const float* bias, int act, const void* residual, void* y, int y_dtype,
             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!a || !a_scale || !b || !b_scale || !y || !flag_ok(a_fmt) || !flag_ok(b_fmt) || !flag_ok(b_square) ||
      act < W4Q_ACT_NONE || act > W4Q_ACT_SILU || !gemm_dtype_ok(y_dtype))
    return W4Q_EINVAL;
  int rc = check_gemm(m, n, k);
  if (rc != W4Q_OK) return rc;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(bias, 4) ||
      !aligned(y, width(y_dtype)) || !aligned(residual, width(y_dtype)))
    return W4Q_EALIGN;
  if ((rc = check_ws(workspace, workspace_bytes, w4q_fp8_gemm_workspace(m, n, k, y_dtype))) != W4Q_OK) return rc;
  const w4q::W4Epilogue ep = {bias, residual, act};
  return w4q_launch_fp8_gemm(a, a_fmt, a_scale, m, b, b_fmt, b_scale, b_square, n, k, ep, y, y_dtype, workspace, stream);
}

int grad_norm_workspace_size(int64_t n_grads, size_t* bytes) {
  if (!bytes) return W4Q_EINVAL;
  if (n_grads <= 0) return W4Q_ESHAPE;
  if (n_grads > 65536) return W4Q_EUNSUPPORTED;
  *bytes = w4q_clip_workspace(n_grads);
  return W4Q_OK;
}

static int grads_call(const w4q_grad* grads, int64_t n_grads, bool clip, double max_norm, double eps, float* norm, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  if (!norm || !finite_value(max_norm) || max_norm < 0.0 || !finite_value(eps) || eps < 0.0) return W4Q_EINVAL;
  int rc = check_grads(grads, n_grads, clip);
  if (rc != W4Q_OK) return rc;
  if (!aligned(norm, 4)) return W4Q_EALIGN;
  if ((rc = check_ws(workspace, workspace_bytes, w4q_clip_workspace(n_grads))) != W4Q_OK) return rc;
  return w4q_launch_clip(grads, n_grads, clip, max_norm, eps, norm, workspace, stream);
}

int grad_norm(const w4q_grad* grads, int64_t n_grads, float* norm, void* workspace, size_t workspace_bytes,
              hipStream_t stream) {
  return grads_call(grads, n_grads, false, 0.0, 0.0, norm, workspace, workspace_bytes, stream);
}

int grad_clip(const w4q_grad* grads, int64_t n_grads, double max_norm, double eps, float* norm, void* workspace,
              size_t workspace_bytes, hipStream_t stream) {
  return grads_call(grads, n_grads, true, max_norm, eps, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
