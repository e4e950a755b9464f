// api_layer.hip -- the extern "C" entry points of w4a16q_layer.h: argument checks on the host, then
// one launcher per call.  As in api.hip: no allocation, no synchronisation, no mutable state.
#include "common.hpp"
#include "w4a16q_layer.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_layer(int64_t m, int64_t d_out, int64_t d_in) {
  if (m <= 0 || d_out <= 0 || d_in <= 0 || d_in % W4Q_GROUP != 0) return W4Q_ESHAPE;
  if (d_out > (int64_t(1) << 40) / d_in || m > (int64_t(1) << 40) / d_in || m > (int64_t(1) << 40) / d_out)
    return W4Q_ESHAPE;
  return W4Q_OK;
}

inline bool act_ok(int act) { return act >= W4Q_ACT_NONE && act <= W4Q_ACT_SILU; }
inline bool dtype_ok(int t) { return t == 0 || t == 1; }
inline uintptr_t width(int dtype) { return dtype == 0 ? 4 : 2; }
inline bool finite_value(double v) { return __builtin_isfinite(v); }

// scratch of exactly or more than `need` bytes (0: none is needed)
int check_ws(const void* ws, size_t have, size_t need) {
  if (ws == nullptr && (have != 0 || need != 0)) return W4Q_EINVAL;
  if (ws != nullptr && !aligned(ws, 256)) return W4Q_EALIGN;
  return have < need ? W4Q_EINVAL : W4Q_OK;
}

int check_matrix(int64_t batch, int64_t rows, int64_t cols) {
  if (batch <= 0 || rows <= 0 || cols <= 0) return W4Q_ESHAPE;
  if (rows > (int64_t(1) << 40) / cols || batch > (int64_t(1) << 40) / (rows * cols)) return W4Q_ESHAPE;
  return w4q_ns_fits(batch, rows, cols) ? W4Q_OK : W4Q_EUNSUPPORTED;
}

bool iteration_ok(int steps, const float* c, double eps) {
  return steps >= 1 && steps <= 64 && finite_value(eps) && eps >= 0.0 && w4q_ns_coeffs_ok(steps, c[0], c[1], c[2]);
}

}  // namespace

extern "C" {

int lsq_linear_fwd_workspace_size(int64_t m, int64_t d_out, int64_t d_in, size_t* bytes) {
  if (!bytes) return W4Q_EINVAL;
  const int rc = check_layer(m, d_out, d_in);
  if (rc != W4Q_OK) return rc;
  if (!w4q_linear_fits(m, d_out, d_in, false)) return W4Q_EUNSUPPORTED;
  *bytes = w4q_linear_fwd_workspace(m, d_out, d_in);
  return W4Q_OK;
}

int lsq_linear_fwd(const uint16_t* x, int64_t m, const float* w, const float* scale, int64_t d_out,
                   int64_t d_in, const float* bias, int act, const void* residual, uint16_t* w_hat,
                   uint16_t* z, void* y, int y_dtype, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
  if (!x || !w_hat || !y || (w == nullptr) != (scale == nullptr) || !act_ok(act) || !dtype_ok(y_dtype))
    return W4Q_EINVAL;
  int rc = check_layer(m, d_out, d_in);
  if (rc != W4Q_OK) return rc;
  if (!w4q_linear_fits(m, d_out, d_in, false)) return W4Q_EUNSUPPORTED;
  if (w != nullptr && !w4q_lsq_fwd16_fits(d_out, d_in)) return W4Q_EUNSUPPORTED;
  if (!aligned(x, 16) || !aligned(w_hat, 16) || (w && !aligned(w, 16)) || (scale && !aligned(scale, 4)) ||
      (bias && !aligned(bias, 4)) || (z && !aligned(z, 2)) || !aligned(y, width(y_dtype)) ||
      (residual && !aligned(residual, width(y_dtype))))
    return W4Q_EALIGN;
  if ((rc = check_ws(workspace, workspace_bytes, 0)) != W4Q_OK) return rc;
  if (w != nullptr && (rc = w4q_launch_lsq_fwd16(w, scale, d_out, d_in, w_hat, stream)) != W4Q_OK) return rc;
  return w4q_launch_linear_fwd(x, m, w_hat, d_out, d_in, bias, act, residual, z, y, y_dtype, workspace,
                               workspace_bytes, stream);
}

static int bwd_args(int64_t m, int64_t d_out, int64_t d_in, int grad_y_dtype, int act) {
  if (!act_ok(act) || !dtype_ok(grad_y_dtype)) return W4Q_EINVAL;
  const int rc = check_layer(m, d_out, d_in);
  if (rc != W4Q_OK) return rc;
  return w4q_linear_fits(m, d_out, d_in, true) ? W4Q_OK : W4Q_EUNSUPPORTED;
}

int lsq_linear_bwd_workspace_size(int64_t m, int64_t d_out, int64_t d_in, int grad_y_dtype, int act,
                                  size_t* bytes) {
  if (!bytes) return W4Q_EINVAL;
  const int rc = bwd_args(m, d_out, d_in, grad_y_dtype, act);
  if (rc != W4Q_OK) return rc;
  *bytes = w4q_linear_bwd_workspace(m, d_out, d_in, grad_y_dtype == 0, act);
  return W4Q_OK;
}

int lsq_linear_bwd(const uint16_t* x, int64_t m, const uint16_t* w_hat, int64_t d_out, int64_t d_in,
                   const void* grad_y, int grad_y_dtype, int act, const uint16_t* z, uint16_t* grad_x,
                   float* grad_w_hat, float* grad_bias, void* workspace, size_t workspace_bytes,
                   hipStream_t stream) {
  if (!x || !w_hat || !grad_y || (!grad_x && !grad_w_hat && !grad_bias)) return W4Q_EINVAL;
  if (act != W4Q_ACT_NONE && !z) return W4Q_EINVAL;
  int rc = bwd_args(m, d_out, d_in, grad_y_dtype, act);
  if (rc != W4Q_OK) return rc;
  if (!aligned(x, 16) || !aligned(w_hat, 16) || !aligned(grad_y, 16) || (z && !aligned(z, 2)) ||
      (grad_x && !aligned(grad_x, 2)) || (grad_w_hat && !aligned(grad_w_hat, 4)) || (grad_bias && !aligned(grad_bias, 4)))
    return W4Q_EALIGN;
  if ((rc = check_ws(workspace, workspace_bytes, w4q_linear_bwd_workspace(m, d_out, d_in, grad_y_dtype == 0, act))) != W4Q_OK)
    return rc;
  return w4q_launch_linear_bwd(x, m, w_hat, d_out, d_in, grad_y, grad_y_dtype == 0, act, z, grad_x, grad_w_hat,
                               grad_bias, workspace, stream);
}

int w4a16_linear_workspace_size(int64_t m, int64_t d_out, int64_t d_in, int w_mode, size_t* bytes) {
  if (!bytes || !dtype_ok(w_mode)) return W4Q_EINVAL;
  const int rc = check_layer(m, d_out, d_in);
  if (rc != W4Q_OK) return rc;
  const size_t dq = w_mode == 1 ? w4q_linear_dq_workspace(m, d_out, d_in) : 0;
  *bytes = dq != 0 ? dq : w4q_gemm_workspace(m, d_out, d_in, w_mode);
  return W4Q_OK;
}

int w4a16_linear(const uint16_t* x, int64_t m, const uint8_t* packed, const uint16_t* scale_f16,
                 int64_t d_out, int64_t d_in, const float* bias, int act, const void* residual, void* y,
                 int y_dtype, int w_mode, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!x || !packed || !scale_f16 || !y || !act_ok(act) || !dtype_ok(y_dtype) || !dtype_ok(w_mode)) return W4Q_EINVAL;
  int rc = check_layer(m, d_out, d_in);
  if (rc != W4Q_OK) return rc;
  if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(scale_f16, 2) || !aligned(y, width(y_dtype)) ||
      (bias && !aligned(bias, 4)) || (residual && !aligned(residual, width(y_dtype))))
    return W4Q_EALIGN;
  if ((rc = check_ws(workspace, workspace_bytes, 0)) != W4Q_OK) return rc;
  const w4q::W4Epilogue ep = {bias, residual, act};
  if (w_mode == 0 && m <= 16)
    return w4q_launch_gemv(x, m, packed, scale_f16, d_out, d_in, y, y_dtype, stream, &ep);
  const size_t dq = w_mode == 1 ? w4q_linear_dq_workspace(m, d_out, d_in) : 0;
  if (dq != 0 && workspace != nullptr && workspace_bytes >= dq)
    return w4q_launch_linear_dq(x, m, packed, scale_f16, d_out, d_in, ep, y, y_dtype, workspace, workspace_bytes, stream);
  return w4q_launch_gemm(x, m, packed, scale_f16, d_out, d_in, y, y_dtype, w_mode, workspace, workspace_bytes, stream,
                         &ep);
}

int newton_schulz_workspace_size(int64_t batch, int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return W4Q_EINVAL;
  const int rc = check_matrix(batch, rows, cols);
  if (rc != W4Q_OK) return rc;
  *bytes = w4q_ns_workspace(batch, rows, cols);
  return W4Q_OK;
}

int newton_schulz(const void* g, int g_dtype, int64_t batch, int64_t rows, int64_t cols, int steps,
                  const float* coeffs, double eps, void* out, int out_dtype, void* workspace,
                  size_t workspace_bytes, hipStream_t stream) {
  if (!g || !out || !coeffs || !dtype_ok(g_dtype) || !dtype_ok(out_dtype) || !iteration_ok(steps, coeffs, eps))
    return W4Q_EINVAL;
  int rc = check_matrix(batch, rows, cols);
  if (rc != W4Q_OK) return rc;
  if (!aligned(g, width(g_dtype)) || !aligned(out, width(out_dtype))) return W4Q_EALIGN;
  if ((rc = check_ws(workspace, workspace_bytes, w4q_ns_workspace(batch, rows, cols))) != W4Q_OK) return rc;
  return w4q_launch_ns(g, g_dtype, batch, rows, cols, steps, coeffs[0], coeffs[1], coeffs[2], eps, out, out_dtype,
                       nullptr, 0.0f, 0, nullptr, 0.0f, 0.0f, 0.0f, workspace, stream);
}

int muon_step(float* w, const float* grad, float* m, int64_t batch, int64_t rows, int64_t cols,
              const w4q_muon_params* hp, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!w || !grad || !m || !hp) return W4Q_EINVAL;
  if (!finite_value(hp->lr) || hp->lr < 0.0f || !(hp->momentum >= 0.0f && hp->momentum < 1.0f) || !finite_value(hp->weight_decay) ||
      hp->weight_decay < 0.0f || !finite_value(hp->update_scale) || (hp->nesterov != 0 && hp->nesterov != 1) ||
      !iteration_ok(hp->steps, hp->coeffs, hp->eps))
    return W4Q_EINVAL;
  int rc = check_matrix(batch, rows, cols);
  if (rc != W4Q_OK) return rc;
  if (!aligned(w, 4) || !aligned(grad, 4) || !aligned(m, 4)) return W4Q_EALIGN;
  if ((rc = check_ws(workspace, workspace_bytes, w4q_ns_workspace(batch, rows, cols))) != W4Q_OK) return rc;
  return w4q_launch_ns(grad, 0, batch, rows, cols, hp->steps, hp->coeffs[0], hp->coeffs[1], hp->coeffs[2], hp->eps,
                       nullptr, 0, m, hp->momentum, hp->nesterov, w, hp->lr, hp->update_scale, hp->weight_decay,
                       workspace, stream);
}

}  // extern "C"
