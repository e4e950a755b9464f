// epilogue.hpp -- bias, activation and residual of the layer products, applied to the fp32 sums in
// registers: y = act(sum + bias[n]) + residual[m][n], one rounding where y is stored.
#pragma once

#include "common.hpp"
#include "w4a16q_layer.h"

namespace w4q {

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }
__device__ __forceinline__ float bf16_val(uint16_t b) { return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16); }

// act(z) in fp32.  gelu is z Phi(z) with Phi by the complementary error function (no cancellation
// for negative z); relu keeps NaN.
__device__ __forceinline__ float act_fwd(float z, int act) {
  switch (act) {
    case W4Q_ACT_RELU: return z <= 0.0f ? 0.0f : z;
    case W4Q_ACT_GELU: return z * 0.5f * erfcf(z * -0.70710678118654752f);
    case W4Q_ACT_SILU: return z / (1.0f + expf(-z));
    default: return z;
  }
}

// act'(z) in fp32
__device__ __forceinline__ float act_grad(float z, int act) {
  switch (act) {
    case W4Q_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case W4Q_ACT_GELU:
      return 0.5f * erfcf(z * -0.70710678118654752f) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    case W4Q_ACT_SILU: {
      const float s = 1.0f / (1.0f + expf(-z));
      return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
  }
}

// the rest of an output after its sum: the residual has y's type (y_dtype 0 fp32, 1 bf16)
__device__ __forceinline__ float finish_output(const W4Epilogue& e, float z, int64_t o, int y_dtype) {
  float v = act_fwd(z, e.act);
  if (e.res != nullptr)
    v += y_dtype == 0 ? static_cast<const float*>(e.res)[o] : bf16_val(static_cast<const uint16_t*>(e.res)[o]);
  return v;
}
__device__ __forceinline__ float apply_epilogue(const W4Epilogue& e, float v, int64_t row, int64_t col, int64_t n,
                                                int y_dtype) {
  if (e.bias != nullptr) v += e.bias[col];
  return finish_output(e, v, row * n + col, y_dtype);
}

}  // namespace w4q
