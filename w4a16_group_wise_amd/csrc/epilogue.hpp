// epilogue.hpp -- bias, activation and residual of the layer products, applied to the fp32 sums in
// registers: y = act(sum + bias[n]) + residual[m][n], one rounding where y is stored.
#pragma once

#include "common.hpp"
#include "w4a16q_layer.h"

namespace w4q {

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }
// a product's value as bf16: with an epilogue it may be any NaN (a bias's), which the rounding by an integer
// addition of common.hpp would carry into 0 where all its bits are set
template <bool kEpi>
__device__ __forceinline__ uint16_t product_bf16(float v) {
  if constexpr (kEpi)
    return bf16_bits(v);
  else
    return f32_to_bf16_bits(v);
}
__device__ __forceinline__ float bf16_val(uint16_t b) { return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16); }

// 1 / (1 + exp(-z)) by the hardware's 2^x and reciprocal (each within one last place): the exponent's
// rounding puts |z| 2^-24 on exp(-z), which reaches the result times 1 - sigmoid, so silu and its
// derivative stay within a few 2^-24 of |z| + 1.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// The normal distribution function Phi(z), and exp(-z^2 / 2) beside it, both to a few 2^-24 of themselves (so
// that gelu keeps its digits far out on the negative side): Phi(-x) = exp(-x^2 / 2) R(x), where R falls smoothly
// from 1/2 like 1 / x; with t = 1 / (1 + 0.345 x), R = t P(t), P the polynomial of degree 8 with the smallest
// largest relative error on 0 <= x <= 15 (1.5 2^-24 with its coefficients in fp32; by least squares
// reweighted until the extremes were level).  The exponent's product is kept in two parts: its rounding alone
// would put x^2 / 2 times 2^-24 on the result.  About 26 instructions (1531x2050x1056 forward 29.6 us, 28.6 with
// 16 instructions for an absolute 2^-22; the library's erfc added 40).  From 2^-126 down (x > 13.2) exp gives 0.
__device__ __forceinline__ float normal_cdf(float z, float& gauss) {
  const float x = __builtin_fminf(__builtin_fabsf(z), 15.0f);  // (past it exp is 0 anyway)
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.345f, x, 1.0f));
  // exp(-x^2 / 2) = 2^(c x^2), c = -log2(e) / 2 = hi + lo
  constexpr float hi = -0.72134752f, lo = -0.72134752044448170 - static_cast<double>(hi);
  const float h = x * x, e = h * hi;
  const float rest = __builtin_fmaf(h, hi, -e) + __builtin_fmaf(h, lo, __builtin_fmaf(x, x, -h) * hi);
  const float g = __builtin_amdgcn_exp2f(e);
  gauss = __builtin_fmaf(g, rest * 0.69314718f, g);
  float q = __builtin_fmaf(-0.028151795f, t, 0.14423357f);
  q = __builtin_fmaf(q, t, -0.26915354f);
  q = __builtin_fmaf(q, t, 0.1850546f);
  q = __builtin_fmaf(q, t, -0.0362379f);
  q = __builtin_fmaf(q, t, 0.11126771f);
  q = __builtin_fmaf(q, t, 0.11736199f);
  q = __builtin_fmaf(q, t, 0.13800524f);
  q = __builtin_fmaf(q, t, 0.1376201f);
  q = q * t * gauss;  // Phi(-|z|)
  return z >= 0.0f ? 1.0f - q : q;
}

// act(z) in fp32; relu keeps NaN
__device__ __forceinline__ float act_fwd(float z, int act) {
  float gauss;
  switch (act) {
    case W4Q_ACT_RELU: return z <= 0.0f ? 0.0f : z;
    case W4Q_ACT_GELU: return z * normal_cdf(z, gauss);
    case W4Q_ACT_SILU: return z * sigmoid(z);
    default: return z;
  }
}

// act'(z) in fp32
__device__ __forceinline__ float act_grad(float z, int act) {
  float gauss;
  switch (act) {
    case W4Q_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case W4Q_ACT_GELU: {
      const float cdf = normal_cdf(z, gauss);
      return __builtin_fmaf(z * gauss, 0.39894228040143268f, cdf);
    }
    case W4Q_ACT_SILU: {
      const float s = sigmoid(z);
      return s * (1.0f + z * (1.0f - s));
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float apply_epilogue(const W4Epilogue& e, float v, int64_t row, int64_t col, int64_t n,
                                                int y_dtype) {
  if (e.bias != nullptr) v += e.bias[col];
  v = act_fwd(v, e.act);
  const int64_t o = row * n + col;
  if (e.res != nullptr)
    v += y_dtype == 0 ? static_cast<const float*>(e.res)[o] : bf16_val(static_cast<const uint16_t*>(e.res)[o]);
  return v;
}

// 8 consecutive values as fp32 from fp32 (dtype 0) or bf16 (1) at element o, and back; 16-byte aligned
__device__ __forceinline__ void unpack8(const u32x4& a, const u32x4& b, int dtype, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dtype == 0) {
      const uint32_t u = a[i], w = b[i];  // (a bit cast of a vector's element itself takes element 0)
      v[i] = __builtin_bit_cast(float, u);
      v[4 + i] = __builtin_bit_cast(float, w);
    } else {
      v[2 * i] = bf16_lo(a[i]);
      v[2 * i + 1] = bf16_hi(a[i]);
    }
  }
}
__device__ __forceinline__ void load8(const void* p, int64_t o, int dtype, u32x4& a, u32x4& b) {
  if (dtype == 0) {
    a = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + o);
    b = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + o + 4);
  } else {
    a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + o);
  }
}
__device__ __forceinline__ u32x4 pack_bf16(const float (&v)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{v[2 * i], v[2 * i + 1]}, bf16x2));
  return u32x4{h[0], h[1], h[2], h[3]};
}
__device__ __forceinline__ void store8(void* p, int64_t o, int dtype, const float (&v)[8]) {
  if (dtype == 0) {
    float* f = static_cast<float*>(p) + o;
    *reinterpret_cast<f32x4*>(f) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(f + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + o) = pack_bf16(v);
  }
}
__device__ __forceinline__ void store1(void* p, int64_t o, int dtype, float v) {
  if (dtype == 0)
    static_cast<float*>(p)[o] = v;
  else
    static_cast<uint16_t*>(p)[o] = bf16_bits(v);
}

}  // namespace w4q
