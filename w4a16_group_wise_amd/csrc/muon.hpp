// muon.hpp -- what muon.hip (products on the matrix cores) and muon_thin.hip (matrices with a short
// side) share: the update's source and the choice between them.
#pragma once

#include "common.hpp"

namespace w4q {

// U: a gradient, or with a momentum buffer m <- mu m + g and U = g + mu m (nesterov) or m
struct Source {
  const void* g;     // gradient, fp32 (dtype 0) or bf16 (1)
  int dtype;
  float* m;          // momentum buffer or null (newton_schulz)
  float mu;
  int nesterov;
};

__device__ __forceinline__ float grad_at(const Source& s, int64_t i) {
  return s.dtype == 0 ? static_cast<const float*>(s.g)[i]
                      : __builtin_bit_cast(float, static_cast<uint32_t>(static_cast<const uint16_t*>(s.g)[i]) << 16);
}

__device__ __forceinline__ float update_at(const Source& s, float g, float m) {
  return s.m == nullptr ? g : s.nesterov ? __builtin_fmaf(s.mu, m, g) : m;
}

// where the result goes: stored (fp32 dtype 0, bf16 1), or applied to fp32 weights (w != null)
struct ThinOut {
  void* out;
  int out_dtype;
  float* w;
  float lr, scale, wd;
};

}  // namespace w4q

bool w4q_thin(int64_t rows, int64_t cols);
bool w4q_thin_steps_ok(int steps, double a);
size_t w4q_thin_workspace(int64_t batch, int64_t rows, int64_t cols);
int w4q_launch_ns_thin(const w4q::Source& src, int64_t batch, int64_t rows, int64_t cols, int steps, float a, float b,
                       float c, double eps, const w4q::ThinOut& o, void* ws, hipStream_t s);
