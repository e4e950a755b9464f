// norm.hip -- block_norm_fwd, block_norm_bwd: the norm after a block, its gate, the scaled addition to the
// residual stream and the norm before the next block in one pass over the rows, and the gradients in another.
//
// With rms(v) = sqrt(mean v^2 + eps), c = weight_offset:
//   u = y / rms(y) (w_post + c),  r = skip h + branch gate u,  n = r / rms(r) (w_pre + c)
// and backwards, a = 1 / rms(r), b = 1 / rms(y), g = grad_n (w_pre + c):
//   dr = grad_r + a g - a^3 r mean(g r),  du = branch gate dr,  q = du (w_post + c),  dy = b q - b^3 y mean(q y)
// mean(q y) needs dr, which needs mean(g r).  As dr is linear in its three terms, with k = branch gate (w_post + c) y
//   sum q y = sum k grad_r + a sum k g - a^3 mean(g r) sum k r
// so all six sums of a row are taken in one reduction, and a row's values stay in registers from the load to
// the store.
//
// A row lies on one workgroup, 8 values a thread, 64 to 1024 threads.  Rows of more than 8192 columns: 16 values a
// thread forwards; backwards they would not fit the registers beside the sums, so one launch takes the rows' sums and
// another makes the gradients, 8192 columns a workgroup.  Several rows a workgroup, one after the other, so that the
// weights are read once and the sums over rows stay in registers; they leave as one partial row a workgroup, summed in
// fp64 by a second kernel.
// A gate row's sum that lies in one workgroup's rows is stored right away; where it spans several, each leaves
// its piece.
//
// HBM bound: every tensor is read or written once (backwards, past 8192 columns, read twice).  8192x4096, residual stream in
// fp32, y and n in bf16: forwards 75 us (5.4 TB/s), backwards 127 and 7 for the sums over workgroups (4.5 TB/s); one row of
// 4096 forwards 3.2; 2048x12288 bf16 forwards 41, backwards 136.
#include "epilogue.hpp"
#include "w4a16q_block.h"

namespace w4q {
namespace {

constexpr int kMaxD = 16384;
constexpr int kFused = 8192;  // columns of a row that 1024 threads hold at 8 values each

// sum over the 64 lanes, in every lane; a fixed order
template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp_add(float v) {
  const int moved = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, kRows, 0xF, false);
  return v + __builtin_bit_cast(float, moved);
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x111, 0xF>(v);  // the lane 1, 2, 4, 8 before it in its row of 16
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // lane 15 of the row before, to rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);  // lane 31, to rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// N sums over a workgroup of `waves` wavefronts.  buf alternates between calls, so one barrier a call is enough: a
// buffer is written again only after the barrier of the call between.  Every wavefront reads all the wavefronts' sums, one a
// lane, and adds them as above (read one after the other they cost a row of 4 wavefronts half a microsecond).
struct SumBuf {
  float v[16];  // wavefronts that are not there count as zeros
};
__device__ __forceinline__ void clear_sums(SumBuf* buf, int n) {
  for (int i = threadIdx.x; i < 16 * n; i += blockDim.x) buf[i >> 4].v[i & 15] = 0.0f;
  __syncthreads();
}
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], int waves, SumBuf* buf) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i].v[threadIdx.x >> 6] = v[i];
  }
  __syncthreads();
  float q[N];
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = buf[i].v[threadIdx.x & 15];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = dpp_add<0x111, 0xF>(q[i]);
    q[i] = dpp_add<0x112, 0xF>(q[i]);
    q[i] = dpp_add<0x114, 0xF>(q[i]);
    q[i] = dpp_add<0x118, 0xF>(q[i]);
    v[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, q[i]), 15));
  }
}

// Eight consecutive columns of a row a thread.  kWhole: rows of whole eights.  kTail: the last thread takes the row's last
// eight columns and skips those that are the thread's before it: they count as zeros and are not stored.  kShort: rows of
// fewer than eight columns, one by one, on thread 0.  Rows need no alignment (one element at a time 1531x1001 took 47 us
// backwards, not 15).
// kAnew: comparisons with skip, d and a type are made anew for each row, as their masks, kept over the rows, take more scalar
// registers than there are (up to 66 spilled, to lanes of a vector register).  Off in the forward kernel of one chunk, which
// has registers for them (1531x1001 7.3 us, made anew 7.9).
enum Kind { kWhole, kTail, kShort };
template <Kind K, bool kAnew = true>
struct Cols {
  int first, skip, d;
  bool some;
  __device__ __forceinline__ Cols(int chunk, int d_) : d(d_) {
    first = 8 * (chunk * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x));
    some = first < d;
    skip = 0;
    if (K == kTail && first > d - 8) {
      skip = first - (d - 8);
      first = d - 8;
    }
  }
  __device__ __forceinline__ void load(const void* p, int64_t row, int dtype, float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    if (p == nullptr || !some) return;
    const int64_t o = row * d + first;
    if (kAnew && !__builtin_constant_p(dtype)) asm volatile("" : "+s"(dtype));
    if constexpr (K == kShort) {
      const int n = skipped();
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < n) v[e] = dtype == 0 ? static_cast<const float*>(p)[o + e] : bf16_val(static_cast<const uint16_t*>(p)[o + e]);
    } else {
      u32x4 a, b;
      load8_any(p, o, dtype, a, b);
      unpack8(a, b, dtype, v);
      if constexpr (K == kTail) {
        const int n = skipped();
#pragma unroll
        for (int e = 0; e < 7; ++e) v[e] = e < n ? 0.0f : v[e];
      }
    }
  }
  // what a group of comparisons is with: skip, or for short rows d
  __device__ __forceinline__ int skipped() const {
    int n = K == kShort ? d : skip;
    if constexpr (kAnew && K == kShort)
      asm volatile("" : "+s"(n));
    else if constexpr (kAnew)
      asm volatile("" : "+v"(n));
    return n;
  }
  // a weight: plus the offset; ones without one
  __device__ __forceinline__ void weight(const float* w, float offset, float (&v)[8]) const {
    load(w, 0, 0, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = w != nullptr ? v[e] + offset : 1.0f;
  }
  __device__ __forceinline__ void store(void* p, int64_t row, int dtype, const float (&v)[8]) const {
    if (!some) return;
    const int64_t o = row * d + first;
    if (kAnew && !__builtin_constant_p(dtype)) asm volatile("" : "+s"(dtype));
    if (K == kShort || (K == kTail && skip != 0)) {
      const int n = skipped();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (K == kShort ? e < n : e >= n) store1(p, o + e, dtype, v[e]);
    } else {
      store8_any(p, o, dtype, v);
    }
  }
};

__device__ __forceinline__ float inv_rms(float sum, int d, float eps) {
  return 1.0f / __builtin_sqrtf(sum / static_cast<float>(d) + eps);
}

struct NormArgs {
  const void *h, *y, *gate;
  const float *w_post, *w_pre;
  int h_dtype, y_dtype, gate_dtype, n_dtype;
  int m, d, run, gate_rows;  // run: rows of a gate row
  w4q_norm_params hp;
  void *r, *n;
};

template <Kind K, int C>
__global__ __launch_bounds__(K == kShort ? 64 : 1024) void norm_fwd_kernel(const NormArgs a) {
  using At = Cols<K, C == 2>;
  __shared__ SumBuf red[2][1];
  const int waves = blockDim.x >> 6;
  clear_sums(red[0], 2);
  float wpost[C][8], wpre[C][8], gate[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const At at(c, a.d);
    at.weight(a.w_post, a.hp.weight_offset, wpost[c]);
    at.weight(a.w_pre, a.hp.weight_offset, wpre[c]);
    at.load(a.gate, 0, a.gate_dtype, gate[c]);
  }
  int par = 0;
#pragma unroll 1
  for (int i = blockIdx.x; i < a.m; i += gridDim.x) {
    const int row = __builtin_amdgcn_readfirstlane(i);  // (as in the backward pass)
    float y[C][8], r[C][8];
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const At at(c, a.d);
      at.load(a.y, row, a.y_dtype, y[c]);
      at.load(a.h, row, a.h_dtype, r[c]);
      if (a.gate_rows > 1) at.load(a.gate, row / a.run, a.gate_dtype, gate[c]);
    }
    if (a.y != nullptr) {
      float b = 1.0f;
      if (a.w_post != nullptr) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(y[c][e], y[c][e], s[0]);
        block_sum(s, waves, red[par]);
        par ^= 1;
        b = inv_rms(s[0], a.d, a.hp.eps);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float u = y[c][e] * b * wpost[c][e];
          if (a.gate != nullptr) u *= gate[c][e];
          r[c][e] = __builtin_fmaf(a.hp.branch_scale, u, a.hp.skip_scale * r[c][e]);
        }
        if (a.r != nullptr) At(c, a.d).store(a.r, row, a.h_dtype, r[c]);
      }
    }
    if (a.n == nullptr) continue;
    s[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(r[c][e], r[c][e], s[0]);
    block_sum(s, waves, red[par]);
    par ^= 1;
    const float b = inv_rms(s[0], a.d, a.hp.eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[c][e] = r[c][e] * b * wpre[c][e];
      At(c, a.d).store(a.n, row, a.n_dtype, r[c]);
    }
  }
}

struct NormBwdArgs {
  const void *gn, *gr, *r, *y, *gate;
  const float *w_post, *w_pre;
  int n_dtype, r_dtype, y_dtype, gate_dtype;
  int m, d, run, gate_rows, rows;  // rows: of a workgroup
  w4q_norm_params hp;
  void *gh, *gy, *ggate;
  float *g_post, *g_pre;
  float* part;  // [pre, post][workgroups][d], then [workgroups][2][d] pieces of gate rows
  f32x4* factors;  // of each row (long rows)
};

// A row's factors from its six sums: dr = gr + f0 (g - f1 (f0 r)),  dy = f2 (q - f3 (f2 y)).  So a^3 is never formed, nor what
// it is multiplied with: they leave fp32's range long before the gradients do.
__device__ __forceinline__ f32x4 row_factors(const NormBwdArgs& a, const float (&s)[6], float inv_d) {
  f32x4 f = {0.0f, 0.0f, 1.0f, 0.0f};
  if (a.gn != nullptr) {
    f[0] = inv_rms(s[0], a.d, a.hp.eps);
    f[1] = f[0] * (s[1] * inv_d);
  }
  if (a.w_post != nullptr) {
    f[2] = inv_rms(s[2], a.d, a.hp.eps);
    f[3] = f[2] * ((s[3] + f[0] * (s[4] - f[1] * (f[0] * s[5]))) * inv_d);
  }
  return f;
}

// kMode 0: everything, for rows of up to 8192 columns.  Longer rows take two launches: kMode 1 takes a row's sums and
// leaves its four factors, kMode 2 makes the gradients of 8192 columns (blockIdx.y) from them.
template <Kind K, int kMode>
__global__ __launch_bounds__(K == kShort ? 64 : 1024) void norm_bwd_kernel(const NormBwdArgs a) {
  __shared__ SumBuf red[2][6];
  const int waves = blockDim.x >> 6;
  if constexpr (kMode != 2) clear_sums(red[0], 12);
  constexpr int kChunks = kMode == 1 ? 2 : 1;
  const int chunk = kMode == 2 ? static_cast<int>(blockIdx.y) : 0;
  const int row0 = blockIdx.x * a.rows;
  const int row1 = a.m - row0 < a.rows ? a.m : row0 + a.rows;
  float s_pre[8], s_post[8], s_gate[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s_pre[e] = s_post[e] = s_gate[e] = 0.0f;

  struct Values {
    float gn[8], gr[8], r[8], y[8], gate[8], wpre[8], wpost[8];
  };
  auto weights = [&](int c, Values& v) {
    const Cols<K> at(c, a.d);
    at.weight(a.w_pre, a.hp.weight_offset, v.wpre);
    at.weight(a.w_post, a.hp.weight_offset, v.wpost);
  };
  auto gates = [&](int c, int g, Values& v) {
    Cols<K>(c, a.d).load(a.gate, g, a.gate_dtype, v.gate);
#pragma unroll
    for (int e = 0; e < 8; ++e) v.gate[e] = a.hp.branch_scale * (a.gate != nullptr ? v.gate[e] : 1.0f);
  };
  auto row_values = [&](int c, int row, Values& v) {
    const Cols<K> at(c, a.d);
    at.load(a.gn, row, a.n_dtype, v.gn);
    at.load(a.gr, row, a.r_dtype, v.gr);
    at.load(a.r, row, a.r_dtype, v.r);
    at.load(a.y, row, a.y_dtype, v.y);
  };
  // a gate row's sum (or this workgroup's piece of it: slot 0 from the first of its rows on, slot 1 behind)
  auto flush_gate = [&](int g) {
    const int64_t g0 = static_cast<int64_t>(g) * a.run;
    const bool all = g0 >= row0 && g0 + a.run <= row1;
    float* part = a.part + (2 * static_cast<int64_t>(gridDim.x) + 2 * blockIdx.x + (g0 > row0 ? 1 : 0)) * a.d;
    const Cols<K> at(chunk, a.d);
    if (all)
      at.store(a.ggate, g, a.gate_dtype, s_gate);
    else
      at.store(part, 0, 0, s_gate);
#pragma unroll
    for (int e = 0; e < 8; ++e) s_gate[e] = 0.0f;
  };

  Values v;
  int g = row0 / a.run, par = 0;
  if constexpr (kMode != 1) {
    weights(chunk, v);
    gates(chunk, g, v);
  }
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const Cols<K> at(chunk, a.d);
#pragma unroll 1
  for (int i = row0; i < row1; ++i) {
    // (taken through a lane, so that no address is kept per element and row by row increased: that spilled registers)
    const int row = __builtin_amdgcn_readfirstlane(i);
    if (row / a.run != g) {
      if (kMode != 1 && a.ggate != nullptr) flush_gate(g);
      g = row / a.run;
      if constexpr (kMode != 1) gates(chunk, g, v);
    }
    if constexpr (kMode != 1) row_values(chunk, row, v);
    f32x4 f;
    if constexpr (kMode != 2) {
      float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c) {
        if constexpr (kMode == 1) {
          weights(c, v);
          gates(c, g, v);
          row_values(c, row, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gg = v.gn[e] * v.wpre[e], k = v.gate[e] * v.wpost[e] * v.y[e];
          s[0] = __builtin_fmaf(v.r[e], v.r[e], s[0]);
          s[1] = __builtin_fmaf(gg, v.r[e], s[1]);
          s[2] = __builtin_fmaf(v.y[e], v.y[e], s[2]);
          s[3] = __builtin_fmaf(k, v.gr[e], s[3]);
          s[4] = __builtin_fmaf(k, gg, s[4]);
          s[5] = __builtin_fmaf(k, v.r[e], s[5]);
        }
      }
      block_sum(s, waves, red[par]);
      par ^= 1;
      f = row_factors(a, s, inv_d);
    }
    if constexpr (kMode == 1) {
      if (threadIdx.x == 0) a.factors[row] = f;
    } else {
      if constexpr (kMode == 2) f = a.factors[row];
      float dh[8], dy[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float rb = v.r[e] * f[0], yb = v.y[e] * f[2];
        const float dr = __builtin_fmaf(f[0], v.gn[e] * v.wpre[e] - f[1] * rb, v.gr[e]);
        const float du = v.gate[e] * dr;
        s_pre[e] = __builtin_fmaf(v.gn[e], rb, s_pre[e]);
        s_post[e] = __builtin_fmaf(du, yb, s_post[e]);
        s_gate[e] = __builtin_fmaf(a.hp.branch_scale * dr, yb * v.wpost[e], s_gate[e]);
        dh[e] = a.hp.skip_scale * dr;
        // (without a norm an infinity in y is not to reach dy: 0 times it is no number)
        dy[e] = f[2] * (du * v.wpost[e] - (a.w_post != nullptr ? f[3] * yb : 0.0f));
      }
      if (a.gh != nullptr) at.store(a.gh, row, a.r_dtype, dh);
      if (a.gy != nullptr) at.store(a.gy, row, a.y_dtype, dy);
    }
  }
  if constexpr (kMode != 1) {
    if (a.ggate != nullptr) flush_gate(g);
    if (a.g_pre != nullptr) at.store(a.part, blockIdx.x, 0, s_pre);
    if (a.g_post != nullptr) at.store(a.part + static_cast<int64_t>(gridDim.x) * a.d, blockIdx.x, 0, s_post);
  }
}

// The same (not for short rows), the next row's loads sent before this row's sums are taken: 1530x1056 bf16 22 -> 14 us,
// 8192x4608 164 -> 98, 1024x8192 28 -> 23.  For bf16 y and grad_n (with fp32 ones two rows do not fit the registers); kR32: r, grad_r and grad_h are
// fp32, not bf16 (whole eights only, again for the registers).
template <bool kWide>
struct Piece {  // eight values as they lie in memory
  u32x4 v[2];
  __device__ __forceinline__ void load(const void* p, int64_t o, bool some) {
    v[0] = v[1] = u32x4{0, 0, 0, 0};
    if (p != nullptr && some) load8_any(p, o, kWide ? 0 : 1, v[0], v[1]);
  }
  __device__ __forceinline__ void clear(int n) {  // the first n of them
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kWide) {
        v[0][i] = i < n ? 0u : v[0][i];
        v[1][i] = i + 4 < n ? 0u : v[1][i];
      } else {
        v[0][i] &= (2 * i < n ? 0u : 0xffffu) | (2 * i + 1 < n ? 0u : 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (kWide) {
      const uint32_t w = v[e >> 2][e & 3];
      return __builtin_bit_cast(float, w);
    }
    return (e & 1) != 0 ? bf16_hi(v[0][e >> 1]) : bf16_lo(v[0][e >> 1]);
  }
};

template <Kind K, bool kR32>
__global__ __launch_bounds__(1024) void norm_bwd_ahead_kernel(const NormBwdArgs a) {
  __shared__ SumBuf red[2][6];
  // this thread's columns of w_pre, w_post and branch gate, four at a time: they would not fit the registers beside two rows
  extern __shared__ f32x4 own[];
  f32x4* const mine = own + threadIdx.x;
  const int t = blockDim.x;
  const int waves = blockDim.x >> 6;
  clear_sums(red[0], 12);
  const int row0 = blockIdx.x * a.rows;
  const int row1 = a.m - row0 < a.rows ? a.m : row0 + a.rows;
  const Cols<K> at(0, a.d);
  constexpr int r_dtype = kR32 ? 0 : 1;
  float s_pre[8], s_gate[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s_pre[e] = s_gate[e] = 0.0f;
  auto keep = [&](int k, const float (&v)[8]) {
    mine[2 * k * t] = f32x4{v[0], v[1], v[2], v[3]};
    mine[(2 * k + 1) * t] = f32x4{v[4], v[5], v[6], v[7]};
  };
  auto kept = [&](int k, int e) { return mine[(2 * k + (e >> 2)) * t][e & 3]; };
  {
    float w[8];
    at.weight(a.w_pre, a.hp.weight_offset, w);
    keep(0, w);
    at.weight(a.w_post, a.hp.weight_offset, w);
    keep(1, w);
  }
  auto gates = [&](int g) {
    float w[8];
    at.load(a.gate, g, a.gate_dtype, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = a.hp.branch_scale * (a.gate != nullptr ? w[e] : 1.0f);
    keep(2, w);
  };
  // A run of rows with one gate row ends: its sum of dr y / rms(y) (in s_gate) gives the gate's gradient and the run's part
  // of w_post's, which is added to this workgroup's partial row (by the thread that wrote it).
  float* const post = a.part + static_cast<int64_t>(gridDim.x) * a.d;
  bool first = true;
  auto flush_gate = [&](int g) {
    const int64_t g0 = static_cast<int64_t>(g) * a.run;
    const bool all = g0 >= row0 && g0 + a.run <= row1;
    float v[8];
    if (a.g_post != nullptr) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = 0.0f;
      if (!first) at.load(post, blockIdx.x, 0, p);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(kept(2, e), s_gate[e], p[e]);
      at.store(post, blockIdx.x, 0, v);
      first = false;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = a.hp.branch_scale * kept(1, e) * s_gate[e];
      s_gate[e] = 0.0f;
    }
    if (a.ggate == nullptr) return;
    float* part = a.part + (2 * static_cast<int64_t>(gridDim.x) + 2 * blockIdx.x + (g0 > row0 ? 1 : 0)) * a.d;
    all ? at.store(a.ggate, g, a.gate_dtype, v) : at.store(part, 0, 0, v);
  };
  struct Row {
    Piece<false> gn, y;
    Piece<kR32> gr, r;
  };
  auto load = [&](int row, Row& x) {
    const int64_t o = static_cast<int64_t>(row) * a.d + at.first;
    x.gn.load(a.gn, o, at.some);
    x.r.load(a.r, o, at.some);
    x.y.load(a.y, o, at.some);
    x.gr.load(a.gr, o, at.some);
  };
  Row ahead;
  load(row0, ahead);
  int g = row0 / a.run, par = 0;
  gates(g);
  const float inv_d = 1.0f / static_cast<float>(a.d);
#pragma unroll 1
  for (int i = row0; i < row1; ++i) {
    const int row = __builtin_amdgcn_readfirstlane(i);
    Row x = ahead;
    if (K == kTail && at.skip != 0) {
      const int n = at.skipped();
      x.gn.clear(n), x.r.clear(n), x.y.clear(n), x.gr.clear(n);
    }
    if (row + 1 < row1) load(row + 1, ahead);
    if (row / a.run != g) {
      flush_gate(g);
      g = row / a.run;
      gates(g);
    }
    float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = x.r.at(e), y = x.y.at(e);
      const float gg = x.gn.at(e) * kept(0, e), k = kept(2, e) * kept(1, e) * y;
      s[0] = __builtin_fmaf(r, r, s[0]);
      s[1] = __builtin_fmaf(gg, r, s[1]);
      s[2] = __builtin_fmaf(y, y, s[2]);
      s[3] = __builtin_fmaf(k, x.gr.at(e), s[3]);
      s[4] = __builtin_fmaf(k, gg, s[4]);
      s[5] = __builtin_fmaf(k, r, s[5]);
    }
    block_sum(s, waves, red[par]);
    par ^= 1;
    const f32x4 f = row_factors(a, s, inv_d);
    float dh[8], dy[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = x.r.at(e), y = x.y.at(e), gn = x.gn.at(e);
      const float rb = r * f[0], yb = y * f[2];
      const float dr = __builtin_fmaf(f[0], gn * kept(0, e) - f[1] * rb, x.gr.at(e));
      s_pre[e] = __builtin_fmaf(gn, rb, s_pre[e]);
      s_gate[e] = __builtin_fmaf(dr, yb, s_gate[e]);
      dh[e] = a.hp.skip_scale * dr;
      dy[e] = f[2] * (kept(2, e) * dr * kept(1, e) - (a.w_post != nullptr ? f[3] * yb : 0.0f));
    }
    if (a.gh != nullptr) at.store(a.gh, row, r_dtype, dh);
    if (a.gy != nullptr) at.store(a.gy, row, 1, dy);
  }
  flush_gate(g);
  if (a.g_pre != nullptr) at.store(a.part, blockIdx.x, 0, s_pre);
}

constexpr int kFinishCols = 32;
// The workgroups' partial rows summed: 32 columns (a cache line) x 32 slices of the workgroups.  blockIdx.y: 0 w_pre, 1
// w_post, then the gate rows (by_row), or the borders between the workgroups, each for the gate row that starts in the
// workgroup before it and reaches over it.  Gate rows that lay in one workgroup are there already.
__global__ __launch_bounds__(1024) void norm_finish_kernel(const NormBwdArgs a, int nwg, int by_row) {
  constexpr int kSlices = 1024 / kFinishCols;
  __shared__ double red[kSlices][kFinishCols];
  const int col = static_cast<int>(blockIdx.x) * kFinishCols + threadIdx.x % kFinishCols, slice = threadIdx.x / kFinishCols;
  int i0 = 0, i1 = nwg - 1;
  const float* part;
  int64_t stride = a.d;
  int odd = 0;  // the first piece lies in slot 1
  int g = static_cast<int>(blockIdx.y) - 2;
  if (g < 0) {
    if ((g == -2 ? a.g_pre : a.g_post) == nullptr) return;
    part = a.part + (g == -2 ? 0 : static_cast<int64_t>(nwg) * a.d);
  } else {
    const int border = (g + 1) * a.rows;
    if (by_row == 0) g = border / a.run;
    const int64_t g0 = static_cast<int64_t>(g) * a.run, g1 = g0 + a.run - 1;
    if (by_row == 0 && (g0 == border || g0 < border - a.rows)) return;
    i0 = static_cast<int>(g0 / a.rows);
    i1 = static_cast<int>(g1 / a.rows);
    if (i0 == i1) return;
    odd = g0 > static_cast<int64_t>(i0) * a.rows ? 1 : 0;
    part = a.part + 2 * static_cast<int64_t>(nwg) * a.d;
    stride = 2 * static_cast<int64_t>(a.d);
  }
  double s = 0.0;
  if (col < a.d) {
#pragma unroll 8
    for (int i = i0 + slice; i <= i1; i += kSlices) s += static_cast<double>(part[i * stride + (i == i0 ? odd * a.d : 0) + col]);
  }
  red[slice][threadIdx.x % kFinishCols] = s;
  __syncthreads();
  if (slice != 0 || col >= a.d) return;
#pragma unroll
  for (int i = 1; i < kSlices; ++i) s += red[i][threadIdx.x];
  const float v = static_cast<float>(s);
  if (g == -2)
    a.g_pre[col] = v;
  else if (g == -1)
    a.g_post[col] = v;
  else
    store1(a.ggate, static_cast<int64_t>(g) * a.d + col, a.gate_dtype, v);
}

// threads of a row: 8 values each, whole wavefronts, up to 1024
int norm_threads(int64_t d) {
  const int64_t t = (d + 511) / 512 * 64;
  return static_cast<int>(t < 1024 ? t : 1024);
}
// rows of a backward workgroup: as many workgroups as the device holds at 16 wavefronts a compute unit, but not fewer rows
// than put one workgroup on each, up to four (each leaves up to four rows of sums.  64x4096 with its sums 15.7 us with four
// rows, 13.0 with one; 300x8192 28.3 with four, 24.0 with two; 1530x1056 19.6 with four, 21.3 with two)
int norm_bwd_rows(int64_t m, int64_t d) {
  const int64_t most = 256 * (1024 / norm_threads(d));
  const int64_t rows = (m + most - 1) / most, one = (m + 255) / 256, least = one < 4 ? one : 4;
  return static_cast<int>(rows < least ? least : rows);
}
int norm_bwd_blocks(int64_t m, int64_t d) {
  const int64_t rows = norm_bwd_rows(m, d);
  return static_cast<int>((m + rows - 1) / rows);
}

}  // namespace
}  // namespace w4q

using namespace w4q;

bool w4q_norm_fits(int64_t m, int64_t d) { return d <= kMaxD && m <= (int64_t(1) << 30); }

int w4q_launch_norm_fwd(const void* h, int h_dtype, const void* y, int y_dtype, int64_t m, int64_t d, const float* w_post,
                        const float* w_pre, const void* gate, int gate_dtype, int64_t gate_rows,
                        const w4q_norm_params& hp, void* r, void* n, int n_dtype, hipStream_t s) {
  const int g = gate != nullptr ? static_cast<int>(gate_rows) : 1;
  const NormArgs a = {h, y, gate, w_post, w_pre, h_dtype, y_dtype, gate_dtype, n_dtype, static_cast<int>(m),
                      static_cast<int>(d), static_cast<int>(m) / g, g, hp, r, n};
  const Kind kind = d % 8 == 0 ? kWhole : d > 8 ? kTail : kShort;
  const int t = norm_threads(d);
  const int64_t most = 256 * (2048 / t);
  const dim3 grid(static_cast<unsigned>(m < most ? m : most)), block(t);
  if (kind == kShort)
    norm_fwd_kernel<kShort, 1><<<grid, block, 0, s>>>(a);
  else if (d > 8 * t)
    kind == kTail ? norm_fwd_kernel<kTail, 2><<<grid, block, 0, s>>>(a) : norm_fwd_kernel<kWhole, 2><<<grid, block, 0, s>>>(a);
  else
    kind == kTail ? norm_fwd_kernel<kTail, 1><<<grid, block, 0, s>>>(a) : norm_fwd_kernel<kWhole, 1><<<grid, block, 0, s>>>(a);
  return w4q_launch_status();
}

size_t w4q_norm_bwd_workspace(int64_t m, int64_t d) {
  const size_t sums = static_cast<size_t>(norm_bwd_blocks(m, d)) * 4 * static_cast<size_t>(d) * sizeof(float);
  return sums + (d > kFused ? static_cast<size_t>(m) * sizeof(f32x4) : 0);
}

int w4q_launch_norm_bwd(const void* gn, int n_dtype, const void* gr, const void* r, int r_dtype, const void* y, int y_dtype,
                        int64_t m, int64_t d, const float* w_post, const float* w_pre, const void* gate, int gate_dtype,
                        int64_t gate_rows, const w4q_norm_params& hp, void* gh, void* gy, float* g_post, float* g_pre,
                        void* ggate, void* ws, hipStream_t s) {
  // what no result needs is not read: an infinity in it is not to reach the others
  if (gn == nullptr) r = nullptr;
  if (w_post == nullptr && ggate == nullptr) y = nullptr;
  const int g = gate != nullptr ? static_cast<int>(gate_rows) : 1;
  const int nwg = norm_bwd_blocks(m, d);
  const NormBwdArgs a = {gn, gr, r, y, gate, w_post, w_pre, n_dtype, r_dtype, y_dtype, gate_dtype, static_cast<int>(m),
                         static_cast<int>(d), static_cast<int>(m) / g, g, norm_bwd_rows(m, d), hp, gh, gy, ggate, g_post,
                         g_pre, static_cast<float*>(ws), reinterpret_cast<f32x4*>(static_cast<float*>(ws) + int64_t(4) * nwg * d)};
  const Kind kind = d % 8 == 0 ? kWhole : d > 8 ? kTail : kShort;
  const int t = norm_threads(d);
  const dim3 grid(nwg), block(t);
  if (kind == kShort) {
    norm_bwd_kernel<kShort, 0><<<grid, block, 0, s>>>(a);
  } else if (d > kFused) {
    kind == kTail ? norm_bwd_kernel<kTail, 1><<<grid, block, 0, s>>>(a) : norm_bwd_kernel<kWhole, 1><<<grid, block, 0, s>>>(a);
    const int first = w4q_launch_status();
    if (first != W4Q_OK) return first;
    const dim3 both(nwg, 2);
    kind == kTail ? norm_bwd_kernel<kTail, 2><<<both, block, 0, s>>>(a) : norm_bwd_kernel<kWhole, 2><<<both, block, 0, s>>>(a);
  } else if ((gn == nullptr || n_dtype == 1) && ((y == nullptr && gy == nullptr) || y_dtype == 1) &&
             (r_dtype == 1 || kind == kWhole)) {
    const unsigned own = static_cast<unsigned>(6 * sizeof(f32x4)) * t;
    if (r_dtype == 0)
      norm_bwd_ahead_kernel<kWhole, true><<<grid, block, own, s>>>(a);
    else
      kind == kTail ? norm_bwd_ahead_kernel<kTail, false><<<grid, block, own, s>>>(a) : norm_bwd_ahead_kernel<kWhole, false><<<grid, block, own, s>>>(a);
  } else {
    kind == kTail ? norm_bwd_kernel<kTail, 0><<<grid, block, 0, s>>>(a) : norm_bwd_kernel<kWhole, 0><<<grid, block, 0, s>>>(a);
  }
  int rc = w4q_launch_status();
  if (rc != W4Q_OK) return rc;
  // gate rows to look at: none where each lies in one workgroup's rows
  const int by_row = g <= nwg - 1;
  const int gates = ggate == nullptr || a.rows % a.run == 0 ? 0 : by_row ? g : nwg - 1;
  if (g_pre == nullptr && g_post == nullptr && gates == 0) return rc;
  norm_finish_kernel<<<dim3(static_cast<unsigned>((d + kFinishCols - 1) / kFinishCols), static_cast<unsigned>(2 + gates)), dim3(1024), 0, s>>>(a, nwg, by_row);
  return w4q_launch_status();
}
