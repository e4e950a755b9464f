// linear.hip -- the layer between the LSQ forward and its backward pass: the product of the bf16
// activations with the fake-quantised weights, with bias, activation and residual in its epilogue
// (lsq_linear_fwd), and its gradients (lsq_linear_bwd).
//
// Method: blog "Opt.Gear-QAT: Preserving On-Device Performance with QAT", section 3 (the forward
// emulates the deployment grid; the loss gradient reaches the weights through the straight-through
// estimator), with the weights in the 16-bit activation format as w4a16_gemm_dq takes them:
//   W  = bf16(D * code(w, D)),  z = x W^T + bias,  y = act(z) + residual
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  dbias = sum over rows of dz
//
// Forward: one pass over (w, scale) writes W (HBM bound: 6 B per weight), one product on the bf16
// matrix cores (nt_gemm.hpp; both operands lie along k already) whose epilogue works on the fp32
// sums.
//
// Backward: the products read their operands across their rows where they lie so (dx: W; dW: dz and
// x), so nothing is transposed in memory.  dW and dbias are fp32 results, so dz may not be rounded
// to bf16: with gelu and silu (or fp32 dy) dz is held as two fp16 parts, 22 bits, and dW = lo x +
// hi x.  The parts are of dz 2^e, which brings the largest |dy| into [2^13, 2^14), and lo's last step is
// 2^-24: below 2^-16 of that largest dz loses bits, an absolute error of at most 2^-38 of it.  A bf16 value has
// 8 bits, so x and W are exact in fp16 times the power of two that brings their largest there (below 2^-30 of
// it they lose bits, at most 2^-38 of it); the exponents come from one maximum over each tensor and are
// taken back in the epilogue.
// dx takes both parts too: with the hi part alone (11 bits) one result in 25 was another bf16 value
// than the sum's own rounding; the second product costs a quarter of the call (8192x12288x4096 2199 ->
// 2710 us).
// Without an activation and with relu dz (dy, or 0) is bf16 already: one exact bf16 product each, no scaling,
// and x, W and (without an activation, unless its rows need padding) dy are read as they are.
#include "epilogue.hpp"
#include "nt_gemm.hpp"
#include "ragged.hpp"

namespace w4q {
namespace {

constexpr int kAmaxBlocks = 1024; // partial maxima of one tensor

// ------------------------------------------------------------------------------ epilogues
struct EpiLinear {
  static constexpr bool kMirror = false;
  static constexpr int kLoads = 0;
  struct Pre {
    u32x4 r0, r1;
  };
  W4Epilogue ep;
  uint16_t* z;  // bf16 [M][N] or null
  void* y;
  int y_dtype;
  int vec;      // 8 columns of a row may be moved in 16-byte pieces

  __device__ __forceinline__ int word(int) const { return 0; }
  __device__ __forceinline__ const EpiLinear& with(int) const { return *this; }
  __device__ __forceinline__ bool whole() const { return vec != 0; }
  __device__ __forceinline__ Pre load(const NtArgs& g, int, int row, int col) const {
    Pre p = {};
    if (ep.res != nullptr && vec && row < g.M && col < g.N) load8(ep.res, static_cast<int64_t>(row) * g.N + col, y_dtype, p.r0, p.r1);
    return p;
  }
  __device__ __forceinline__ void activate(float (&v)[8]) const {  // one branch for all eight values
    switch (ep.act) {
      case W4Q_ACT_RELU: act8<W4Q_ACT_RELU>(v); break;
      case W4Q_ACT_GELU: act8<W4Q_ACT_GELU>(v); break;
      case W4Q_ACT_SILU: act8<W4Q_ACT_SILU>(v); break;
      default: break;
    }
  }
  __device__ __forceinline__ void store(const NtArgs& g, int, int row, int col, float (&v)[8], const Pre& p) const {
    if (row >= g.M || col >= g.N) return;
    const int64_t o = static_cast<int64_t>(row) * g.N + col;
    if (ep.bias != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += ep.bias[col + e];
    }
    if (z != nullptr) store8(z, o, 1, v);
    activate(v);
    if (ep.res != nullptr) {
      float r[8];
      unpack8(p.r0, p.r1, y_dtype, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
    store8(y, o, y_dtype, v);
  }
  __device__ __forceinline__ void load_rows(const NtArgs& g, int, int row, int col, float (&r)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = 0.0f;
    if (ep.res == nullptr) return;
    int64_t o[8];
    ragged8(row, g.M, col, g.N, [&](int e, int rr, int c) { o[e] = element_at(0, rr, g.M, c, g.N); });
    if (y_dtype == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = static_cast<const float*>(ep.res)[o[e]];
    } else {
      uint16_t h[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = static_cast<const uint16_t*>(ep.res)[o[e]];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = bf16_val(h[e]);
    }
  }
  __device__ __forceinline__ void store_rows(const NtArgs& g, int, int row, int col, float (&v)[8], const float (&r)[8]) const {
    const int64_t o = static_cast<int64_t>(row) * g.N + col;
    const float bv = ep.bias != nullptr ? ep.bias[col] : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] += bv;
      if (z != nullptr && row + e < g.M) z[o + static_cast<int64_t>(e) * g.N] = bf16_bits(v[e]);
    }
    activate(v);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (row + e < g.M) store1(y, o + static_cast<int64_t>(e) * g.N, y_dtype, v[e] + r[e]);
  }
  template <int kAct>
  static __device__ __forceinline__ void act8(float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_fwd(v[e], kAct);
  }
};

// a gradient product: the operands' powers of two taken back, stored as fp32 or bf16
struct EpiGrad {
  static constexpr bool kMirror = false;
  static constexpr int kLoads = 1;
  struct Pre {
    int e;
  };
  const int* e0;  // exponents of the operands' scales (device), or null
  const int* e1;
  void* out;
  int out_dtype, vec;

  __device__ __forceinline__ int word(int) const { return 0; }
  __device__ __forceinline__ const EpiGrad& with(int) const { return *this; }
  __device__ __forceinline__ bool whole() const { return vec != 0; }
  __device__ __forceinline__ int exponent() const { return e0 != nullptr ? -(*e0 + *e1) : 0; }
  __device__ __forceinline__ Pre load(const NtArgs&, int, int, int) const { return Pre{exponent()}; }
  __device__ __forceinline__ void store(const NtArgs& g, int, int row, int col, float (&v)[8], const Pre& p) const {
    if (row >= g.M || col >= g.N) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_ldexpf(v[e], p.e);
    store8(out, static_cast<int64_t>(row) * g.N + col, out_dtype, v);
  }
  __device__ __forceinline__ void load_rows(const NtArgs&, int, int, int, float (&)[8]) const {}
  __device__ __forceinline__ void store_rows(const NtArgs& g, int, int row, int col, float (&v)[8], const float (&)[8]) const {
    const int x = exponent();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (row + e < g.M) store1(out, static_cast<int64_t>(row + e) * g.N + col, out_dtype, __builtin_ldexpf(v[e], x));
  }
};

// --------------------------------------------------------------- the backward's operands
// Largest finite magnitude of dy, x and W (blockIdx.y 0, 1, 2), one partial per workgroup.  HBM bound:
// one read of each (8192x12288x4096: 368 MB in 75 us).
struct AmaxArgs {
  const void* p[3];
  int64_t n[3];
  int f32[3];
};
__global__ __launch_bounds__(256) void amax_kernel(const AmaxArgs a, float* __restrict__ parts) {
  const int t = blockIdx.y;
  const int64_t n = a.n[t];
  if (n == 0) return;  // not wanted
  float best = 0.0f;
  auto take = [&](float v) {
    v = __builtin_fabsf(v);
    if (v < __builtin_huge_valf()) best = __builtin_fmaxf(best, v);  // NaN and infinities are left out
  };
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t step = static_cast<int64_t>(kAmaxBlocks) * 256;
  if (a.f32[t]) {
    const float* p = static_cast<const float*>(a.p[t]);
#pragma unroll 4
    for (int64_t i = tid; i < n / 4; i += step) {
      const f32x4 v = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) take(v[e]);
    }
    if (tid < n % 4) take(p[n / 4 * 4 + tid]);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.p[t]);
#pragma unroll 4
    for (int64_t i = tid; i < n / 8; i += step) {
      const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        take(bf16_lo(v[e]));
        take(bf16_hi(v[e]));
      }
    }
    if (tid < n % 8) take(bf16_val(p[n / 8 * 8 + tid]));
  }
  __shared__ float red[256];
  red[threadIdx.x] = best;
  __syncthreads();
#pragma unroll
  for (int o = 128; o >= 1; o >>= 1) {
    if (static_cast<int>(threadIdx.x) < o) red[threadIdx.x] = __builtin_fmaxf(red[threadIdx.x], red[threadIdx.x + o]);
    __syncthreads();
  }
  if (threadIdx.x == 0) parts[t * kAmaxBlocks + blockIdx.x] = red[0];
}

// The exponent e of a tensor's scale from its partial maxima (all 256 threads of the workgroup):
// amax * 2^e in [2^13, 2^14), and dz 2^e below 2^15: |act'| <= 1.1290 (gelu), 1.0999 (silu), 1 (relu,
// none).  e = 0 for a tensor of zeros.
__device__ __forceinline__ int scale_exp(const float* __restrict__ parts) {
  __shared__ float red[4];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kAmaxBlocks / 256; ++i) m = __builtin_fmaxf(m, parts[threadIdx.x + 256 * i]);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = __builtin_fmaxf(__builtin_fmaxf(red[0], red[1]), __builtin_fmaxf(red[2], red[3]));
  __syncthreads();
  if (m == 0.0f) return 0;
  int e;
  (void)__builtin_frexpf(m, &e);  // m = f 2^e, f in [0.5, 1)
  return 14 - e;
}

// x and W as fp16 times the power of two of their maxima (exact within 2^-30 of those: 8 bits), whose
// exponents go to exps[1] and exps[2].  HBM bound: 4 B per value.
struct ConvertArgs {
  const uint16_t* src[2];
  uint16_t* dst[2];
  int64_t n8[2];   // eights of values
  int blocks[2];   // workgroups that convert it; 0: not wanted
  int* exps;
};
__device__ __forceinline__ void convert_part(const ConvertArgs& a, int t, int block, const float* __restrict__ parts) {
  const int64_t first = static_cast<int64_t>(block) * 256 + threadIdx.x;
  const u32x4 ahead = first < a.n8[t] ? reinterpret_cast<const u32x4*>(a.src[t])[first] : u32x4{0, 0, 0, 0};
  const int e = scale_exp(parts + (t + 1) * kAmaxBlocks);
  if (block == 0 && threadIdx.x == 0) a.exps[t + 1] = e;
  const int64_t step = static_cast<int64_t>(a.blocks[t]) * 256;
  auto put = [&](int64_t i, const u32x4& v) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = f32_to_f16_bits(__builtin_ldexpf(bf16_lo(v[j]), e)) |
             (static_cast<uint32_t>(f32_to_f16_bits(__builtin_ldexpf(bf16_hi(v[j]), e))) << 16);
    reinterpret_cast<u32x4*>(a.dst[t])[i] = o;
  };
  if (first < a.n8[t]) put(first, ahead);
#pragma unroll 2
  for (int64_t i = first + step; i < a.n8[t]; i += step) put(i, reinterpret_cast<const u32x4*>(a.src[t])[i]);
}

// dz = dy act'(z), rows padded to np values with zeros: as two fp16 parts of dz 2^e (kSplit; the parts of
// 32 columns side by side, as nt_gemm.hpp takes them along and across), or as bf16 (bf16 dy and no
// activation or relu: exact); and column sums over the workgroup's 64 rows for dbias.  A thread has
// 8 columns of a row, a workgroup 256 columns x 64 rows, 8 rows at a time.  HBM bound: dy and z read,
// 4 (2) B written per value (8192x12288x4096
// with the conversions: 1.14 GB in 208 us).
constexpr int kDzRows = 64;
struct DzArgs {
  const void* dy;
  int dy_f32;
  const uint16_t* z;
  int act;
  int64_t m, n, np;
  uint16_t* out;      // [m][np], or with two parts [m][np / 32][hi 32, lo 32]; null (not with parts): not wanted
  float* bsum;        // [ceil(m / 64)][n] or null
  const float* parts;
  int* exp_out;
  int cols, blocks;   // workgroups along a row, and of the whole pass; those behind them convert x and W
};
// the fp16 parts of v 2^e; an infinite v stays infinite (its rest is NaN)
__device__ __forceinline__ void dz_split(float v, int e, uint16_t& h, uint16_t& l) {
  const float s = __builtin_ldexpf(v, e);
  const _Float16 hi = static_cast<_Float16>(s);
  const float rest = s - static_cast<float>(hi);
  h = __builtin_bit_cast(uint16_t, hi);
  l = rest == rest ? f32_to_f16_bits(rest) : 0;
}
template <int kAct>
__device__ __forceinline__ void dact8(float (&v)[8], const float (&z)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= act_grad(z[j], kAct);
}
// the conversion, for a workgroup behind those of the pass over dz (one launch for both)
template <bool kSplit>
__device__ __forceinline__ bool dz_converts(const DzArgs& a, const ConvertArgs& c) {
  if constexpr (kSplit) {
    const int b = static_cast<int>(blockIdx.x) - a.blocks;
    if (b < 0) return false;
    b < c.blocks[0] ? convert_part(c, 0, b, a.parts) : convert_part(c, 1, b - c.blocks[0], a.parts);
    return true;
  }
  return false;
}
template <bool kSplit>
__global__ __launch_bounds__(256) void dz_kernel(const DzArgs a, const ConvertArgs c) {
  __shared__ float cs[8][257];
  if (dz_converts<kSplit>(a, c)) return;
  int e = 0;
  if constexpr (kSplit) {
    e = scale_exp(a.parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.exp_out = e;
  }
  const int bx = static_cast<int>(blockIdx.x) % a.cols, by = static_cast<int>(blockIdx.x) / a.cols;
  const int64_t col = static_cast<int64_t>(bx) * 256 + 8 * (threadIdx.x & 31);
  const int64_t r0 = static_cast<int64_t>(by) * kDzRows + (threadIdx.x >> 5);
  float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (int i = 0; i < kDzRows / 8; ++i) {
    const int64_t row = r0 + 8 * i;
    if (row >= a.m || col >= a.np) continue;
    const int64_t o = row * a.n + col;
    float v[8], zv[8];
    u32x4 d0 = {0, 0, 0, 0}, d1 = {0, 0, 0, 0}, z0 = {0, 0, 0, 0};
    if (col < a.n) {  // n is a multiple of 8
      load8(a.dy, o, a.dy_f32 ? 0 : 1, d0, d1);
      if (a.act != W4Q_ACT_NONE) z0 = *reinterpret_cast<const u32x4*>(a.z + o);
    }
    unpack8(d0, d1, a.dy_f32 ? 0 : 1, v);
    unpack8(z0, z0, 1, zv);
    switch (a.act) {  // (padding columns: 0 times a finite slope)
      case W4Q_ACT_RELU: dact8<W4Q_ACT_RELU>(v, zv); break;
      case W4Q_ACT_GELU: dact8<W4Q_ACT_GELU>(v, zv); break;
      case W4Q_ACT_SILU: dact8<W4Q_ACT_SILU>(v, zv); break;
      default: break;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += v[j];
    if (a.out == nullptr) continue;
    if constexpr (kSplit) {
      uint16_t* q = a.out + row * (2 * a.np) + (col / 32) * 64 + col % 32;
      u32x4 h, l;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint16_t h0, l0, h1, l1;
        dz_split(v[2 * j], e, h0, l0);
        dz_split(v[2 * j + 1], e, h1, l1);
        h[j] = h0 | (static_cast<uint32_t>(h1) << 16);
        l[j] = l0 | (static_cast<uint32_t>(l1) << 16);
      }
      *reinterpret_cast<u32x4*>(q) = h;
      *reinterpret_cast<u32x4*>(q + 32) = l;
    } else {
      *reinterpret_cast<u32x4*>(a.out + row * a.np + col) = pack_bf16(v);  // dy or 0 (bf16): exact
    }
  }
  if (a.bsum == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) cs[threadIdx.x >> 5][8 * (threadIdx.x & 31) + j] = sum[j];
  __syncthreads();
  const int64_t oc = static_cast<int64_t>(bx) * 256 + threadIdx.x;
  if (oc >= a.n) return;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s += cs[j][threadIdx.x];
  a.bsum[by * a.n + oc] = s;
}

// The same where rows are not multiples of 16 bytes: a thread has one column, so that accesses of a row
// are consecutive, and 16 rows at a time; 64 columns x 64 rows to a workgroup.
template <bool kSplit>
__global__ __launch_bounds__(256) void dz_ragged_kernel(const DzArgs a, const ConvertArgs c) {
  __shared__ float cs[4][64];
  if (dz_converts<kSplit>(a, c)) return;
  const int bx = static_cast<int>(blockIdx.x) % a.cols, by = static_cast<int>(blockIdx.x) / a.cols;
  const int64_t col = static_cast<int64_t>(bx) * 64 + (threadIdx.x & 63);
  const int64_t r0 = static_cast<int64_t>(by) * kDzRows + 16 * (threadIdx.x >> 6);
  // everything the thread reads, in flight together and while the exponent is found (places past the
  // matrix read its first value)
  uint32_t dr[16], zr[16];
  auto at = [&](int j) { return r0 + j < a.m && col < a.n ? (r0 + j) * a.n + col : 0; };
  if (a.dy_f32) {
#pragma unroll
    for (int j = 0; j < 16; ++j) dr[j] = static_cast<const uint32_t*>(a.dy)[at(j)];
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) dr[j] = static_cast<const uint16_t*>(a.dy)[at(j)];
  }
  if (a.act != W4Q_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < 16; ++j) zr[j] = a.z[at(j)];
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) zr[j] = 0;
  }
  int e = 0;
  if constexpr (kSplit) {
    e = scale_exp(a.parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.exp_out = e;
  }
  float sum = 0.0f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float v[8], zv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = r0 + 8 * half + j < a.m && col < a.n;
      const uint32_t d = dr[8 * half + j];
      v[j] = in ? __builtin_bit_cast(float, a.dy_f32 ? d : d << 16) : 0.0f;
      zv[j] = __builtin_bit_cast(float, zr[8 * half + j] << 16);
    }
    switch (a.act) {
      case W4Q_ACT_RELU: dact8<W4Q_ACT_RELU>(v, zv); break;
      case W4Q_ACT_GELU: dact8<W4Q_ACT_GELU>(v, zv); break;
      case W4Q_ACT_SILU: dact8<W4Q_ACT_SILU>(v, zv); break;
      default: break;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t row = r0 + 8 * half + j;
      if (row >= a.m || col >= a.np) continue;
      if (col >= a.n) v[j] = 0.0f;  // (0 times another column's slope may be NaN)
      sum += v[j];
      if constexpr (kSplit) {
        uint16_t h, l;
        dz_split(v[j], e, h, l);
        uint16_t* q = a.out + row * (2 * a.np) + (col / 32) * 64 + col % 32;
        q[0] = h;
        q[32] = l;
      } else if (a.out != nullptr) {
        a.out[row * a.np + col] = bf16_bits(v[j]);  // dy or 0 (bf16): exact
      }
    }
  }
  if (a.bsum == nullptr) return;
  cs[threadIdx.x >> 6][threadIdx.x & 63] = sum;
  __syncthreads();
  if (threadIdx.x < 64 && col < a.n)
    a.bsum[by * a.n + col] = (cs[0][threadIdx.x] + cs[1][threadIdx.x]) + (cs[2][threadIdx.x] + cs[3][threadIdx.x]);
}

// dbias: the tiles' column sums added in fp64 (one rounding at the end), in a fixed order: 32 columns x 8
// runs of tiles to a workgroup, each thread its run in row order, then the runs (latency bound: 262144 x 256
// with the pass over dz: 179 us with one thread per column, 39 us so)
__global__ __launch_bounds__(256) void bias_kernel(const float* __restrict__ bsum, int64_t tiles, int64_t n,
                                                   float* __restrict__ db) {
  __shared__ double runs[8][32];
  const int c = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + c;
  const int64_t per = (tiles + 7) / 8, t0 = run * per, t1 = t0 + per < tiles ? t0 + per : tiles;
  double s = 0.0;
  if (col < n) {
#pragma unroll 16
    for (int64_t t = t0; t < t1; ++t) s += static_cast<double>(bsum[t * n + col]);
  }
  runs[run][c] = s;
  __syncthreads();
  if (run != 0 || col >= n) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += runs[i][c];
  db[col] = static_cast<float>(s);
}

// ------------------------------------------------------------------------------ products
template <int PA, bool F16, bool AT, bool BT>
using Big = NtCfg<256, 256, 128, 64, PA, 1, F16, AT, BT>;
template <int PA, bool F16, bool AT, bool BT>
using Mid = NtCfg<128, 128, 64, 64, PA, 1, F16, AT, BT>;
// where no compute unit gets two workgroups, eight wavefronts a tile rather than four, two on each SIMD
// (1531x2050x1056 forward: 38.5 -> 34.3 us; with two workgroups on a compute unit four are better,
// 2048x4096x4096: 95 and 105 us), and a third stage buffer (2048x2048x4096 forward 49 -> 45.5 us)
template <int PA, bool F16, bool AT, bool BT>
using MidAlone = NtCfg<128, 128, 64, 32, PA, 1, F16, AT, BT, false, 3>;
template <int PA, bool F16, bool AT, bool BT>
using Small = NtCfg<64, 64, 32, 32, PA, 1, F16, AT, BT, false, 3>;

// parts: of the first operand; tiny: whether the small-product kernel takes the form (both along k)
NtPlan lin_plan(int64_t M, int64_t N, int64_t K, int parts, bool tiny, bool split = true) {
  return nt_plan(1, M, N, K, false, parts == 1 ? 64 : 32, parts == 1 ? 2.0 : 1.8, split, tiny);
}

template <int PA, bool F16, bool AT, bool BT, class Epi>
int lin_product(const NtArgs& g, const NtPlan& p, const Epi& e, void* ws, hipStream_t s) {
  if (p.kind == 0) return nt_launch<Big<PA, F16, AT, BT>, Epi>(g, p, 0, e, ws, s);
  if (p.kind == 1 && p.nblk <= kNtCus) return nt_launch<MidAlone<PA, F16, AT, BT>, Epi>(g, p, 0, e, ws, s);
  if (p.kind == 1) return nt_launch<Mid<PA, F16, AT, BT>, Epi>(g, p, 0, e, ws, s);
  if constexpr (!AT && !BT) {
    if (p.kind == 3) return nt_launch_tiny<NtTinyCfg<PA, 1, F16, AT, BT>, Epi>(g, p, 0, e, s);
  }
  return nt_launch<Small<PA, F16, AT, BT>, Epi>(g, p, 0, e, ws, s);
}

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
inline bool at16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }  // (null too)
inline int64_t up32(int64_t v) { return (v + 31) / 32 * 32; }

struct BwdLayout {
  bool split;        // dz in two fp16 parts
  bool direct;       // the products read dy as it lies
  int64_t np, mt;
  NtPlan px, pw;
  size_t parts, exps, dz, x16, w16, bsum, part, total;
};
BwdLayout bwd_layout(int64_t m, int64_t n, int64_t k, int dy_f32, int act) {
  BwdLayout l;
  l.split = act == W4Q_ACT_GELU || act == W4Q_ACT_SILU || dy_f32 != 0;
  l.np = up32(n);
  l.mt = (m + kDzRows - 1) / kDzRows;
  l.direct = !l.split && act == W4Q_ACT_NONE && l.np == n;
  l.px = lin_plan(m, k, l.np, l.split ? 2 : 1, false);
  l.pw = lin_plan(n, k, m, l.split ? 2 : 1, false);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up256(bytes);
    return at;
  };
  l.parts = take(l.split ? 3 * kAmaxBlocks * sizeof(float) : 0);
  l.exps = take(l.split ? 3 * sizeof(int) : 0);
  l.dz = take(l.direct ? 0 : size_t(l.split ? 4 : 2) * m * l.np);
  l.x16 = take(l.split ? size_t(2) * m * k : 0);
  l.w16 = take(l.split ? size_t(2) * n * k : 0);
  l.bsum = take(sizeof(float) * l.mt * n);
  const size_t most = l.px.ws > l.pw.ws ? l.px.ws : l.pw.ws;
  l.part = take(most);
  l.total = o;
  return l;
}

// The deployed weights as w4a16_gemm_dq reads them, bf16_RNE(s * q), written out for the product of many
// rows: 8 codes per thread (so that a wavefront's stores are consecutive), s * (q + 8) - 8 s in one exact
// fused multiply-add.  HBM bound: 2.6 B per weight (4096x4096: 10 us, the launch included).
__global__ __launch_bounds__(256) void dequant_kernel(const uint32_t* __restrict__ packed, const uint16_t* __restrict__ s16,
                                                      int64_t words, u32x4* __restrict__ w) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
#pragma unroll 4
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < words; i += step) {
    const float s = f16_bits_to_f32(s16[i >> 2]), ms = -8.0f * s;
    const uint32_t word = packed[i] ^ 0x88888888u;  // codes in offset binary
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(s, static_cast<float>((word >> (4 * e)) & 15u), ms);
    w[i] = pack_bf16(v);
  }
}

// row lengths whose 256-row tiles stay within 32-bit buffer offsets, and iteration and thread counts of
// the products
bool product_fits(int64_t M, int64_t N, int64_t K) { return nt_fits(nt_plan_tile(2, 1, M, N, K, false, 32)); }
bool fits(int64_t M, int64_t N, int64_t K) {
  return M <= 0x3FFFFFFF && N <= 0x3FFFFFFF && K <= (1 << 21) && product_fits(M, N, K);
}

}  // namespace
}  // namespace w4q

using namespace w4q;

bool w4q_linear_fits(int64_t m, int64_t d_out, int64_t d_in, bool backward) {
  if (!backward) return fits(m, d_out, d_in);
  // workgroups of the pass over dz and the conversions (64 rows x 64 columns at least); 32 rows of an
  // operand within 32-bit buffer offsets
  const int64_t mt = (m + kDzRows - 1) / kDzRows;
  if (mt > 65535 || d_in > (1 << 21) || d_out > (1 << 20) || mt * ((d_out + 63) / 64) > (1 << 24) - (1 << 13)) return false;
  return fits(m, d_in, up32(d_out)) && product_fits(d_out, d_in, m);
}

size_t w4q_linear_fwd_workspace(int64_t m, int64_t d_out, int64_t d_in) { return lin_plan(m, d_out, d_in, 1, true).ws; }
size_t w4q_linear_bwd_workspace(int64_t m, int64_t d_out, int64_t d_in, int dy_f32, int act) {
  return bwd_layout(m, d_out, d_in, dy_f32, act).total;
}

int w4q_launch_linear_fwd(const uint16_t* x, int64_t m, const uint16_t* w_hat, int64_t d_out, int64_t d_in,
                          const float* bias, int act, const void* res, uint16_t* z, void* y, int y_dtype, void* ws,
                          size_t ws_bytes, hipStream_t s) {
  NtPlan p = lin_plan(m, d_out, d_in, 1, true);
  if (p.ws > (ws != nullptr ? ws_bytes : 0)) p = lin_plan(m, d_out, d_in, 1, true, false);
  NtArgs g = {};
  g.a = x;
  g.b = w_hat;
  g.M = static_cast<int>(m);
  g.N = static_cast<int>(d_out);
  g.K = g.lda = g.ldb = static_cast<int>(d_in);
  const bool vec = d_out % 8 == 0 && at16(y) && at16(z) && at16(res);
  const EpiLinear e = {{bias, res, act}, z, y, y_dtype, vec ? 1 : 0};
  return lin_product<1, false, false, false>(g, p, e, ws, s);
}

// Rows from which w4a16_linear writes the dequantised weights out and runs the layer product on them,
// rather than dequantising in the product's registers (gemm.hip): any number up to 2^24 weights, 1536 on
// larger ones, where the write costs what it saves before (and the scratch is large).  Measured (in
// registers / written out): 2048x2048 24 rows 43 / 18 us, 2048 rows 107 / 35; 4096x4096 24 rows 51 / 25, 256
// rows 49 / 35, 2048 rows 153 / 81; 12288x4096 17 rows 56 / 49, 64 rows 62 / 58, 256 rows 62 / 66, 768 rows
// 123 / 129, 2048 rows 375 / 245; 4096x12288 17 rows 54 / 51, 256 rows 59 / 70, 2048 rows 270 / 230; 20480x4096
// 17 rows 69 / 74.
constexpr int64_t kDqRows = 1536, kDqWeights = int64_t(1) << 24;
size_t w4q_linear_dq_workspace(int64_t m, int64_t d_out, int64_t d_in) {
  if ((m < kDqRows && d_out * d_in > kDqWeights) || d_in % 256 != 0 || !fits(m, d_out, d_in)) return 0;
  return up256(size_t(2) * d_out * d_in) + lin_plan(m, d_out, d_in, 1, true).ws;
}

int w4q_launch_linear_dq(const uint16_t* x, int64_t m, const uint8_t* packed, const uint16_t* s16, int64_t d_out,
                         int64_t d_in, const W4Epilogue& ep, void* y, int y_dtype, void* ws, size_t ws_bytes,
                         hipStream_t s) {
  const int64_t words = d_out * (d_in / 8), blocks = (words + 1023) / 1024;
  uint16_t* w = static_cast<uint16_t*>(ws);
  const size_t used = up256(size_t(2) * d_out * d_in);
  hipLaunchKernelGGL(dequant_kernel, dim3(static_cast<unsigned>(blocks < 8192 ? blocks : 8192)), dim3(256), 0, s,
                     reinterpret_cast<const uint32_t*>(packed), s16, words, reinterpret_cast<u32x4*>(w));
  const int rc = w4q_launch_status();
  if (rc != W4Q_OK) return rc;
  return w4q_launch_linear_fwd(x, m, w, d_out, d_in, ep.bias, ep.act, ep.res, nullptr, y, y_dtype,
                               static_cast<uint8_t*>(ws) + used, ws_bytes - used, s);
}

int w4q_launch_linear_bwd(const uint16_t* x, int64_t m, const uint16_t* w_hat, int64_t d_out, int64_t d_in,
                          const void* dy, int dy_f32, int act, const uint16_t* z, uint16_t* dx, float* dw, float* db,
                          void* ws, hipStream_t s) {
  const BwdLayout l = bwd_layout(m, d_out, d_in, dy_f32, act);
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto u16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(base + off); };
  float* parts = l.split ? reinterpret_cast<float*>(base + l.parts) : nullptr;
  int* exps = l.split ? reinterpret_cast<int*>(base + l.exps) : nullptr;  // dy, x, W
  float* bsum = db != nullptr ? reinterpret_cast<float*>(base + l.bsum) : nullptr;
  void* part = base + l.part;
  const bool products = dx != nullptr || dw != nullptr;
  int rc = W4Q_OK;
  if (l.split && products) {
    const AmaxArgs a = {{dy, x, w_hat}, {m * d_out, dw != nullptr ? m * d_in : 0, dx != nullptr ? d_out * d_in : 0}, {dy_f32, 0, 0}};
    hipLaunchKernelGGL(amax_kernel, dim3(kAmaxBlocks, 3), dim3(256), 0, s, a, parts);
    if ((rc = w4q_launch_status()) != W4Q_OK) return rc;
  }
  const bool need = products && !l.direct;
  if (need || db != nullptr) {
    const bool whole = d_out % 8 == 0 && at16(z);
    const int64_t cols = whole ? (l.np + 255) / 256 : (l.np + 63) / 64;
    const DzArgs a = {dy, dy_f32, z, act, m, d_out, l.np, need ? u16(l.dz) : nullptr, bsum, parts, exps, static_cast<int>(cols),
                      static_cast<int>(cols * l.mt)};
    ConvertArgs c = {{x, w_hat}, {u16(l.x16), u16(l.w16)}, {m * d_in / 8, d_out * d_in / 8}, {0, 0}, exps};
    auto blocks = [](int64_t n8) { return static_cast<int>(n8 / 512 + 1 < 2048 ? n8 / 512 + 1 : 2048); };
    if (l.split && dw != nullptr) c.blocks[0] = blocks(c.n8[0]);
    if (l.split && dx != nullptr) c.blocks[1] = blocks(c.n8[1]);
    const dim3 grid(static_cast<unsigned>(a.blocks + c.blocks[0] + c.blocks[1]));
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, c); };
    if (l.split && need)
      whole ? run(dz_kernel<true>) : run(dz_ragged_kernel<true>);
    else
      whole ? run(dz_kernel<false>) : run(dz_ragged_kernel<false>);
    if ((rc = w4q_launch_status()) != W4Q_OK) return rc;
  }
  if (db != nullptr) {
    hipLaunchKernelGGL(bias_kernel, dim3(static_cast<unsigned>((d_out + 31) / 32)), dim3(256), 0, s, bsum, l.mt, d_out, db);
    if ((rc = w4q_launch_status()) != W4Q_OK) return rc;
  }
  const uint16_t* dz = l.direct ? static_cast<const uint16_t*>(dy) : u16(l.dz);
  const int ldz = static_cast<int>(l.split ? 2 * l.np : l.np);
  const bool vec = at16(dx) && at16(dw);  // (rows of d_in, a multiple of 32, values)
  if (dx != nullptr) {  // dx [m][d_in] = dz W: dz along n, W across
    NtArgs g = {};
    g.a = dz;
    g.b = l.split ? u16(l.w16) : w_hat;
    g.M = static_cast<int>(m);
    g.N = g.ldb = static_cast<int>(d_in);
    g.lda = ldz;
    g.K = static_cast<int>(l.np);
    g.kb = static_cast<int>(d_out);
    const EpiGrad e = {exps, l.split ? exps + 2 : nullptr, dx, 1, vec ? 1 : 0};
    rc = l.split ? lin_product<2, true, false, true>(g, l.px, e, part, s) : lin_product<1, false, false, true>(g, l.px, e, part, s);
    if (rc != W4Q_OK) return rc;
  }
  if (dw != nullptr) {  // dW [d_out][d_in] = dz^T x: both across
    NtArgs g = {};
    g.a = dz;
    g.b = l.split ? u16(l.x16) : x;
    g.M = static_cast<int>(d_out);
    g.N = g.ldb = static_cast<int>(d_in);
    g.lda = ldz;
    g.K = g.ka = g.kb = static_cast<int>(m);
    const EpiGrad e = {exps, l.split ? exps + 1 : nullptr, dw, 0, vec ? 1 : 0};
    rc = l.split ? lin_product<2, true, true, true>(g, l.pw, e, part, s) : lin_product<1, false, true, true>(g, l.pw, e, part, s);
  }
  return rc;
}
