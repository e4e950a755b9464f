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
// Backward: both products run along an axis their operands do not lie along, so one pass over each
// operand writes it transposed (2 B read, 2 B written per value, against 2 d flop of product).  dW
// and dbias are fp32 results, so dz may not be rounded to bf16: with an activation (or fp32 dy)
// dz is held as two fp16 parts, 22 bits, and dW = lo x + hi x.  A bf16 value has 8 bits, so x
// and W are exact in fp16 once a power of two brings their largest value to 2^14 (values below 2^-32
// of the largest lose bits, an absolute error of 2^-40 of it); the exponents come from one maximum
// over each tensor and are taken back in the epilogue.  dx is a bf16 result and takes the hi part
// alone (11 bits, an eighth of the output's own rounding).  Without an activation dz = dy is bf16
// already: one exact bf16 product each, no scaling.
#include "epilogue.hpp"
#include "nt_gemm.hpp"

namespace w4q {
namespace {

constexpr int kAmaxBlocks = 256;  // partial maxima of one tensor
constexpr float kDactMax = 1.13f; // |act'| <= 1.1290 (gelu), 1.0999 (silu), 1 (relu, none)

// ------------------------------------------------------------------------------ epilogues
struct EpiLinear {
  W4Epilogue ep;
  uint16_t* z;  // bf16 [M][N] or null
  void* y;
  int y_dtype;

  __device__ __forceinline__ void operator()(const NtArgs& g, int, int row0, int col0, bool, const f32x16& acc,
                                             int lane) const {
    const int col = col0 + (lane & 31);
    if (col >= g.N) return;
    const float bv = ep.bias != nullptr ? ep.bias[col] : 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = row0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (row >= g.M) continue;
      const int64_t o = static_cast<int64_t>(row) * g.N + col;
      const float zv = acc[r] + bv;
      if (z != nullptr) z[o] = bf16_bits(zv);
      const float v = finish_output(ep, zv, o, y_dtype);
      if (y_dtype == 0)
        static_cast<float*>(y)[o] = v;
      else
        static_cast<uint16_t*>(y)[o] = bf16_bits(v);
    }
  }
};

// a gradient product: the operands' powers of two taken back (each on its own, so that no
// intermediate leaves fp32's range), stored as fp32 or bf16
struct EpiGrad {
  const int* e0;  // exponents of the operands' scales (device), or null
  const int* e1;
  void* out;
  int out_dtype;

  __device__ __forceinline__ void operator()(const NtArgs& g, int, int row0, int col0, bool, const f32x16& acc,
                                             int lane) const {
    const int col = col0 + (lane & 31);
    if (col >= g.N) return;
    const int e = e0 != nullptr ? -(*e0 + *e1) : 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = row0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (row >= g.M) continue;
      const int64_t o = static_cast<int64_t>(row) * g.N + col;
      const float v = __builtin_ldexpf(acc[r], e);
      if (out_dtype == 0)
        static_cast<float*>(out)[o] = v;
      else
        static_cast<uint16_t*>(out)[o] = bf16_bits(v);
    }
  }
};

// --------------------------------------------------------------- the backward's operands
// Largest finite magnitude of dy, x and W (blockIdx.y 0, 1, 2), one partial per workgroup.  HBM bound:
// one read of each.
struct AmaxArgs {
  const void* p[3];
  int64_t n[3];
  int f32[3];
};
__global__ __launch_bounds__(256) void amax_kernel(const AmaxArgs a, float* __restrict__ parts) {
  const int t = blockIdx.y;
  const int64_t n = a.n[t];
  float best = 0.0f;
  auto take = [&](float v) {
    v = __builtin_fabsf(v);
    if (v < __builtin_huge_valf()) best = __builtin_fmaxf(best, v);  // NaN and infinities are left out
  };
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t step = static_cast<int64_t>(kAmaxBlocks) * 256;
  if (a.f32[t]) {
    const float* p = static_cast<const float*>(a.p[t]);
    for (int64_t i = tid; i < n / 4; i += step) {
      const f32x4 v = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) take(v[e]);
    }
    if (tid < n % 4) take(p[n / 4 * 4 + tid]);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.p[t]);
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
// bound * amax * 2^e in (2^13, 2^15].  e = 0 for a tensor of zeros.
__device__ __forceinline__ int scale_exp(const float* __restrict__ parts, float bound) {
  __shared__ float red[256];
  red[threadIdx.x] = parts[threadIdx.x];
  __syncthreads();
#pragma unroll
  for (int o = 128; o >= 1; o >>= 1) {
    if (static_cast<int>(threadIdx.x) < o) red[threadIdx.x] = __builtin_fmaxf(red[threadIdx.x], red[threadIdx.x + o]);
    __syncthreads();
  }
  const float m = red[0];
  __syncthreads();
  if (m == 0.0f) return 0;
  int e;
  (void)__builtin_frexpf(m, &e);  // m = f 2^e, f in [0.5, 1)
  return 14 - e;                  // m 2^(14 - e) in [2^13, 2^14); times 1.13 below 2^15
}
static_assert(kAmaxBlocks == 256, "one partial per thread");

__device__ __forceinline__ uint16_t f16_scaled(float v, int e) { return f32_to_f16_bits(__builtin_ldexpf(v, e)); }

// src [rows][cols] bf16 -> dst [cols][rp], rows' ends up to rp (rows rounded up to 32) zero; as bf16, or
// as fp16 times the power of two of the tensor's maximum (parts != null), whose exponent goes to
// *exp_out.  64x64 tiles through LDS.
__device__ __forceinline__ void transpose_tile(const uint16_t* __restrict__ src, int64_t rows, int64_t cols, int64_t rp,
                                               uint16_t* __restrict__ dst, const float* __restrict__ parts,
                                               int* __restrict__ exp_out, int64_t bx, int64_t by) {
  __shared__ uint16_t tile[64][66];
  int e = 0;
  if (parts != nullptr) {
    e = scale_exp(parts, 1.0f);
    if (bx == 0 && by == 0 && threadIdx.x == 0) *exp_out = e;
  }
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int64_t r0 = by * 64, c0 = bx * 64;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int64_t row = r0 + ty + 4 * i, col = c0 + tx;
    uint16_t v = 0;
    if (row < rows && col < cols) {
      v = src[row * cols + col];
      if (parts != nullptr) v = f16_scaled(bf16_val(v), e);
    }
    tile[ty + 4 * i][tx] = v;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int64_t col = c0 + ty + 4 * i, row = r0 + tx;
    if (col < cols && row < rp) dst[col * rp + row] = tile[tx][ty + 4 * i];
  }
}

struct TransposeArgs {
  const uint16_t* src;
  uint16_t* dst;
  int64_t rows, cols, rp;
  const float* parts;
  int* exp_out;
  int64_t tiles_x;
};
// x and W in one launch: workgroups below `first` take x's tiles, the others W's
__global__ __launch_bounds__(256) void transpose_kernel(const TransposeArgs a, const TransposeArgs b, int64_t first) {
  const int64_t t = blockIdx.x;
  if (t < first)
    transpose_tile(a.src, a.rows, a.cols, a.rp, a.dst, a.parts, a.exp_out, t % a.tiles_x, t / a.tiles_x);
  else
    transpose_tile(b.src, b.rows, b.cols, b.rp, b.dst, b.parts, b.exp_out, (t - first) % b.tiles_x,
                   (t - first) / b.tiles_x);
}

// dz = dy act'(z) for 64 x 64 values: hi part along the features (D, for dx) and hi and lo parts along
// the tokens (T, for dW), the ends up to the next multiple of 32 zero; and the column sums of the tile
// (fp32, 64 terms) for dbias.  kSplit: fp16 parts of dz 2^e; otherwise (no activation, bf16 dy) dz = dy
// itself in bf16.
struct DzArgs {
  const void* dy;
  int dy_f32;
  const uint16_t* z;
  int act;
  int64_t m, n, np, mp;
  uint16_t *d, *th, *tl;  // d, th may be null
  float* bsum;            // [ceil(m / 64)][n] or null
  const float* parts;
  int* exp_out;
};
template <bool kSplit>
__global__ __launch_bounds__(256) void dz_kernel(const DzArgs a) {
  __shared__ uint32_t tile[64][65];
  __shared__ float cs[4][64];
  int e = 0;
  if constexpr (kSplit) {
    e = scale_exp(a.parts, kDactMax);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.exp_out = e;
  }
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  float sum = 0.0f;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int64_t row = r0 + ty + 4 * i, col = c0 + tx;
    uint32_t packed = 0;
    if (row < a.m && col < a.n) {
      const int64_t o = row * a.n + col;
      float v = a.dy_f32 ? static_cast<const float*>(a.dy)[o] : bf16_val(static_cast<const uint16_t*>(a.dy)[o]);
      if (a.act != W4Q_ACT_NONE) v *= act_grad(bf16_val(a.z[o]), a.act);
      sum += v;
      if constexpr (kSplit) {
        const float s = __builtin_ldexpf(v, e);
        const _Float16 hi = static_cast<_Float16>(s);
        const float rest = s - static_cast<float>(hi);
        // an infinite dz stays infinite (its rest is NaN)
        const uint16_t lo = rest == rest ? f32_to_f16_bits(rest) : 0;
        packed = __builtin_bit_cast(uint16_t, hi) | (static_cast<uint32_t>(lo) << 16);
      } else {
        packed = static_cast<const uint16_t*>(a.dy)[o];
      }
    }
    tile[ty + 4 * i][tx] = packed;
    if (a.d != nullptr && row < a.m && col < a.np) a.d[row * a.np + col] = static_cast<uint16_t>(packed);
  }
  if (a.bsum != nullptr) cs[ty][tx] = sum;
  __syncthreads();
  if (a.bsum != nullptr && ty == 0 && c0 + tx < a.n)
    a.bsum[blockIdx.y * a.n + c0 + tx] = (cs[0][tx] + cs[1][tx]) + (cs[2][tx] + cs[3][tx]);
  if (a.th == nullptr) return;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int64_t col = c0 + ty + 4 * i, row = r0 + tx;
    if (col < a.n && row < a.mp) {
      const uint32_t packed = tile[tx][ty + 4 * i];
      a.th[col * a.mp + row] = static_cast<uint16_t>(packed);
      if constexpr (kSplit) a.tl[col * a.mp + row] = static_cast<uint16_t>(packed >> 16);
    }
  }
}

// dbias: the tiles' column sums added in row order, in fp64 (one rounding at the end)
__global__ __launch_bounds__(256) void bias_kernel(const float* __restrict__ bsum, int64_t tiles, int64_t n,
                                                   float* __restrict__ db) {
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (col >= n) return;
  double s = 0.0;
  for (int64_t t = 0; t < tiles; ++t) s += static_cast<double>(bsum[t * n + col]);
  db[col] = static_cast<float>(s);
}

// ------------------------------------------------------------------------------ products
template <int PA, bool F16>
using Big = NtCfg<256, 256, 128, 64, PA, 1, F16, PA == 1 ? 4 : 3>;
template <int PA, bool F16>
using Mid = NtCfg<128, 128, 64, 64, PA, 1, F16, PA == 1 ? 4 : 3>;
template <int PA, bool F16>
using Small = NtCfg<64, 64, 32, 32, PA, 1, F16, 4>;

struct LinPlan {
  int kind;  // 0 Big, 1 Mid, 2 Small
  NtPlan p;
};
// Tile size by how many tiles there are: the largest one that still gives most compute units work.
LinPlan lin_plan(int64_t M, int64_t N, int64_t K) {
  LinPlan r;
  r.p = nt_plan(1, M, N, K, false, 256, 256, kNtCus);
  r.kind = 0;
  if (r.p.per_batch >= 96) return r;
  r.p = nt_plan(1, M, N, K, false, 128, 128, 2 * kNtCus);
  r.kind = 1;
  if (r.p.per_batch >= 128) return r;
  r.p = nt_plan(1, M, N, K, false, 64, 64, 4 * kNtCus);
  r.kind = 2;
  return r;
}

// a plan whose partial tiles fit ws_bytes: the plan itself, or one tile per workgroup
void fit_plan(LinPlan& r, size_t ws_bytes) {
  if (r.p.ws <= ws_bytes) return;
  r.p.chunk = r.p.S;
  r.p.nblk = r.p.total / r.p.S;
  r.p.ws = 0;
}

template <int PA, bool F16, class Epi>
int lin_product(const NtArgs& g, const LinPlan& r, const Epi& e, void* ws, hipStream_t s) {
  if (r.kind == 0) return nt_launch<Big<PA, F16>, Epi>(g, r.p, 0, e, ws, s);
  if (r.kind == 1) return nt_launch<Mid<PA, F16>, Epi>(g, r.p, 0, e, ws, s);
  return nt_launch<Small<PA, F16>, Epi>(g, r.p, 0, e, ws, s);
}

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
inline int64_t up32(int64_t v) { return (v + 31) / 32 * 32; }

struct BwdLayout {
  bool split;        // dz in two fp16 parts
  bool direct;       // dx reads dy as it lies
  int64_t np, mp, mt;
  LinPlan px, pw;
  size_t parts, exps, d, th, tl, xt, wt, bsum, part, total;
};
BwdLayout bwd_layout(int64_t m, int64_t n, int64_t k, int dy_f32, int act) {
  BwdLayout l;
  l.split = act != W4Q_ACT_NONE || dy_f32 != 0;
  l.np = up32(n);
  l.mp = up32(m);
  l.mt = (m + 63) / 64;
  l.direct = !l.split && l.np == n;
  l.px = lin_plan(m, k, l.np);
  l.pw = lin_plan(n, k, l.mp);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up256(bytes);
    return at;
  };
  l.parts = take(l.split ? 3 * kAmaxBlocks * sizeof(float) : 0);
  l.exps = take(l.split ? 3 * sizeof(int) : 0);
  l.d = take(l.direct ? 0 : size_t(2) * m * l.np);
  l.th = take(size_t(2) * n * l.mp);
  l.tl = take(l.split ? size_t(2) * n * l.mp : 0);
  l.xt = take(size_t(2) * k * l.mp);
  l.wt = take(size_t(2) * k * l.np);
  l.bsum = take(sizeof(float) * l.mt * n);
  const size_t most = l.px.p.ws > l.pw.p.ws ? l.px.p.ws : l.pw.p.ws;
  l.part = take(most);
  l.total = o;
  return l;
}

// row lengths whose 256-row tiles stay within 32-bit buffer offsets, and iteration counts of the products
bool fits(int64_t M, int64_t N, int64_t K) {
  if (M > 0x3FFFFFFF || N > 0x3FFFFFFF || K > (1 << 21)) return false;
  return lin_plan(M, N, K).p.total <= 0x3FFFFFFF;
}

}  // namespace
}  // namespace w4q

using namespace w4q;

bool w4q_linear_fits(int64_t m, int64_t d_out, int64_t d_in, bool backward) {
  if (!backward) return fits(m, d_out, d_in);
  // one workgroup per 64x64 tile in the passes over the operands
  if ((m + 63) / 64 > 65535 || (d_out + 63) / 64 > 0x7FFFFFFF || d_in > (1 << 21)) return false;
  if (((d_in + 63) / 64) * ((m + 63) / 64 + (d_out + 63) / 64 + 2) > 0x7FFFFFFF) return false;
  return fits(m, d_in, up32(d_out)) && fits(d_out, d_in, up32(m));
}

size_t w4q_linear_fwd_workspace(int64_t m, int64_t d_out, int64_t d_in) { return lin_plan(m, d_out, d_in).p.ws; }
size_t w4q_linear_bwd_workspace(int64_t m, int64_t d_out, int64_t d_in, int dy_f32, int act) {
  return bwd_layout(m, d_out, d_in, dy_f32, act).total;
}

int w4q_launch_linear_fwd(const uint16_t* x, int64_t m, const uint16_t* w_hat, int64_t d_out, int64_t d_in,
                          const float* bias, int act, const void* res, uint16_t* z, void* y, int y_dtype, void* ws,
                          size_t ws_bytes, hipStream_t s) {
  LinPlan p = lin_plan(m, d_out, d_in);
  fit_plan(p, ws != nullptr ? ws_bytes : 0);
  NtArgs g = {};
  g.a[0] = x;
  g.b[0] = w_hat;
  g.M = static_cast<int>(m);
  g.N = static_cast<int>(d_out);
  g.K = g.lda = g.ldb = static_cast<int>(d_in);
  const EpiLinear e = {{bias, res, act}, z, y, y_dtype};
  return lin_product<1, false>(g, p, e, ws, s);
}

int w4q_launch_linear_bwd(const uint16_t* x, int64_t m, const uint16_t* w_hat, int64_t d_out, int64_t d_in,
                          const void* dy, int dy_f32, int act, const uint16_t* z, uint16_t* dx, float* dw, float* db,
                          void* ws, hipStream_t s) {
  const BwdLayout l = bwd_layout(m, d_out, d_in, dy_f32, act);
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto u16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(base + off); };
  float* parts = l.split ? reinterpret_cast<float*>(base + l.parts) : nullptr;
  int* exps = l.split ? reinterpret_cast<int*>(base + l.exps) : nullptr;  // dy, x, W
  void* part = base + l.part;
  int rc = W4Q_OK;
  if (l.split) {
    AmaxArgs a = {{dy, x, w_hat}, {m * d_out, m * d_in, d_out * d_in}, {dy_f32, 0, 0}};
    hipLaunchKernelGGL(amax_kernel, dim3(kAmaxBlocks, 3), dim3(256), 0, s, a, parts);
    if ((rc = w4q_launch_status()) != W4Q_OK) return rc;
  }
  const bool need_d = dx != nullptr && !l.direct;
  if (need_d || dw != nullptr || db != nullptr) {
    DzArgs a = {dy, dy_f32, z, act, m, d_out, l.np, l.mp, need_d ? u16(l.d) : nullptr, dw != nullptr ? u16(l.th) : nullptr,
                u16(l.tl), db != nullptr ? reinterpret_cast<float*>(base + l.bsum) : nullptr, parts, exps};
    const dim3 grid(static_cast<unsigned>((l.np + 63) / 64), static_cast<unsigned>(l.mt));
    if (l.split)
      hipLaunchKernelGGL(dz_kernel<true>, grid, dim3(256), 0, s, a);
    else
      hipLaunchKernelGGL(dz_kernel<false>, grid, dim3(256), 0, s, a);
    if ((rc = w4q_launch_status()) != W4Q_OK) return rc;
  }
  if (db != nullptr) {
    hipLaunchKernelGGL(bias_kernel, dim3(static_cast<unsigned>((d_out + 255) / 256)), dim3(256), 0, s,
                       reinterpret_cast<const float*>(base + l.bsum), l.mt, d_out, db);
    if ((rc = w4q_launch_status()) != W4Q_OK) return rc;
  }
  if (dx == nullptr && dw == nullptr) return rc;
  const int64_t tk = (d_in + 63) / 64;
  const TransposeArgs tx = {x, u16(l.xt), m, d_in, l.mp, l.split ? parts + kAmaxBlocks : nullptr,
                            l.split ? exps + 1 : nullptr, tk};
  const TransposeArgs tw = {w_hat, u16(l.wt), d_out, d_in, l.np, l.split ? parts + 2 * kAmaxBlocks : nullptr,
                            l.split ? exps + 2 : nullptr, tk};
  const int64_t nx = dw != nullptr ? tk * l.mt : 0;
  const int64_t nw = dx != nullptr ? tk * ((d_out + 63) / 64) : 0;
  hipLaunchKernelGGL(transpose_kernel, dim3(static_cast<unsigned>(nx + nw)), dim3(256), 0, s, tx, tw, nx);
  if ((rc = w4q_launch_status()) != W4Q_OK) return rc;
  if (dx != nullptr) {  // dx [m][d_in] = dz W
    NtArgs g = {};
    g.a[0] = l.direct ? static_cast<const uint16_t*>(dy) : u16(l.d);
    g.b[0] = u16(l.wt);
    g.M = static_cast<int>(m);
    g.N = static_cast<int>(d_in);
    g.K = g.lda = g.ldb = static_cast<int>(l.np);
    const EpiGrad e = {exps, exps + 2, dx, 1};
    rc = l.split ? lin_product<1, true>(g, l.px, e, part, s) : lin_product<1, false>(g, l.px, EpiGrad{nullptr, nullptr, dx, 1}, part, s);
    if (rc != W4Q_OK) return rc;
  }
  if (dw != nullptr) {  // dW [d_out][d_in] = dz^T x
    NtArgs g = {};
    g.a[0] = u16(l.th);
    g.a[1] = u16(l.tl);
    g.b[0] = u16(l.xt);
    g.M = static_cast<int>(d_out);
    g.N = static_cast<int>(d_in);
    g.K = g.lda = g.ldb = static_cast<int>(l.mp);
    const EpiGrad e = {exps, exps + 1, dw, 0};
    rc = l.split ? lin_product<2, true>(g, l.pw, e, part, s) : lin_product<1, false>(g, l.pw, EpiGrad{nullptr, nullptr, dw, 0}, part, s);
  }
  return rc;
}
