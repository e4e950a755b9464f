// muon.hip -- the orthogonalised update of Newton-Schulz products and the optimiser step around it
// (newton_schulz, muon_step), next to the fused Adam step of pack_lsq.hip.
//
// Mathematics (the Muon optimiser's published update): with n = min(rows, cols), k = max,
//   X0 = U / (||U||_F + eps)   (transposed where rows > cols, so that X is n x k)
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X        `steps` times
// which applies the odd polynomial a s + b s^3 + c s^5 to every singular value; with the published
// (a, b, c) five steps take singular values from about 0.01 upwards to between 0.7 and 1.2.
//
// Precision: outputs are fp32.  Each step multiplies small singular directions by up to a = 3.44, and
// with bf16 operands five steps end 1e-3 .. 2e-2 off (2-norm).  So X, A and B are kept as two fp16
// parts, hi + lo = 2^13 v in 22 bits, and every product is three matrix-core products summed in fp32
// (nt_gemm.hpp): the error is that of fp32 products, at a third of the 16-bit matrix-core rate.
// 2^13: |X| <= 1.21, |A| <= 1.45, |B| <= 2.81 for the published coefficients (spectral bounds, so they
// bound the entries), and 2^13 * 7.99 is fp16's largest value; other coefficients are checked against
// these limits on the host.
// Where ||U|| is below eps X0 is small, and a fixed point would leave it few bits.  So X is held times 2^e as
// well: e_0 = E, one exponent for each matrix with 2^E ||X0||_F in [1/2, 1), and after s steps max(0, E - h_s),
// h_s = ceil(s log2 g): a step multiplies singular values up to 1 by at most g = max |a + b t + c t^2| over
// 0 <= t <= 1, so 2^e X stays within norm 1 until e is 0.  The epilogues take the power of two back (A) or
// on (X); ordinary inputs have E = 0 and the bits they had without it.
//
// Work per step: A and A^2 are symmetric (tiles on and below the diagonal only, the others stored
// mirrored), B X is whole: n^2 k + n^3 + 2 n^2 k flop, times three products.  Matrix-core bound from
// n of about 1024 up; below that the chain of dependent launches is what costs.
//
// Layouts: X stays as U lies, [rows][cols] with rows padded to a multiple of 32 values, in two buffers
// that alternate (other tiles still read the old one).  Where rows > cols the iteration is written
// for Y = X^T: A = Y^T Y, Y <- a Y + Y B (B is symmetric).  The products read operands along or across
// their rows, so nothing is transposed in memory.
#include "epilogue.hpp"
#include "muon.hpp"
#include "nt_gemm.hpp"
#include "ragged.hpp"

namespace w4q {
namespace {

constexpr float kSplitInv = 1.0f / 8192.0f;  // 2^-13

// hi and lo of a scaled value (both RNE)
__device__ __forceinline__ void split16(float v, uint16_t& h, uint16_t& l) {
  const _Float16 hi = static_cast<_Float16>(v);
  h = __builtin_bit_cast(uint16_t, hi);
  l = f32_to_f16_bits(v - static_cast<float>(hi));
}

// ------------------------------------------------------------------------- epilogues
__device__ __forceinline__ void split8(const float (&v)[8], u32x4& h, u32x4& l) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t h0, l0, h1, l1;
    split16(v[2 * i], h0, l0);
    split16(v[2 * i + 1], h1, l1);
    h[i] = h0 | (static_cast<uint32_t>(h1) << 16);
    l[i] = l0 | (static_cast<uint32_t>(l1) << 16);
  }
}
__device__ __forceinline__ void join8(const u32x4& h, const u32x4& l, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = f16_bits_to_f32(static_cast<uint16_t>(h[i])) + f16_bits_to_f32(static_cast<uint16_t>(l[i]));
    v[2 * i + 1] = f16_bits_to_f32(static_cast<uint16_t>(h[i] >> 16)) + f16_bits_to_f32(static_cast<uint16_t>(l[i] >> 16));
  }
}

// a split matrix per batch (nt_gemm.hpp): rows of ld columns, ld a multiple of 32; the parts of 32
// columns side by side
struct Split {
  uint16_t* p;
  int ld;
  int64_t stride;  // 16-bit values between batches (2 * rows * ld)

  // of the hi part of (row, col); the lo part is 32 further
  __device__ __forceinline__ int64_t at(int batch, int64_t row, int col) const { return split_at(batch, stride, row, ld, col); }
};
struct Pair8 {
  u32x4 h, l;
};
__device__ __forceinline__ void store_pair(const Split& m, int batch, int64_t row, int col, const float (&v)[8]) {
  u32x4 h, l;
  split8(v, h, l);
  uint16_t* q = m.p + m.at(batch, row, col);
  *reinterpret_cast<u32x4*>(q) = h;
  *reinterpret_cast<u32x4*>(q + 32) = l;
}
__device__ __forceinline__ Pair8 load_pair(const Split& m, int batch, int row, int col) {
  const uint16_t* q = m.p + m.at(batch, row, col);
  return Pair8{*reinterpret_cast<const u32x4*>(q), *reinterpret_cast<const u32x4*>(q + 32)};
}

// The power of two by which an epilogue's result is multiplied, from the matrix's exponent E: X comes with
// e = max(0, E - from), `times` times (once, or twice in X X^T), and leaves with max(0, E - to)
constexpr int kNoExponent = 1 << 30;  // as `to`: leaves without
struct Exponent {
  const int* e;  // E of each matrix, or null: no power of two
  int from, times, to;
  // a factor of the result times it, once per tile and in a scalar register (0 where a large negative power
  // takes it below fp32's range: so is what it would multiply)
  __device__ __forceinline__ float scaled(float v, int x) const {
    const float f = __builtin_ldexpf(v, (x > to ? x - to : 0) - (x > from ? times * (x - from) : 0));
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, f)));
  }
};

// (alpha * C + beta * acc) 2^exponent, split, as the output (its rows' padding, where both terms are zero, included);
// kSym: a symmetric result of which only the tiles on and below the diagonal are computed: the
// others get the transposed values
template <bool kSym>
struct EpiSplit {
  static constexpr bool kMirror = kSym;
  static constexpr int kLoads = 2;
  using Pre = Pair8;
  Split c;  // C term; c.p null: none
  float alpha, beta;
  Split o;
  Exponent ex;

  __device__ __forceinline__ int word(int batch) const { return ex.e != nullptr ? ex.e[batch] : 0; }
  __device__ __forceinline__ EpiSplit with(int word) const {
    EpiSplit e = *this;
    e.alpha = ex.scaled(alpha, word);
    e.beta = ex.scaled(beta, word);
    return e;
  }
  __device__ __forceinline__ bool whole() const { return true; }
  __device__ __forceinline__ void load_rows(const NtArgs&, int, int, int, float (&)[8]) const {}
  __device__ __forceinline__ void store_rows(const NtArgs&, int, int, int, const float (&)[8], const float (&)[8]) const {}
  __device__ __forceinline__ Pre load(const NtArgs& g, int batch, int row, int col) const {
    Pre p = {};
    if (c.p != nullptr && row < g.M && col < c.ld) p = load_pair(c, batch, row, col);
    return p;
  }
  __device__ __forceinline__ void store(const NtArgs& g, int batch, int row, int col, float (&v)[8], const Pre& p) const {
    float t[8];
    join8(p.h, p.l, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(alpha, t[e], beta * v[e]);
    if (row < g.M && col < o.ld) store_pair(o, batch, row, col, v);
  }
  __device__ __forceinline__ void store_t(const NtArgs& g, int batch, int col, int row, const float (&v)[8]) const {
    if (col < g.N && row < o.ld) store_pair(o, batch, col, row, v);
  }
};

// the last update: o = (alpha * X + beta * acc) 2^(-13 - e), stored as the result or applied to the weights
struct EpiLast {
  static constexpr bool kMirror = false;
  static constexpr int kLoads = 1;
  struct Pre {
    Pair8 x;
    u32x4 w0, w1;
  };
  Split x;
  Exponent ex;
  float alpha, beta;
  void* out;      // newton_schulz: [M][N] fp32 (dtype 0) or bf16 (1)
  int out_dtype;
  float* w;       // muon_step: fp32 [M][N], updated in place (out is null then)
  float lr, scale, wd;
  int vec;        // 8 columns of a row may be moved in 16-byte pieces

  __device__ __forceinline__ int word(int batch) const { return ex.e[batch]; }
  __device__ __forceinline__ EpiLast with(int word) const {
    EpiLast e = *this;
    e.alpha = ex.scaled(alpha, word);
    e.beta = ex.scaled(beta, word);
    return e;
  }
  __device__ __forceinline__ bool whole() const { return vec != 0; }
  __device__ __forceinline__ Pre load(const NtArgs& g, int batch, int row, int col) const {
    Pre p = {};
    if (vec && row < g.M && col < g.N) {
      p.x = load_pair(x, batch, row, col);
      if (w != nullptr) load8(w, (static_cast<int64_t>(batch) * g.M + row) * g.N + col, 0, p.w0, p.w1);
    }
    return p;
  }
  __device__ __forceinline__ void store(const NtArgs& g, int batch, int row, int col, float (&v)[8], const Pre& p) const {
    if (row >= g.M || col >= g.N) return;
    const int64_t o = (static_cast<int64_t>(batch) * g.M + row) * g.N + col;
    float t[8], wv[8];
    join8(p.x.h, p.x.l, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(alpha, t[e], beta * v[e]) * kSplitInv;
    if (w != nullptr) {
      unpack8(p.w0, p.w1, 0, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = wv[e] - lr * (scale * v[e] + wd * wv[e]);
      store8(w, o, 0, v);
    } else {
      store8(out, o, out_dtype, v);
    }
  }
  __device__ __forceinline__ void load_rows(const NtArgs& g, int batch, int row, int col, float (&t)[8]) const {
    uint16_t h[8], l[8];
    ragged8(row, g.M, col, x.ld, [&](int e, int r, int c) {
      const uint16_t* q = x.p + x.at(batch, r, c);
      h[e] = q[0];
      l[e] = q[32];
    });
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = f16_bits_to_f32(h[e]) + f16_bits_to_f32(l[e]);
  }
  __device__ __forceinline__ void store_rows(const NtArgs& g, int batch, int row, int col, const float (&v)[8],
                                             const float (&t)[8]) const {
    const int64_t o = (static_cast<int64_t>(batch) * g.M + row) * g.N + col;
    float u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = __builtin_fmaf(alpha, t[e], beta * v[e]) * kSplitInv;
    if (w != nullptr) {
      float wv[8];
      ragged8(row, g.M, col, g.N, [&](int e, int r, int c) { wv[e] = w[element_at(batch, r, g.M, c, g.N)]; });
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = wv[e] - lr * (scale * u[e] + wd * wv[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (row + e >= g.M) continue;
      if (w != nullptr)
        w[o + static_cast<int64_t>(e) * g.N] = u[e];
      else
        store1(out, o + static_cast<int64_t>(e) * g.N, out_dtype, u[e]);
    }
  }
};

// --------------------------------------------------------------- norm, momentum, first split
constexpr int kPartMax = 512;    // partial sums of one matrix
constexpr int kPerPart = 8192;   // elements of one partial sum at least

// Where a matrix's elements start on a 16-byte boundary (vec), values are taken four at a time.
__device__ __forceinline__ void grad4(const Source& s, int64_t i, float (&g)[4]) {
  if (s.dtype == 0) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(static_cast<const float*>(s.g) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = v[e];
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(s.g) + i);
    g[0] = bf16_lo(v[0]);
    g[1] = bf16_hi(v[0]);
    g[2] = bf16_lo(v[1]);
    g[3] = bf16_hi(v[1]);
  }
}

// sum over a workgroup of 256 in a fixed order (all threads get it)
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[4];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// sum of the squares of U over one share of a matrix, in fp64 (exact products); with a momentum
// buffer, m <- mu m + g first and U = g + mu m (nesterov) or m.  HBM bound: one read of g (and of m,
// with its write: 12288x4096 600 MB in 100 us).
__global__ __launch_bounds__(256) void norm_kernel(const Source s, int64_t elems, int parts, int vec, double* __restrict__ sums) {
  const int batch = blockIdx.y;
  const int64_t base = static_cast<int64_t>(batch) * elems;
  double acc = 0.0;
  auto one = [&](float g, float& m) {
    float u = g;
    if (s.m != nullptr) {
      m = __builtin_fmaf(s.mu, m, g);
      u = s.nesterov ? __builtin_fmaf(s.mu, m, g) : m;
    }
    acc = __builtin_fma(static_cast<double>(u), static_cast<double>(u), acc);
  };
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<int64_t>(parts) * 256;
  if (vec) {
#pragma unroll 4
    for (int64_t i = t; i < elems / 4; i += step) {
      float g[4], m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      grad4(s, base + 4 * i, g);
      if (s.m != nullptr) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(s.m + base + 4 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = v[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) one(g[e], m[e]);
      if (s.m != nullptr) *reinterpret_cast<f32x4*>(s.m + base + 4 * i) = f32x4{m[0], m[1], m[2], m[3]};
    }
  } else {
    for (int64_t i = t; i < elems; i += step) {
      float m = s.m != nullptr ? s.m[base + i] : 0.0f;
      one(grad_at(s, base + i), m);
      if (s.m != nullptr) s.m[base + i] = m;
    }
  }
  acc = block_sum(acc);
  if (threadIdx.x == 0) sums[static_cast<int64_t>(batch) * parts + blockIdx.x] = acc;
}

// U / (||U|| + eps) 2^E, split, [rows][ld] with the rows' ends zero, and E; 8 values of a row per thread.  HBM
// bound: one read of g (and m), 4 bytes written per value (12288x4096: 600 MB in 112 us).
__global__ __launch_bounds__(256) void first_split_kernel(const Source s, int64_t rows, int cols, int parts, int vec,
                                                          const double* __restrict__ sums, double eps, int* __restrict__ exps,
                                                          const Split o) {
  const int batch = blockIdx.y;
  const double* sb = sums + static_cast<int64_t>(batch) * parts;
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) acc += sb[i];
  const double norm = __builtin_sqrt(block_sum(acc)), inv = 1.0 / (norm + eps);
  int top = 0;
  (void)__builtin_frexp(norm * inv, &top);  // ||X0|| < 2^top (a norm of 0, infinity or NaN: no exponent)
  const int up = norm * inv > 0.0 && top < 0 ? -top : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) exps[batch] = up;
  const double factor = __builtin_ldexp(inv, 13 + up);
  const int64_t base = static_cast<int64_t>(batch) * rows * cols;
  const int per_row = o.ld / 8;
  const int64_t n8 = rows * per_row;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / per_row;
    const int col = static_cast<int>(i - row * per_row) * 8;
    const int64_t at = base + row * cols + col;
    float g[8], m[8], v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = m[e] = 0.0f;
    if (vec) {  // cols is a multiple of 8: all eight values or none
      if (col < cols) {
        float a[4], b[4];
        grad4(s, at, a);
        grad4(s, at + 4, b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = a[e];
          g[4 + e] = b[e];
        }
        if (s.m != nullptr) {
          const f32x4 c = *reinterpret_cast<const f32x4*>(s.m + at), d = *reinterpret_cast<const f32x4*>(s.m + at + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            m[e] = c[e];
            m[4 + e] = d[e];
          }
        }
      }
    } else {
      for (int e = 0; e < 8; ++e)
        if (col + e < cols) {
          g[e] = grad_at(s, at + e);
          if (s.m != nullptr) m[e] = s.m[at + e];
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = s.m == nullptr ? g[e] : s.nesterov ? __builtin_fmaf(s.mu, m[e], g[e]) : m[e];
      // the padding stays zero even where the norm is not finite
      v[e] = col + e < cols ? static_cast<float>(static_cast<double>(u) * factor) : 0.0f;
    }
    store_pair(o, batch, row, col, v);
  }
}

// ------------------------------------------------------------------------- the products
template <bool AT, bool BT>
using Big = NtCfg<256, 256, 128, 64, 2, 2, true, AT, BT>;
template <bool AT, bool BT>
using Mid = NtCfg<128, 128, 64, 64, 2, 2, true, AT, BT>;
// no compute unit with two workgroups: eight wavefronts a tile (two on each SIMD) and a third stage buffer
// (2048x2048, five steps: 783 -> 772 and 765 -> 749 us)
template <bool AT, bool BT>
using MidAlone = NtCfg<128, 128, 64, 32, 2, 2, true, AT, BT, false, 3>;
template <bool AT, bool BT>
using Small = NtCfg<64, 64, 32, 32, 2, 2, true, AT, BT, true, 3>;

NtPlan ns_plan(int64_t batch, int64_t M, int64_t N, int64_t K, bool tri) {
  return nt_plan(batch, M, N, K, tri, 32, 2.4, true, true);
}

template <bool AT, bool BT, class Epi>
int ns_product(const NtArgs& g, const NtPlan& p, int tri, const Epi& e, void* ws, hipStream_t s) {
  if (p.kind == 0) return nt_launch<Big<AT, BT>, Epi>(g, p, tri, e, ws, s);
  if (p.kind == 1 && p.nblk <= kNtCus) return nt_launch<MidAlone<AT, BT>, Epi>(g, p, tri, e, ws, s);
  if (p.kind == 1) return nt_launch<Mid<AT, BT>, Epi>(g, p, tri, e, ws, s);
  if (p.kind == 2) return nt_launch<Small<AT, BT>, Epi>(g, p, tri, e, ws, s);
  return nt_launch_tiny<NtTinyCfg<2, 2, true, AT, BT, true>, Epi>(g, p, tri, e, s);
}

struct NsLayout {
  bool wide;            // rows <= cols
  int64_t n, np, ld;    // the smaller side, padded; X's row length (cols, padded)
  NtPlan gram, poly, upd;
  int parts;
  size_t sums, exps, x0, x1, aa, bb, part, total;  // byte offsets, end
};

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

NsLayout ns_layout(int64_t batch, int64_t rows, int64_t cols) {
  NsLayout l;
  l.wide = rows <= cols;
  l.n = l.wide ? rows : cols;
  l.np = (l.n + 31) / 32 * 32;
  l.ld = (cols + 31) / 32 * 32;
  l.gram = ns_plan(batch, l.n, l.n, l.wide ? l.ld : rows, true);
  l.poly = ns_plan(batch, l.n, l.n, l.np, true);
  l.upd = ns_plan(batch, rows, cols, l.np, false);
  const int64_t parts = (rows * cols + kPerPart - 1) / kPerPart;
  l.parts = static_cast<int>(parts < kPartMax ? parts : kPartMax);
  const size_t x_bytes = size_t(4) * batch * rows * l.ld, n_bytes = size_t(4) * batch * l.n * l.np;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up256(bytes);
    return at;
  };
  l.sums = take(sizeof(double) * batch * l.parts);
  l.exps = take(sizeof(int) * batch);
  l.x0 = take(x_bytes);
  l.x1 = take(x_bytes);
  l.aa = take(n_bytes);
  l.bb = take(n_bytes);
  size_t most = 0;
  for (const NtPlan* p : {&l.gram, &l.poly, &l.upd}) most = p->ws > most ? p->ws : most;
  l.part = take(most);
  l.total = o;
  return l;
}

}  // namespace
}  // namespace w4q

using namespace w4q;

bool w4q_ns_fits(int64_t batch, int64_t rows, int64_t cols) {
  if (batch > 65535 || rows > 131072 || cols > 131072) return false;
  const NsLayout l = ns_layout(batch, rows, cols);
  return nt_fits(l.gram) && nt_fits(l.poly) && nt_fits(l.upd);
}

size_t w4q_ns_workspace(int64_t batch, int64_t rows, int64_t cols) {
  // (short sides take either way, by the steps and coefficients of the call)
  const size_t products = ns_layout(batch, rows, cols).total;
  if (!w4q_thin(rows, cols)) return products;
  const size_t thin = w4q_thin_workspace(batch, rows, cols);
  return thin > products ? thin : products;
}

// The largest singular value that can occur before each step, from 1 at the start: the extremes of
// p(s) = a s + b s^3 + c s^5 on [0, M] are at M and where p' = 0.  false where X, A = X X^T or
// B = b A + c A^2 could leave the range of the fp16 parts.
bool w4q_ns_coeffs_ok(int steps, double a, double b, double c) {
  if (!__builtin_isfinite(a) || !__builtin_isfinite(b) || !__builtin_isfinite(c)) return false;
  const double lim = 7.9;  // 2^13 * 7.9 < 65504
  double top = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double t = top * top;
    if (t > lim) return false;
    double most = __builtin_fabs(b * t + c * t * t);
    if (c != 0.0) {
      const double v = -b / (2.0 * c);
      if (v > 0.0 && v < t) most = __builtin_fmax(most, __builtin_fabs(b * v + c * v * v));
    }
    if (most > lim) return false;
    auto p = [&](double s) { return __builtin_fabs(s * (a + s * s * (b + c * s * s))); };
    double next = p(top);
    double roots[2];
    int nr = 0;
    if (c != 0.0) {
      const double d = 9.0 * b * b - 20.0 * a * c;
      if (d >= 0.0) {
        roots[nr++] = (-3.0 * b + __builtin_sqrt(d)) / (10.0 * c);
        roots[nr++] = (-3.0 * b - __builtin_sqrt(d)) / (10.0 * c);
      }
    } else if (b != 0.0) {
      roots[nr++] = -a / (3.0 * b);
    }
    for (int r = 0; r < nr; ++r)
      if (roots[r] > 0.0 && roots[r] < t) next = __builtin_fmax(next, p(__builtin_sqrt(roots[r])));
    top = next * 1.001;  // roundings of the step
    if (!(top < 1e30)) return false;
  }
  return true;
}

// h_s of the exponents (at the top): the bits by which singular values up to 1 can grow in s steps
static int growth_bits(int s, double a, double b, double c) {
  double g = __builtin_fmax(1.0, __builtin_fmax(__builtin_fabs(a), __builtin_fabs(a + b + c)));
  const double t = c != 0.0 ? -b / (2.0 * c) : 0.0;  // where a + b t + c t^2 turns
  if (t > 0.0 && t < 1.0) g = __builtin_fmax(g, __builtin_fabs(a + t * (b + c * t)));
  return static_cast<int>(__builtin_ceil(s * __builtin_log2(g)));
}

// newton_schulz: g -> out.  muon_step: m != null, w updated in place.
int w4q_launch_ns(const void* g, int g_dtype, int64_t batch, int64_t rows, int64_t cols, int steps, float a, float b,
                  float c, double eps, void* out, int out_dtype, float* m, float mu, int nesterov, float* w, float lr,
                  float scale, float wd, void* ws, hipStream_t s) {
  const Source src = {g, g_dtype, m, mu, nesterov};
  if (w4q_thin(rows, cols) && w4q_thin_steps_ok(steps, a)) {
    const ThinOut o = {out, out_dtype, w, lr, scale, wd};
    return w4q_launch_ns_thin(src, batch, rows, cols, steps, a, b, c, eps, o, ws, s);
  }
  const NsLayout l = ns_layout(batch, rows, cols);
  uint8_t* base = static_cast<uint8_t*>(ws);
  double* sums = reinterpret_cast<double*>(base + l.sums);
  int* exps = reinterpret_cast<int*>(base + l.exps);
  auto split = [&](size_t off, int64_t m_rows, int64_t ld) {
    return Split{reinterpret_cast<uint16_t*>(base + off), static_cast<int>(ld), 2 * m_rows * ld};
  };
  const Split x[2] = {split(l.x0, rows, l.ld), split(l.x1, rows, l.ld)};
  const Split A = split(l.aa, l.n, l.np), B = split(l.bb, l.n, l.np);
  void* part = base + l.part;
  const int n = static_cast<int>(l.n), np = static_cast<int>(l.np);

  auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool vec = cols % 8 == 0 && at16(g) && (m == nullptr || at16(m));
  hipLaunchKernelGGL(norm_kernel, dim3(static_cast<unsigned>(l.parts), static_cast<unsigned>(batch)), dim3(256), 0, s, src,
                     rows * cols, l.parts, vec ? 1 : 0, sums);
  int rc = w4q_launch_status();
  if (rc != W4Q_OK) return rc;
  const int64_t blocks = (rows * l.ld / 8 + 255) / 256;
  hipLaunchKernelGGL(first_split_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096), static_cast<unsigned>(batch)),
                     dim3(256), 0, s, src, rows, static_cast<int>(cols), l.parts, vec ? 1 : 0, sums, eps, exps, x[0]);
  rc = w4q_launch_status();

  auto operand = [](const Split& m, const uint16_t*& p, int64_t& stride, int& ld) {
    p = m.p;
    stride = m.stride;
    ld = 2 * m.ld;
  };
  int cur = 0;
  for (int i = 0; i < steps && rc == W4Q_OK; ++i, cur ^= 1) {
    const Split& X = x[cur];
    const int h = growth_bits(i, a, b, c), next = growth_bits(i + 1, a, b, c);
    // A = X X^T (Y^T Y)
    NtArgs ga = {};
    operand(X, ga.a, ga.sa, ga.lda);
    operand(X, ga.b, ga.sb, ga.ldb);
    ga.M = ga.N = n;
    ga.K = static_cast<int>(l.wide ? l.ld : rows);
    ga.ka = ga.kb = static_cast<int>(rows);
    EpiSplit<true> e = {};
    e.beta = kSplitInv;
    e.o = A;
    e.ex = {exps, h, 2, kNoExponent};
    rc = l.wide ? ns_product<false, false>(ga, l.gram, 1, e, part, s) : ns_product<true, true>(ga, l.gram, 1, e, part, s);
    if (rc != W4Q_OK) break;
    // B = b A + c A A
    NtArgs gb = {};
    operand(A, gb.a, gb.sa, gb.lda);
    operand(A, gb.b, gb.sb, gb.ldb);
    gb.M = gb.N = n;
    gb.K = np;
    e.c = A;
    e.alpha = b;
    e.beta = c * kSplitInv;
    e.o = B;
    e.ex = {};
    if ((rc = ns_product<false, false>(gb, l.poly, 1, e, part, s)) != W4Q_OK) break;
    // X <- a X + B X (Y <- a Y + Y B)
    NtArgs gx = {};
    operand(l.wide ? B : X, gx.a, gx.sa, gx.lda);
    operand(l.wide ? X : B, gx.b, gx.sb, gx.ldb);
    gx.M = static_cast<int>(rows);
    gx.N = static_cast<int>(cols);
    gx.K = np;
    gx.kb = static_cast<int>(rows);
    if (i + 1 < steps) {
      EpiSplit<false> u = {};
      u.c = X;
      u.alpha = a;
      u.beta = kSplitInv;
      u.o = x[cur ^ 1];
      u.ex = {exps, h, 1, next};
      rc = l.wide ? ns_product<false, true>(gx, l.upd, 0, u, part, s) : ns_product<false, false>(gx, l.upd, 0, u, part, s);
    } else {
      EpiLast u = {};
      u.x = X;
      u.ex = {exps, h, 1, kNoExponent};
      u.alpha = a;
      u.beta = kSplitInv;
      u.out = out;
      u.out_dtype = out_dtype;
      u.w = w;
      u.lr = lr;
      u.scale = scale;
      u.wd = wd;
      u.vec = cols % 8 == 0 && at16(w != nullptr ? static_cast<void*>(w) : out);
      rc = l.wide ? ns_product<false, true>(gx, l.upd, 0, u, part, s) : ns_product<false, false>(gx, l.upd, 0, u, part, s);
    }
  }
  return rc;
}
