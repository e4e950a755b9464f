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
//
// Work per step: A and A^2 are symmetric (tiles on and below the diagonal only, the others stored
// mirrored), B X is whole: n^2 k + n^3 + 2 n^2 k flop, times three products.  Matrix-core bound from
// n of about 1024 up; below that the chain of dependent launches is what costs.
//
// Layouts: the products run along rows of both operands, so X is kept as XN [n][k] (the Gram
// product) and XT [k][n] (the update); each epilogue writes both.  XN is updated in place (element by
// element), XT alternates between two buffers (other tiles still read the old one).
#include "nt_gemm.hpp"

namespace w4q {
namespace {

constexpr float kSplitScale = 8192.0f;  // 2^13
constexpr float kSplitInv = 1.0f / 8192.0f;

// hi and lo of a scaled value (both RNE)
__device__ __forceinline__ void split16(float v, uint16_t& h, uint16_t& l) {
  const _Float16 hi = static_cast<_Float16>(v);
  h = __builtin_bit_cast(uint16_t, hi);
  l = f32_to_f16_bits(v - static_cast<float>(hi));
}

// ------------------------------------------------------------------------- epilogues
// alpha * C + beta * acc, split, to the output and (transposed) to the second output
struct EpiSplit {
  const uint16_t *ch, *cl;  // C term or null
  int ldc;
  int64_t sc;
  float alpha, beta;
  uint16_t *oh, *ol;
  int ldo;
  int64_t so;
  uint16_t *th, *tl;  // transposed output [N][ldt]
  int ldt;
  int64_t st;
  int mirror;  // symmetric result: the transposed store only off the diagonal tiles

  __device__ __forceinline__ void operator()(const NtArgs& g, int batch, int row0, int col0, bool diag,
                                             const f32x16& acc, int lane) const {
    const int col = col0 + (lane & 31);
    const bool tr = col < g.N && !(mirror != 0 && diag);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int rq = row0 + 8 * q + 4 * (lane >> 5);
      u16x4 h4, l4;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = rq + e;
        const bool in = row < g.M && col < ldo;
        float v = beta * acc[4 * q + e];
        if (ch != nullptr && in) {
          const int64_t o = batch * sc + static_cast<int64_t>(row) * ldc + col;
          v = __builtin_fmaf(alpha, f16_bits_to_f32(ch[o]) + f16_bits_to_f32(cl[o]), v);
        }
        uint16_t h, l;
        split16(v, h, l);
        h4[e] = h;
        l4[e] = l;
        if (in) {
          const int64_t o = batch * so + static_cast<int64_t>(row) * ldo + col;
          oh[o] = h;
          ol[o] = l;
        }
      }
      if (tr && rq < ldt) {  // ldt is a multiple of 32 and rq of 4: all four rows or none
        const int64_t o = batch * st + static_cast<int64_t>(col) * ldt + rq;
        *reinterpret_cast<u16x4*>(th + o) = h4;
        *reinterpret_cast<u16x4*>(tl + o) = l4;
      }
    }
  }
};

// the last update: o = (alpha * C + beta * acc) 2^-13, stored as the result or applied to the weights
struct EpiLast {
  const uint16_t *ch, *cl;
  int ldc;
  int64_t sc;
  float alpha, beta;
  void* out;       // newton_schulz: [M][N] fp32 (dtype 0) or bf16 (1)
  int out_dtype;
  float* w;        // muon_step: fp32 [M][N], updated in place (out is null then)
  float lr, scale, wd;

  __device__ __forceinline__ void operator()(const NtArgs& g, int batch, int row0, int col0, bool, const f32x16& acc,
                                             int lane) const {
    const int col = col0 + (lane & 31);
    if (col >= g.N) return;
    const int64_t base = static_cast<int64_t>(batch) * g.M * g.N;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = row0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (row >= g.M) continue;
      const int64_t o = batch * sc + static_cast<int64_t>(row) * ldc + col;
      const float x = f16_bits_to_f32(ch[o]) + f16_bits_to_f32(cl[o]);
      const float v = __builtin_fmaf(alpha, x, beta * acc[r]) * kSplitInv;
      const int64_t y = base + static_cast<int64_t>(row) * g.N + col;
      if (w != nullptr) {
        const float wv = w[y];
        w[y] = wv - lr * (scale * v + wd * wv);
      } else if (out_dtype == 0) {
        static_cast<float*>(out)[y] = v;
      } else {
        static_cast<uint16_t*>(out)[y] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
      }
    }
  }
};

// --------------------------------------------------------------- norm, momentum, first split
constexpr int kPartMax = 512;    // partial sums of one matrix
constexpr int kPerPart = 8192;   // elements of one partial sum at least

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

// sum of the squares of U over one share of a matrix, in fp64 (exact products); with a momentum
// buffer, m <- mu m + g first and U = g + mu m (nesterov) or m.  HBM bound: one read of g (and of m,
// with its write).
__global__ __launch_bounds__(256) void norm_kernel(const Source s, int64_t elems, int parts, double* __restrict__ sums) {
  const int batch = blockIdx.y;
  const int64_t base = static_cast<int64_t>(batch) * elems;
  double acc = 0.0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < elems; i += static_cast<int64_t>(parts) * 256) {
    const float g = grad_at(s, base + i);
    float u = g;
    if (s.m != nullptr) {
      const float m = __builtin_fmaf(s.mu, s.m[base + i], g);
      s.m[base + i] = m;
      u = s.nesterov ? __builtin_fmaf(s.mu, m, g) : m;
    }
    acc = __builtin_fma(static_cast<double>(u), static_cast<double>(u), acc);
  }
  __shared__ double red[256];
  red[threadIdx.x] = acc;
  __syncthreads();
#pragma unroll
  for (int o = 128; o >= 1; o >>= 1) {
    if (static_cast<int>(threadIdx.x) < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) sums[static_cast<int64_t>(batch) * parts + blockIdx.x] = red[0];
}

// U / (||U|| + eps), split, in both layouts: P [rows][cp] as U lies and Q [cols][rp] transposed, the
// rows' ends up to the next multiple of 32 zero.  64x64 tiles through LDS.
__global__ __launch_bounds__(256) void first_split_kernel(const Source s, int rows, int cols, int parts,
                                                          const double* __restrict__ sums, double eps,
                                                          uint16_t* __restrict__ ph, uint16_t* __restrict__ pl, int cp,
                                                          uint16_t* __restrict__ qh, uint16_t* __restrict__ ql, int rp) {
  __shared__ double red[256];
  __shared__ uint32_t tile[64][65];
  const int batch = blockIdx.z;
  const double* sb = sums + static_cast<int64_t>(batch) * parts;
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) acc += sb[i];
  red[threadIdx.x] = acc;
  __syncthreads();
#pragma unroll
  for (int o = 128; o >= 1; o >>= 1) {
    if (static_cast<int>(threadIdx.x) < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  const double inv = 1.0 / (__builtin_sqrt(red[0]) + eps);

  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int64_t base = static_cast<int64_t>(batch) * rows * cols;
  const int64_t pb = static_cast<int64_t>(batch) * rows * cp, qb = static_cast<int64_t>(batch) * cols * rp;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int row = r0 + ty + 4 * i, col = c0 + tx;
    uint32_t packed = 0;
    if (row < rows && col < cols) {
      const int64_t o = base + static_cast<int64_t>(row) * cols + col;
      const float g = grad_at(s, o);
      float u = g;
      if (s.m != nullptr) u = s.nesterov ? __builtin_fmaf(s.mu, s.m[o], g) : s.m[o];
      const float x = static_cast<float>(static_cast<double>(u) * inv) * kSplitScale;
      uint16_t h, l;
      split16(x, h, l);
      packed = h | (static_cast<uint32_t>(l) << 16);
    }
    tile[ty + 4 * i][tx] = packed;
    if (row < rows && col < cp) {
      ph[pb + static_cast<int64_t>(row) * cp + col] = static_cast<uint16_t>(packed);
      pl[pb + static_cast<int64_t>(row) * cp + col] = static_cast<uint16_t>(packed >> 16);
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int col = c0 + ty + 4 * i, row = r0 + tx;
    if (col < cols && row < rp) {
      const uint32_t packed = tile[tx][ty + 4 * i];
      qh[qb + static_cast<int64_t>(col) * rp + row] = static_cast<uint16_t>(packed);
      ql[qb + static_cast<int64_t>(col) * rp + row] = static_cast<uint16_t>(packed >> 16);
    }
  }
}

// ------------------------------------------------------------------------- the products
using Big = NtCfg<256, 256, 128, 64, 2, 2, true, 2>;
using Mid = NtCfg<128, 128, 64, 64, 2, 2, true, 2>;
using Small = NtCfg<64, 64, 32, 32, 2, 2, true, 3>;

struct NsPlan {
  int kind;  // 0 Big, 1 Mid, 2 Small
  NtPlan p;
};

// Tile size by how many tiles there are: the largest one that still gives most compute units work.
NsPlan ns_plan(int64_t batch, int64_t M, int64_t N, int64_t K, bool tri) {
  NsPlan r;
  r.p = nt_plan(batch, M, N, K, tri, Big::BM, Big::BN, kNtCus);
  r.kind = 0;
  if (batch * r.p.per_batch >= 96) return r;
  r.p = nt_plan(batch, M, N, K, tri, Mid::BM, Mid::BN, 2 * kNtCus);
  r.kind = 1;
  if (batch * r.p.per_batch >= 128) return r;
  r.p = nt_plan(batch, M, N, K, tri, Small::BM, Small::BN, 3 * kNtCus);
  r.kind = 2;
  return r;
}

template <class Epi>
int ns_product(const NtArgs& g, const NsPlan& r, int tri, const Epi& e, void* ws, hipStream_t s) {
  if (r.kind == 0) return nt_launch<Big, Epi>(g, r.p, tri, e, ws, s);
  if (r.kind == 1) return nt_launch<Mid, Epi>(g, r.p, tri, e, ws, s);
  return nt_launch<Small, Epi>(g, r.p, tri, e, ws, s);
}

struct NsLayout {
  int64_t n, k, np, kp;
  NsPlan gram, poly, upd, last;
  int parts;
  size_t sums, xn, xt, aa, bb, part, total;  // byte offsets (each hi then lo), end
  size_t xn1, xt1, nn1;                      // bytes of one part
};

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

NsLayout ns_layout(int64_t batch, int64_t rows, int64_t cols) {
  NsLayout l;
  l.n = rows < cols ? rows : cols;
  l.k = rows < cols ? cols : rows;
  l.np = (l.n + 31) / 32 * 32;
  l.kp = (l.k + 31) / 32 * 32;
  l.gram = ns_plan(batch, l.n, l.n, l.kp, true);
  l.poly = ns_plan(batch, l.n, l.n, l.np, true);
  l.upd = ns_plan(batch, l.n, l.k, l.np, false);
  l.last = rows <= cols ? l.upd : ns_plan(batch, l.k, l.n, l.np, false);
  const int64_t parts = (rows * cols + kPerPart - 1) / kPerPart;
  l.parts = static_cast<int>(parts < kPartMax ? parts : kPartMax);
  l.xn1 = up256(size_t(2) * batch * l.n * l.kp);
  l.xt1 = up256(size_t(2) * batch * l.k * l.np);
  l.nn1 = up256(size_t(2) * batch * l.n * l.np);
  size_t o = 0;
  l.sums = o;
  o += up256(sizeof(double) * batch * l.parts);
  l.xn = o;
  o += 2 * l.xn1;
  l.xt = o;
  o += 4 * l.xt1;  // two of them
  l.aa = o;
  o += 2 * l.nn1;
  l.bb = o;
  o += 2 * l.nn1;
  l.part = o;
  size_t most = 0;
  for (const NsPlan* p : {&l.gram, &l.poly, &l.upd, &l.last}) most = p->p.ws > most ? p->p.ws : most;
  l.total = o + up256(most);
  return l;
}

}  // namespace
}  // namespace w4q

using namespace w4q;

bool w4q_ns_fits(int64_t batch, int64_t rows, int64_t cols) {
  if (batch > 65535 || rows > 131072 || cols > 131072) return false;
  const NsLayout l = ns_layout(batch, rows, cols);
  for (const NsPlan* p : {&l.gram, &l.poly, &l.upd, &l.last})
    if (p->p.total > 0x3FFFFFFF) return false;
  return true;
}

size_t w4q_ns_workspace(int64_t batch, int64_t rows, int64_t cols) { return ns_layout(batch, rows, cols).total; }

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

// newton_schulz: g -> out.  muon_step: m != null, w updated in place.
int w4q_launch_ns(const void* g, int g_dtype, int64_t batch, int64_t rows, int64_t cols, int steps, float a, float b,
                  float c, double eps, void* out, int out_dtype, float* m, float mu, int nesterov, float* w, float lr,
                  float scale, float wd, void* ws, hipStream_t s) {
  const NsLayout l = ns_layout(batch, rows, cols);
  uint8_t* base = static_cast<uint8_t*>(ws);
  double* sums = reinterpret_cast<double*>(base + l.sums);
  auto u16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(base + off); };
  uint16_t *xnh = u16(l.xn), *xnl = u16(l.xn + l.xn1);
  uint16_t* xth[2] = {u16(l.xt), u16(l.xt + 2 * l.xt1)};
  uint16_t* xtl[2] = {u16(l.xt + l.xt1), u16(l.xt + 3 * l.xt1)};
  uint16_t *ah = u16(l.aa), *al = u16(l.aa + l.nn1);
  uint16_t *bh = u16(l.bb), *bl = u16(l.bb + l.nn1);
  void* part = base + l.part;
  const bool wide = rows <= cols;
  const int n = static_cast<int>(l.n), k = static_cast<int>(l.k), np = static_cast<int>(l.np), kp = static_cast<int>(l.kp);
  const int64_t sxn = l.n * l.kp, sxt = l.k * l.np, snn = l.n * l.np;

  const Source src = {g, g_dtype, m, mu, nesterov};
  hipLaunchKernelGGL(norm_kernel, dim3(static_cast<unsigned>(l.parts), static_cast<unsigned>(batch)), dim3(256), 0, s, src,
                     rows * cols, l.parts, sums);
  int rc = w4q_launch_status();
  if (rc != W4Q_OK) return rc;
  const int cp = wide ? kp : np, rp = wide ? np : kp;
  hipLaunchKernelGGL(first_split_kernel,
                     dim3(static_cast<unsigned>((cols + 63) / 64), static_cast<unsigned>((rows + 63) / 64),
                          static_cast<unsigned>(batch)),
                     dim3(256), 0, s, src, static_cast<int>(rows), static_cast<int>(cols), l.parts, sums, eps,
                     wide ? xnh : xth[0], wide ? xnl : xtl[0], cp, wide ? xth[0] : xnh, wide ? xtl[0] : xnl, rp);
  rc = w4q_launch_status();
  int cur = 0;
  for (int i = 0; i < steps && rc == W4Q_OK; ++i) {
    // A = X X^T
    NtArgs ga = {};
    ga.a[0] = ga.b[0] = xnh;
    ga.a[1] = ga.b[1] = xnl;
    ga.sa = ga.sb = sxn;
    ga.M = ga.N = n;
    ga.K = kp;
    ga.lda = ga.ldb = kp;
    EpiSplit e = {};
    e.beta = kSplitInv;
    e.oh = e.th = ah;
    e.ol = e.tl = al;
    e.ldo = e.ldt = np;
    e.so = e.st = snn;
    e.mirror = 1;
    if ((rc = ns_product(ga, l.gram, 1, e, part, s)) != W4Q_OK) break;
    // B = b A + c A A
    NtArgs gb = ga;
    gb.a[0] = gb.b[0] = ah;
    gb.a[1] = gb.b[1] = al;
    gb.sa = gb.sb = snn;
    gb.K = np;
    gb.lda = gb.ldb = np;
    e.ch = ah;
    e.cl = al;
    e.ldc = np;
    e.sc = snn;
    e.alpha = b;
    e.beta = c * kSplitInv;
    e.oh = e.th = bh;
    e.ol = e.tl = bl;
    if ((rc = ns_product(gb, l.poly, 1, e, part, s)) != W4Q_OK) break;
    // X <- a X + B X
    NtArgs gx = {};
    gx.K = np;
    gx.lda = gx.ldb = np;
    if (i + 1 < steps) {
      gx.a[0] = bh;
      gx.a[1] = bl;
      gx.sa = snn;
      gx.b[0] = xth[cur];
      gx.b[1] = xtl[cur];
      gx.sb = sxt;
      gx.M = n;
      gx.N = k;
      EpiSplit u = {};
      u.ch = xnh;
      u.cl = xnl;
      u.ldc = kp;
      u.sc = sxn;
      u.alpha = a;
      u.beta = kSplitInv;
      u.oh = xnh;
      u.ol = xnl;
      u.ldo = kp;
      u.so = sxn;
      u.th = xth[cur ^ 1];
      u.tl = xtl[cur ^ 1];
      u.ldt = np;
      u.st = sxt;
      rc = ns_product(gx, l.upd, 0, u, part, s);
      cur ^= 1;
    } else {
      EpiLast u = {};
      u.alpha = a;
      u.beta = kSplitInv;
      u.out = out;
      u.out_dtype = out_dtype;
      u.w = w;
      u.lr = lr;
      u.scale = scale;
      u.wd = wd;
      if (wide) {
        gx.a[0] = bh;
        gx.a[1] = bl;
        gx.sa = snn;
        gx.b[0] = xth[cur];
        gx.b[1] = xtl[cur];
        gx.sb = sxt;
        gx.M = n;
        gx.N = k;
        u.ch = xnh;
        u.cl = xnl;
        u.ldc = kp;
        u.sc = sxn;
      } else {
        gx.a[0] = xth[cur];
        gx.a[1] = xtl[cur];
        gx.sa = sxt;
        gx.b[0] = bh;
        gx.b[1] = bl;
        gx.sb = snn;
        gx.M = k;
        gx.N = n;
        u.ch = xth[cur];
        u.cl = xtl[cur];
        u.ldc = np;
        u.sc = sxt;
      }
      rc = ns_product(gx, l.last, 0, u, part, s);
    }
  }
  return rc;
}
