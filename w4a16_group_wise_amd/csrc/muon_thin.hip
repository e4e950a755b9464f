// muon_thin.hip -- the orthogonalised update for matrices with a short side n <= 64 and few steps
// (muon.hip has the others): three launches instead of two and three per step.
//
// Every iterate is a polynomial in A = X0 X0^T applied to X0, and those polynomials commute, so the
// steps can be taken on n x n matrices alone (X is n x k, k >= n):
//   Q = I;   steps times:  P = a I + b A + c A^2;  Q <- P Q;  A <- P A P;      result Q X0
// Squaring costs half the digits of small singular values, which later steps multiply by up to a^2 =
// 11.9 each: A and all products of it are fp64 (fp32 inputs give exact products), which leaves them
// beyond fp32's digits after five steps.  ||X||_F^2 is the trace of the unscaled A, so the norm needs
// no pass of its own.
//
//   thin_gram_kernel     partial sums of U U^T over ranges of k (and the momentum update)
//   thin_steps_kernel    one workgroup per matrix: sum of the partials, the steps, in LDS
//   thin_apply_kernel    Q U / (||U|| + eps), with the weight update
// Bound by the three launches and the chain of n x n products up to a few thousand k; beyond, by the at most 32
// workgroups of thin_gram_kernel that a single matrix gets, each walking its range tile by tile.
// Measured, five steps: n up to 32 21 to 24 us (86 with the products on X), 64x1024 56 us, 12288x48 64 us.
#include "epilogue.hpp"
#include "muon.hpp"

namespace w4q {
namespace {

constexpr int kThinMax = 64;
constexpr int kThinK = 64;       // k of a tile in LDS
constexpr int kThinParts = 32;   // ranges of k at most

// Element (j, kk) of U as X lies: wide U is [n][k], tall U is [k][n]
struct Thin {
  int n, wide;
  int64_t k, stride;  // values of one matrix
  __device__ __forceinline__ int64_t at(int j, int64_t kk) const { return wide ? j * k + kk : kk * n + j; }
};

// Tile kk0 .. kk0 + kThinK - 1 of U in memory order (accesses of a wavefront are consecutive), eight
// elements per thread at a time with their loads in flight together: v = load(position), then
// use(row, column in the tile, position, v).  256 threads.
template <class Load, class Use>
__device__ __forceinline__ void thin_tile(const Thin& t, int64_t kk0, Load load, Use use) {
  constexpr int B = 8;
  const int left = static_cast<int>(t.k - kk0 < kThinK ? t.k - kk0 : kThinK);
  const int total = t.n * left;
  const int len = t.wide ? left : t.n;  // values of a row of the tile in memory
  const float inv_len = 1.0f / static_cast<float>(len);
  for (int e0 = threadIdx.x; e0 < total; e0 += 256 * B) {
    int j[B], kk[B];
    int64_t at[B];
    decltype(load(int64_t(0))) v[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int e = e0 + 256 * i < total ? e0 + 256 * i : e0;  // past the end: the first again, not used
      // e / len by the reciprocal: e < 2^12, so half a unit in e outweighs the roundings
      const int row = static_cast<int>((static_cast<float>(e) + 0.5f) * inv_len), col = e - row * len;
      j[i] = t.wide ? row : col;
      kk[i] = t.wide ? col : row;
      at[i] = t.at(j[i], kk0 + kk[i]);
      v[i] = load(at[i]);
    }
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (e0 + 256 * i < total) use(j[i], kk[i], at[i], v[i]);
  }
}

// Products on the fp64 matrix cores (16x16x4): lane l supplies A[l % 16][l / 16] and B[l / 16][l % 16],
// and result register r is D[4 r + l / 16][l % 16].
typedef double f64x4 __attribute__((ext_vector_type(4)));

// tile p of those on and below the diagonal, row by row (at most 10 of them)
__device__ __forceinline__ void thin_lower(int p, int& ti, int& tj) {
  ti = p >= 6 ? 3 : p >= 3 ? 2 : p >= 1 ? 1 : 0;
  tj = p - ti * (ti + 1) / 2;
}

struct GradMom {
  float g, m;
};

template <int N>
__global__ __launch_bounds__(256) void thin_gram_kernel(const Source s, const Thin t, int parts, int64_t per,
                                                        double* __restrict__ sums) {
  // 16x16 tiles on and below the diagonal, dealt to the four wavefronts
  constexpr int kTiles = N / 16, kLower = kTiles * (kTiles + 1) / 2, kPerWave = (kLower + 3) / 4;
  __shared__ float u[kThinK][N + 1];
  const int batch = blockIdx.y;
  const int64_t base = batch * t.stride;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  int ti[kPerWave], tj[kPerWave];
#pragma unroll
  for (int c = 0; c < kPerWave; ++c) thin_lower(wid + 4 * c < kLower ? wid + 4 * c : 0, ti[c], tj[c]);
  f64x4 acc[kPerWave];
#pragma unroll
  for (int c = 0; c < kPerWave; ++c) acc[c] = f64x4{0.0, 0.0, 0.0, 0.0};
  const int64_t k0 = blockIdx.x * per, k1 = k0 + per < t.k ? k0 + per : t.k;
  for (int64_t kk0 = k0; kk0 < k1; kk0 += kThinK) {
    for (int e = threadIdx.x; e < kThinK * (N + 1); e += 256) (&u[0][0])[e] = 0.0f;
    __syncthreads();
    thin_tile(
        t, kk0,
        [&](int64_t at) { return GradMom{grad_at(s, base + at), s.m != nullptr ? s.m[base + at] : 0.0f}; },
        [&](int j, int kk, int64_t at, GradMom v) {
          if (s.m != nullptr) {
            v.m = __builtin_fmaf(s.mu, v.m, v.g);
            s.m[base + at] = v.m;
          }
          u[kk][j] = update_at(s, v.g, v.m);
        });
    __syncthreads();
#pragma unroll 8
    for (int kk = 0; kk < kThinK; kk += 4) {
      const float* row = u[kk + (lane >> 4)];
#pragma unroll
      for (int c = 0; c < kPerWave; ++c)
        acc[c] = __builtin_amdgcn_mfma_f64_16x16x4f64(static_cast<double>(row[16 * ti[c] + (lane & 15)]),
                                                      static_cast<double>(row[16 * tj[c] + (lane & 15)]), acc[c], 0, 0, 0);
    }
    __syncthreads();
  }
  double* o = sums + (static_cast<int64_t>(batch) * parts + blockIdx.x) * (kLower * 256);
#pragma unroll
  for (int c = 0; c < kPerWave; ++c) {
    if (wid + 4 * c >= kLower) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[((wid + 4 * c) * 4 + r) * 64 + lane] = acc[c][r];  // tile by tile
  }
}

// The wavefront's 16x16 tile (ti, tj) of X Y and, with kTwo, of X Z, for N x N matrices in LDS (pitch N + 1)
template <int N, bool kTwo>
__device__ __forceinline__ void thin_mul(const double* x, const double* y, const double* z, int ti, int tj, int lane,
                                         f64x4& xy, f64x4& xz) {
  constexpr int L = N + 1;
  f64x4 y0 = {0.0, 0.0, 0.0, 0.0}, y1 = y0, z0 = y0, z1 = y0;
  const double* a = x + (16 * ti + (lane & 15)) * L + (lane >> 4);
  const int b = (lane >> 4) * L + 16 * tj + (lane & 15);
#pragma unroll
  for (int p = 0; p < N; p += 8) {  // two chains of sums each, so that products overlap
    const double a0 = a[p], a1 = a[p + 4];
    y0 = __builtin_amdgcn_mfma_f64_16x16x4f64(a0, y[b + p * L], y0, 0, 0, 0);
    if constexpr (kTwo) z0 = __builtin_amdgcn_mfma_f64_16x16x4f64(a0, z[b + p * L], z0, 0, 0, 0);
    y1 = __builtin_amdgcn_mfma_f64_16x16x4f64(a1, y[b + (p + 4) * L], y1, 0, 0, 0);
    if constexpr (kTwo) z1 = __builtin_amdgcn_mfma_f64_16x16x4f64(a1, z[b + (p + 4) * L], z1, 0, 0, 0);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    xy[r] = y0[r] + y1[r];
    if constexpr (kTwo) xz[r] = z0[r] + z1[r];
  }
}

template <int N>
constexpr int step_threads() { return 64 * (N / 16) * (N / 16 + 1) / 2; }  // a wavefront per tile

template <int N>
__global__ __launch_bounds__(step_threads<N>()) void thin_steps_kernel(int n, int parts, const double* __restrict__ sums,
                                                                      int steps, double a, double b, double c, double eps,
                                                                      float* __restrict__ q_out, double* __restrict__ inv_out) {
  constexpr int L = N + 1, kLower = (N / 16) * (N / 16 + 1) / 2;
  __shared__ double A[N * L], P[N * L], Q[N * L];
  const int batch = blockIdx.x;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  int ti, tj;
  thin_lower(wid, ti, tj);
  // the wavefront's entries (16 ti + 4 r + lane / 16, 16 tj + lane % 16); all matrices are symmetric, so each
  // is stored with its mirror image
  const int i0 = 16 * ti + (lane >> 4), j0 = 16 * tj + (lane & 15);
  auto at = [&](int r) { return (i0 + 4 * r) * L + j0; };
  auto put = [&](double* m, int r, double v) {
    m[at(r)] = v;
    if (ti != tj) m[j0 * L + i0 + 4 * r] = v;
  };
  const double* sb = sums + static_cast<int64_t>(batch) * parts * (kLower * 256) + wid * 256 + lane;
  f64x4 x = {0.0, 0.0, 0.0, 0.0}, y = x;
#pragma unroll 8
  for (int p = 0; p < parts; ++p)
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] += sb[p * (kLower * 256) + 64 * r];
#pragma unroll
  for (int r = 0; r < 4; ++r) put(A, r, x[r]);
  __syncthreads();
  double trace = lane < n ? A[lane * L + lane] : 0.0;  // n <= 64: one entry per lane
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) trace += __shfl_xor(trace, o);
  const double inv = 1.0 / (__builtin_sqrt(trace) + eps);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 4; ++r) put(A, r, x[r] * inv * inv);
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    thin_mul<N, false>(A, A, nullptr, ti, tj, lane, x, y);
#pragma unroll
    for (int r = 0; r < 4; ++r) put(P, r, (i0 + 4 * r == j0 ? a : 0.0) + b * A[at(r)] + c * x[r]);
    __syncthreads();
    if (s == 0) {  // Q = P
#pragma unroll
      for (int r = 0; r < 4; ++r) put(Q, r, P[at(r)]);
      thin_mul<N, false>(P, A, nullptr, ti, tj, lane, x, y);
    } else {
      thin_mul<N, true>(P, A, Q, ti, tj, lane, x, y);
    }
    __syncthreads();
    if (s > 0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) put(Q, r, y[r]);
    }
    if (s + 1 == steps) break;
#pragma unroll
    for (int r = 0; r < 4; ++r) put(A, r, x[r]);  // P A
    __syncthreads();
    thin_mul<N, false>(A, P, nullptr, ti, tj, lane, x, y);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r) put(A, r, x[r]);  // P A P
    __syncthreads();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < N * N; e += step_threads<N>())
    q_out[static_cast<int64_t>(batch) * (N * N) + e] = static_cast<float>(Q[(e / N) * L + e % N]);
  if (threadIdx.x == 0) inv_out[batch] = inv;
}

// kThinK columns of the result: thread = (column, quarter of the rows); Q is symmetric, so its rows are
// read as columns.  The results go back through the tile, to be stored in memory order.
template <int N>
__global__ __launch_bounds__(256) void thin_apply_kernel(const Source s, const Thin t, const float* __restrict__ q_in,
                                                         const double* __restrict__ inv_in, const ThinOut o) {
  __shared__ float u[kThinK][N + 1];
  __shared__ __attribute__((aligned(16))) float q[N][N];
  const int batch = blockIdx.y;
  const int64_t base = batch * t.stride;
  const double inv = inv_in[batch];
  for (int i = threadIdx.x; i < N * N / 4; i += 256)
    reinterpret_cast<f32x4*>(&q[0][0])[i] = reinterpret_cast<const f32x4*>(q_in + static_cast<int64_t>(batch) * (N * N))[i];
  for (int e = threadIdx.x; e < kThinK * (N + 1); e += 256) (&u[0][0])[e] = 0.0f;
  __syncthreads();
  const int64_t kk0 = static_cast<int64_t>(blockIdx.x) * kThinK;
  thin_tile(
      t, kk0, [&](int64_t at) { return update_at(s, grad_at(s, base + at), s.m != nullptr ? s.m[base + at] : 0.0f); },
      [&](int j, int kk, int64_t, float v) { u[kk][j] = static_cast<float>(static_cast<double>(v) * inv); });
  __syncthreads();
  constexpr int kPer = N / 4;  // rows per thread
  const int kk = threadIdx.x & (kThinK - 1), row0 = threadIdx.x / kThinK * kPer;
  float acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < N; ++j) {
    const float x = u[kk][j];
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const f32x4 w = *reinterpret_cast<const f32x4*>(&q[j][row0 + 4 * i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[4 * i + e] = __builtin_fmaf(w[e], x, acc[4 * i + e]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) u[kk][row0 + i] = acc[i];
  __syncthreads();
  thin_tile(
      t, kk0, [&](int64_t at) { return o.w != nullptr ? o.w[base + at] : 0.0f; },
      [&](int j, int k1, int64_t at, float wv) {
        const float v = u[k1][j];
        if (o.w != nullptr)
          o.w[base + at] = wv - o.lr * (o.scale * v + o.wd * wv);
        else
          store1(o.out, base + at, o.out_dtype, v);
      });
}

struct ThinLayout {
  int n, N, parts;
  int64_t k, per;
  size_t sums, q, inv, total;
};
ThinLayout thin_layout(int64_t batch, int64_t rows, int64_t cols) {
  ThinLayout l;
  l.n = static_cast<int>(rows < cols ? rows : cols);
  l.k = rows < cols ? cols : rows;
  l.N = l.n <= 32 ? 32 : l.n <= 48 ? 48 : 64;
  const int64_t tiles = (l.k + kThinK - 1) / kThinK;
  const int64_t each = (tiles + kThinParts - 1) / kThinParts;
  l.per = each * kThinK;
  l.parts = static_cast<int>((tiles + each - 1) / each);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) & ~size_t(255);
    return at;
  };
  l.sums = take(sizeof(double) * batch * l.parts * l.N * l.N);
  l.q = take(sizeof(float) * batch * l.N * l.N);
  l.inv = take(sizeof(double) * batch);
  l.total = o;
  return l;
}

template <int N>
int launch_thin(const ThinLayout& l, const Source& src, int64_t batch, int64_t rows, int64_t cols, int steps, float a, float b,
                float c, double eps, const ThinOut& o, uint8_t* ws, hipStream_t s) {
  double* sums = reinterpret_cast<double*>(ws + l.sums);
  float* q = reinterpret_cast<float*>(ws + l.q);
  double* inv = reinterpret_cast<double*>(ws + l.inv);
  const Thin t = {l.n, rows <= cols ? 1 : 0, l.k, rows * cols};
  const unsigned nb = static_cast<unsigned>(batch);
  hipLaunchKernelGGL(thin_gram_kernel<N>, dim3(static_cast<unsigned>(l.parts), nb), dim3(256), 0, s, src, t, l.parts, l.per, sums);
  int rc = w4q_launch_status();
  if (rc != W4Q_OK) return rc;
  hipLaunchKernelGGL(thin_steps_kernel<N>, dim3(nb), dim3(step_threads<N>()), 0, s, l.n, l.parts, sums, steps,
                     static_cast<double>(a), static_cast<double>(b), static_cast<double>(c), eps, q, inv);
  if ((rc = w4q_launch_status()) != W4Q_OK) return rc;
  hipLaunchKernelGGL(thin_apply_kernel<N>, dim3(static_cast<unsigned>((l.k + kThinK - 1) / kThinK), nb), dim3(256), 0, s, src, t,
                     q, inv, o);
  return w4q_launch_status();
}

}  // namespace
}  // namespace w4q

using namespace w4q;

bool w4q_thin(int64_t rows, int64_t cols) { return (rows < cols ? rows : cols) <= kThinMax; }

// Where X has (nearly) lost rank, roundings leave A eigenvalues of either sign near zero, about 2^-50 of its
// trace, and every step multiplies those by up to a^2: a negative one that reaches the size of the others
// runs away, as no singular value of X can.  So steps that could bring it to 2^-24 are taken on X itself
// (muon.hip); with the published coefficients that is from 8 steps on.
bool w4q_thin_steps_ok(int steps, double a) {
  double grown = 1.0;
  for (int i = 0; i < steps; ++i) grown *= a * a;
  return grown <= 67108864.0;  // 2^26
}

size_t w4q_thin_workspace(int64_t batch, int64_t rows, int64_t cols) { return thin_layout(batch, rows, cols).total; }

int w4q_launch_ns_thin(const Source& src, int64_t batch, int64_t rows, int64_t cols, int steps, float a, float b, float c,
                       double eps, const ThinOut& o, void* ws, hipStream_t s) {
  const ThinLayout l = thin_layout(batch, rows, cols);
  uint8_t* base = static_cast<uint8_t*>(ws);
  if (l.N == 48) return launch_thin<48>(l, src, batch, rows, cols, steps, a, b, c, eps, o, base, s);
  if (l.N == 32) return launch_thin<32>(l, src, batch, rows, cols, steps, a, b, c, eps, o, base, s);
  return launch_thin<64>(l, src, batch, rows, cols, steps, a, b, c, eps, o, base, s);
}
