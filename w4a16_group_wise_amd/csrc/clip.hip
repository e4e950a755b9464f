// clip.hip -- grad_norm, grad_clip: the norm over all gradients of a model and the gradients scaled by it.
//
//   norm = sqrt(sum g^2),  c = fl32(1 where norm + eps <= max_norm, else max_norm / (norm + eps)),  out = c g
//
// Squares and sums in fp64: no gradient is too large or small for its square, and the fp64 units have room to spare
// under a stream of loads.  One pass reads every tensor and leaves a partial sum a workgroup; the pass that scales sums
// the partials first, every workgroup for itself and in the same order (16 KB at most, from the L2: cheaper than
// a launch between the two).  The tables of tensors travel as launch arguments, up to 128 a launch, the sums of later
// launches added to those of the ones before: nothing is copied to the device beforehand and a captured graph holds its
// own.
//
// The workgroups take pieces of 4096 elements in turn, so that all of them work on neighbouring memory: with a range of its
// own for each the scaling of 386 M fp32 gradients took 660 us, not 620.  (One workgroup for each piece and the sums
// joined by a launch between: 600, but 10 to 70 more where nothing is to be scaled.)
//
// HBM bound: two reads and a write of every gradient.  386 M elements, fp32 to fp32: 882 us (under the profiler 294 for the
// norm and 602), 5.2 TB/s.
#include "epilogue.hpp"
#include "w4a16q_block.h"

namespace w4q {
namespace {

constexpr int kTable = 128;         // tensors of a launch
constexpr int kMostBlocks = 2048;   // workgroups of a launch, and partial sums
constexpr int kPiece = 4096;        // elements a workgroup takes at a time, 8 of each half a thread

struct ClipTable {
  const void* g[kTable];
  void* out[kTable];
  int64_t n[kTable];    // elements; bit 62: g is bf16, bit 61: out is
  int first[kTable];    // first piece of this launch that lies in it
  int count, pieces;
  int sums;             // partial sums that the launches before have left
  int in_place;         // every tensor's out is g
};
constexpr int64_t kGBf16 = int64_t(1) << 62, kOutBf16 = int64_t(1) << 61, kCount = (int64_t(1) << 61) - 1;
static_assert(sizeof(ClipTable) <= 4096 - 256, "launch arguments");

// f(g, g's type, out, out's type, first element, elements) for each of this workgroup's pieces
template <class F>
__device__ __forceinline__ void clip_pieces(const ClipTable& t, const F& f) {
  int p = blockIdx.x, i = 0, top = t.count - 1;
  while (i < top) {
    const int mid = (i + top + 1) / 2;
    t.first[mid] <= p ? i = mid : top = mid - 1;
  }
  for (; p < t.pieces; p += gridDim.x) {
    while (i + 1 < t.count && t.first[i + 1] <= p) ++i;
    const int64_t n = t.n[i], begin = static_cast<int64_t>(p - t.first[i]) * kPiece, left = (n & kCount) - begin;
    f(t.g[i], (n & kGBf16) != 0 ? 1 : 0, t.out[i], (n & kOutBf16) != 0 ? 1 : 0, begin, static_cast<int>(left < kPiece ? left : kPiece));
  }
}
// eight(first of 8 elements), or one(element), for this thread's of n elements from `begin` on
template <class Eight, class One>
__device__ __forceinline__ void clip_walk(int64_t begin, int n, const Eight& eight, const One& one) {
  if (n == kPiece) {
#pragma unroll
    for (int h = 0; h < 2; ++h) eight(begin + h * (kPiece / 2) + 8 * threadIdx.x);
    return;
  }
  for (int at = 8 * threadIdx.x; at < n; at += kPiece / 2) {
    if (at + 8 <= n)
      eight(begin + at);
    else
      for (int e = at; e < n; ++e) one(begin + e);
  }
}

__device__ __forceinline__ double block_sum_f64(double v) {
  __shared__ double red[4];
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ __launch_bounds__(256) void clip_square_kernel(const ClipTable t, double* __restrict__ parts) {
  double s0 = 0.0, s1 = 0.0;
  clip_pieces(t, [&](const void* g, int g_dtype, void*, int, int64_t begin, int n) {
    clip_walk(
        begin, n,
        [&](int64_t i) {
          u32x4 a, b;
          load8_any(g, i, g_dtype, a, b);
          float v[8];
          unpack8(a, b, g_dtype, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const double x = v[2 * e], y = v[2 * e + 1];
            s0 = __builtin_fma(x, x, s0);
            s1 = __builtin_fma(y, y, s1);
          }
        },
        [&](int64_t i) {
          const double x = g_dtype == 0 ? static_cast<const float*>(g)[i] : bf16_val(static_cast<const uint16_t*>(g)[i]);
          s0 = __builtin_fma(x, x, s0);
        });
  });
  const double s = block_sum_f64(s0 + s1);
  const int b = blockIdx.x;
  if (threadIdx.x == 0) parts[b] = b < t.sums ? parts[b] + s : s;
}

__device__ __forceinline__ double sum_parts(const double* parts, int n) {
  double s = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += 256) s += parts[i];
  return block_sum_f64(s);
}

__global__ __launch_bounds__(256) void clip_norm_kernel(const double* __restrict__ parts, int n, float* norm) {
  const double s = sum_parts(parts, n);
  if (threadIdx.x == 0) *norm = static_cast<float>(__builtin_sqrt(s));
}

__global__ __launch_bounds__(256) void clip_scale_kernel(const ClipTable t, const double* __restrict__ parts, double max_norm,
                                                         double eps, float* __restrict__ norm_out) {
  const double norm = __builtin_sqrt(sum_parts(parts, t.sums));
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
  const double top = norm + eps;
  const float c = top <= max_norm ? 1.0f : static_cast<float>(max_norm / top);
  if (c == 1.0f && t.in_place != 0) return;
  clip_pieces(t, [&](const void* g, int g_dtype, void* out, int out_dtype, int64_t begin, int n) {
    if (c == 1.0f && out == g) return;
    clip_walk(
        begin, n,
        [&](int64_t i) {
          u32x4 a, b;
          load8_any(g, i, g_dtype, a, b);
          float v[8];
          unpack8(a, b, g_dtype, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= c;
          store8_any(out, i, out_dtype, v);
        },
        [&](int64_t i) {
          const float x = g_dtype == 0 ? static_cast<const float*>(g)[i] : bf16_val(static_cast<const uint16_t*>(g)[i]);
          store1(out, i, out_dtype, x * c);
        });
  });
}

}  // namespace
}  // namespace w4q

using namespace w4q;

size_t w4q_clip_workspace(int64_t) { return kMostBlocks * sizeof(double); }

int w4q_launch_clip(const w4q_grad* grads, int64_t n_grads, bool scale, double max_norm, double eps, float* norm, void* ws,
                    hipStream_t s) {
  double* parts = static_cast<double*>(ws);
  int sums = 0;
  for (int pass = 0; pass < (scale ? 2 : 1); ++pass) {
    for (int64_t i = 0; i < n_grads; i += kTable) {
      ClipTable t;
      t.count = static_cast<int>(n_grads - i < kTable ? n_grads - i : kTable);
      t.sums = sums;
      t.pieces = 0;
      t.in_place = 1;
      for (int j = 0; j < t.count; ++j) {
        const w4q_grad& g = grads[i + j];
        t.g[j] = g.g;
        t.out[j] = g.out;
        if (g.out != g.g) t.in_place = 0;  // (in place the types are equal)
        t.n[j] = g.numel | (g.g_dtype != 0 ? kGBf16 : 0) | (g.out_dtype != 0 ? kOutBf16 : 0);
        t.first[j] = t.pieces;
        t.pieces += static_cast<int>((g.numel + kPiece - 1) / kPiece);
      }
      const int blocks = t.pieces < kMostBlocks ? t.pieces : kMostBlocks;
      if (pass == 0) {
        clip_square_kernel<<<dim3(blocks), dim3(256), 0, s>>>(t, parts);
        sums = sums > blocks ? sums : blocks;
      } else {
        clip_scale_kernel<<<dim3(blocks), dim3(256), 0, s>>>(t, parts, max_norm, eps, i == 0 ? norm : nullptr);
      }
      const int rc = w4q_launch_status();
      if (rc != W4Q_OK) return rc;
    }
  }
  if (!scale) {
    clip_norm_kernel<<<dim3(1), dim3(256), 0, s>>>(parts, sums, norm);
    return w4q_launch_status();
  }
  return W4Q_OK;
}
