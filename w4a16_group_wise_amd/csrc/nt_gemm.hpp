// nt_gemm.hpp -- the tiled matrix-core product shared by the linear layer's forward and backward
// pass (linear.hip) and the Newton-Schulz products (muon.hip):
//
//   C[b][i][j] = sum_k A[b][i][k] * B[b][j][k],    both operands with k running along their rows,
//
// where an operand is one 16-bit matrix (bf16, or fp16) or two fp16 matrices hi + lo that hold a
// value in 22 bits: v = hi + lo with hi = RNE(v), lo = RNE(v - hi).  Products of the parts:
//   1 x 1 parts: hi hi;   2 x 1: lo hi + hi hi;   2 x 2: hi lo + lo hi + hi hi
// (lo lo is below 2^-22 of the product and is left out), each exact in fp32 and summed in fp32 by
// the matrix cores.  What becomes of C is the epilogue's (a functor), so that no C is stored
// and read again.
//
// Mapping: BM x BN output tiles, wavefronts of WM x WN (32x32 blocks of
// v_mfma_f32_32x32x16), stages of 32 k.  Every part's tile of a stage is a 64-byte row per matrix
// row, copied to LDS by buffer loads straight to LDS, 16-byte chunk c of row r at position
// c ^ nt_swz(r): the fragment reads (lane l: row l % 32, chunk 2 kk + l / 32) then touch every
// bank slot once per pass.  NBUF stage buffers; the loads run NBUF - 1 stages ahead, and one
// barrier per stage both publishes a stage's tiles and frees the buffer of the stage before it.
// Rows past the operand's end read as zeros (the buffer's bounds), k is a multiple of 32.
//
// Work split: the (tile, stage) iterations of all tiles lie on one line, cut into nblk equal
// ranges, one per workgroup.  A range that covers a whole tile ends in the epilogue; partial tiles
// go to fp32 scratch and are summed by nt_fixup_kernel in k order (a fixed order: results do not
// depend on timing).  With chunk = stages per tile this is one tile per workgroup and no scratch.
#pragma once

#include "common.hpp"

namespace w4q {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// position of 16-byte chunk c in row r (64-byte rows): see gemm.hip for the LDS passes this suits
__device__ __forceinline__ int nt_swz(int r) { return (((r >> 1) ^ (r >> 4)) & 1) | ((r >> 1) & 2); }

struct NtArgs {
  const uint16_t* a[2];
  const uint16_t* b[2];
  int64_t sa, sb;     // elements between the batches of A and B
  int M, N, K;        // K a multiple of 32
  int lda, ldb;       // elements per row, >= K, multiples of 8
  int tm, tn;         // tiles along M and N
  int tri;            // 1: M == N and only tiles with row tile >= column tile
  int per_batch;      // tiles of one batch
  int S;              // stages per tile (K / 32)
  int total;          // iterations (batches * per_batch * S)
  int chunk, nblk, per_xcd;
  float* ws;
};

// tile t of the launch -> batch and tile coordinates.  Whole grids run in bands of 4 row tiles,
// column by column, so that the run of tiles on one XCD is near a square and shares its panels.
__device__ __forceinline__ void nt_tile(const NtArgs& g, int t, int& batch, int& ti, int& tj) {
  batch = t / g.per_batch;
  const int p = t - batch * g.per_batch;
  if (g.tri) {
    int i = static_cast<int>((__builtin_sqrtf(8.0f * static_cast<float>(p) + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > p) --i;
    while ((i + 1) * (i + 2) / 2 <= p) ++i;
    ti = i;
    tj = p - i * (i + 1) / 2;
  } else {
    const int band = p / (4 * g.tn);
    const int rows = g.tm - 4 * band < 4 ? g.tm - 4 * band : 4;
    const int q = p - band * 4 * g.tn;
    tj = q / rows;
    ti = 4 * band + (q - tj * rows);
  }
}

template <int BM_, int BN_, int WM_, int WN_, int PA_, int PB_, bool F16_, int NBUF_>
struct NtCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, PA = PA_, PB = PB_, NBUF = NBUF_;
  static constexpr bool F16 = F16_;
  static constexpr int kWavesM = BM / WM, kWavesN = BN / WN, kWaves = kWavesM * kWavesN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int MB = WM / 32, NB = WN / 32;
  static constexpr int LA = BM / 16 / kWaves, LB = BN / 16 / kWaves;  // 1 KB loads per wave and part
  static constexpr int kOps = PA * LA + PB * LB;                      // loads per wave and stage
  static constexpr int kBytesA = BM * 64, kBytesB = BN * 64;
  static constexpr int kStage = PA * kBytesA + PB * kBytesB;
  static constexpr int kLds = NBUF * kStage;
  static constexpr int kTileElems = BM * BN;
  static_assert(LA >= 1 && LB >= 1 && LA <= 2 && LB <= 2, "1 or 2 loads per wave and part");
  static_assert(kLds <= 160 * 1024, "LDS");
};

template <bool F16>
__device__ __forceinline__ f32x16 nt_mfma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// partial-tile layout: wavefront, block, 16-byte quarter, lane (1 KB per store instruction)
template <class C>
__device__ __forceinline__ int64_t nt_part_off(int w, int blk, int q, int lane) {
  return static_cast<int64_t>(((w * (C::MB * C::NB) + blk) * 4 + q) * 256 + 4 * lane);
}

template <class C, class Epi>
__global__ __launch_bounds__(C::kThreads) void nt_kernel(const NtArgs g, const Epi epi) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  constexpr int D = C::NBUF - 1;  // stages the loads run ahead
  const int lb = static_cast<int>(blockIdx.x & 7) * g.per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (lb >= g.nblk) return;
  const int it_begin = lb * g.chunk;
  const int it_end = g.total - it_begin < g.chunk ? g.total : it_begin + g.chunk;

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / C::kWavesN, wn = wid % C::kWavesN;
  const int fr = lane & 31, fh = lane >> 5;
  const uint32_t lds0 = lds_addr(lds);

  int avo[C::LA], bvo[C::LB];
#pragma unroll
  for (int q = 0; q < C::LA; ++q) {
    const int r = 16 * (wid * C::LA + q) + (lane >> 2);
    avo[q] = r * g.lda * 2 + 16 * ((lane & 3) ^ nt_swz(r));
  }
#pragma unroll
  for (int q = 0; q < C::LB; ++q) {
    const int r = 16 * (wid * C::LB + q) + (lane >> 2);
    bvo[q] = r * g.ldb * 2 + 16 * ((lane & 3) ^ nt_swz(r));
  }
  // byte offsets of this lane's fragments within a part's tile, step 0; step 1 flips bit 5
  int aro[C::MB], bro[C::NB];
#pragma unroll
  for (int i = 0; i < C::MB; ++i) {
    const int r = wm * C::WM + 32 * i + fr;
    aro[i] = r * 64 + 16 * (fh ^ nt_swz(r));
  }
#pragma unroll
  for (int j = 0; j < C::NB; ++j) {
    const int r = wn * C::WN + 32 * j + fr;
    bro[j] = r * 64 + 16 * (fh ^ nt_swz(r));
  }

  int it = it_begin;
  while (it < it_end) {
    const int t = it / g.S;
    const int s0 = it - t * g.S;
    const int s1 = g.S - s0 < it_end - it ? g.S : s0 + (it_end - it);
    int batch, ti, tj;
    nt_tile(g, t, batch, ti, tj);
    const int m0 = ti * C::BM, n0 = tj * C::BN;
    const int arows = g.M - m0 < C::BM ? g.M - m0 : C::BM;
    const int brows = g.N - n0 < C::BN ? g.N - n0 : C::BN;
    const int abytes = arows * g.lda * 2, bbytes = brows * g.ldb * 2;
    const int64_t ao = batch * g.sa + static_cast<int64_t>(m0) * g.lda;
    const int64_t bo = batch * g.sb + static_cast<int64_t>(n0) * g.ldb;

    // loads of stage s into buffer `buf` (past the range: empty loads, which write zeros)
    auto issue = [&](int s, int buf) {
      const bool live = s < s1;
      const int so = live ? s * 32 : 0;
      uint32_t dst = lds0 + buf * C::kStage;
#pragma unroll
      for (int p = 0; p < C::PA; ++p) {
        const v4i32 rs = buffer_rsrc(g.a[p] + ao + so, live ? abytes - so * 2 : 0);
        if constexpr (C::LA == 2)
          dma_x2(dst + wid * 2048, rs, avo[0], avo[1]);
        else
          dma_x1(dst + wid * 1024, rs, avo[0]);
        dst += C::kBytesA;
      }
#pragma unroll
      for (int p = 0; p < C::PB; ++p) {
        const v4i32 rs = buffer_rsrc(g.b[p] + bo + so, live ? bbytes - so * 2 : 0);
        if constexpr (C::LB == 2)
          dma_x2(dst + wid * 2048, rs, bvo[0], bvo[1]);
        else
          dma_x1(dst + wid * 1024, rs, bvo[0]);
        dst += C::kBytesB;
      }
    };

    f32x16 acc[C::MB][C::NB];
#pragma unroll
    for (int i = 0; i < C::MB; ++i)
#pragma unroll
      for (int j = 0; j < C::NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    auto step = [&](const uint8_t* base, int kk) {
      const uint8_t* pa = base;
      const uint8_t* pb = base + C::PA * C::kBytesA;
      u32x4 a[C::PA][C::MB], b[C::PB][C::NB];
#pragma unroll
      for (int p = 0; p < C::PA; ++p)
#pragma unroll
        for (int i = 0; i < C::MB; ++i)
          a[p][i] = *reinterpret_cast<const u32x4*>(pa + p * C::kBytesA + (aro[i] ^ (32 * kk)));
#pragma unroll
      for (int p = 0; p < C::PB; ++p)
#pragma unroll
        for (int j = 0; j < C::NB; ++j)
          b[p][j] = *reinterpret_cast<const u32x4*>(pb + p * C::kBytesB + (bro[j] ^ (32 * kk)));
      if constexpr (C::PB == 2) {
#pragma unroll
        for (int i = 0; i < C::MB; ++i)
#pragma unroll
          for (int j = 0; j < C::NB; ++j) acc[i][j] = nt_mfma<C::F16>(a[0][i], b[1][j], acc[i][j]);
      }
      if constexpr (C::PA == 2) {
#pragma unroll
        for (int i = 0; i < C::MB; ++i)
#pragma unroll
          for (int j = 0; j < C::NB; ++j) acc[i][j] = nt_mfma<C::F16>(a[1][i], b[0][j], acc[i][j]);
      }
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int j = 0; j < C::NB; ++j) acc[i][j] = nt_mfma<C::F16>(a[0][i], b[0][j], acc[i][j]);
    };

#pragma unroll
    for (int d = 0; d < D; ++d) issue(s0 + d, d);
    int buf = 0;
    for (int s = s0; s < s1; ++s) {
      // this wave's loads of stage s have landed and its reads of the stage before are done;
      // after the barrier that holds for every wave
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0((D - 1) * C::kOps));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      const int nb = buf + D >= C::NBUF ? buf + D - C::NBUF : buf + D;
      issue(s + D, nb);
      const uint8_t* base = lds + buf * C::kStage;
      step(base, 0);
      step(base, 1);
      buf = buf + 1 == C::NBUF ? 0 : buf + 1;
    }
    // nothing of this tile is in flight or still being read when the next tile's loads are issued
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);

    if (s0 == 0 && s1 == g.S) {
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int j = 0; j < C::NB; ++j) {
          epi(g, batch, m0 + wm * C::WM + 32 * i, n0 + wn * C::WN + 32 * j, ti == tj, acc[i][j], lane);
          asm volatile("" ::: "memory");
        }
    } else {
      float* slot = g.ws + static_cast<int64_t>(2 * lb + (it == it_begin ? 0 : 1)) * C::kTileElems;
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int j = 0; j < C::NB; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& v = acc[i][j];
            *reinterpret_cast<f32x4*>(slot + nt_part_off<C>(wid, i * C::NB + j, q, lane)) =
                f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          }
    }
    it += s1 - s0;
  }
}

// Tiles whose stages were spread over several workgroups: the partial tiles summed in k order,
// then the epilogue.  One wavefront per 32x32 block (four to a workgroup).
template <class C, class Epi>
__global__ __launch_bounds__(256) void nt_fixup_kernel(const NtArgs g, const Epi epi) {
  constexpr int kBlocks = C::kWaves * C::MB * C::NB;  // 32x32 blocks of a tile, a multiple of 4
  static_assert(kBlocks % 4 == 0, "four blocks per workgroup");
  const int t = static_cast<int>(blockIdx.x) / (kBlocks / 4);
  const int lane = threadIdx.x & 63;
  const int blk = 4 * (static_cast<int>(blockIdx.x) % (kBlocks / 4)) +
                  __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int64_t b0 = static_cast<int64_t>(t) * g.S;
  const int first = static_cast<int>(b0 / g.chunk);
  const int last = static_cast<int>((b0 + g.S - 1) / g.chunk);
  if (first == last) return;  // one workgroup held the whole tile
  const int wid = blk / (C::MB * C::NB), ij = blk % (C::MB * C::NB);
  f32x16 v;
#pragma unroll
  for (int r = 0; r < 16; ++r) v[r] = 0.0f;
  for (int b = first; b <= last; ++b) {
    const int slot = 2 * b + (static_cast<int64_t>(b) * g.chunk >= b0 ? 0 : 1);
    const float* p = g.ws + static_cast<int64_t>(slot) * C::kTileElems;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p + nt_part_off<C>(wid, ij, q, lane));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] += x[e];
    }
  }
  int batch, ti, tj;
  nt_tile(g, t, batch, ti, tj);
  epi(g, batch, ti * C::BM + (wid / C::kWavesN) * C::WM + 32 * (ij / C::NB),
      tj * C::BN + (wid % C::kWavesN) * C::WN + 32 * (ij % C::NB), ti == tj, v, lane);
}

// ------------------------------------------------------------------------------ host side
constexpr int kNtCus = 256;
constexpr int kNtMinChunk = 16;  // stages a range covers at least

struct NtPlan {
  int64_t tm, tn, per_batch, S, total, chunk, nblk;
  size_t ws;  // scratch bytes (0: no tile is split)
};

// The split of `batch` products of M x N x K on BM x BN tiles where `slots` workgroups run at once:
// one tile per workgroup when the tiles fill (nearly) whole rounds of the device, else equal
// ranges of stages, one per slot.
inline NtPlan nt_plan(int64_t batch, int64_t M, int64_t N, int64_t K, bool tri, int BM, int BN, int slots) {
  NtPlan p;
  p.tm = (M + BM - 1) / BM;
  p.tn = (N + BN - 1) / BN;
  p.per_batch = tri ? p.tm * (p.tm + 1) / 2 : p.tm * p.tn;
  p.S = K / 32;
  const int64_t tiles = batch * p.per_batch;
  p.total = tiles * p.S;
  p.chunk = p.S;
  const int64_t rounds = (tiles + slots - 1) / slots;
  if (tiles * 100 < rounds * slots * 85 && rounds <= 4) {
    int64_t chunk = (p.total + slots - 1) / slots;
    if (chunk < kNtMinChunk) chunk = kNtMinChunk;
    if (chunk < p.S || (rounds > 1 && chunk < p.S * rounds)) p.chunk = chunk;
  }
  p.nblk = (p.total + p.chunk - 1) / p.chunk;
  p.ws = p.chunk % p.S != 0 ? static_cast<size_t>(p.nblk) * 2 * BM * BN * sizeof(float) : 0;
  return p;
}

// one product: fills in the plan, launches the product and, where tiles were split, the fixup
template <class C, class Epi>
int nt_launch(NtArgs g, const NtPlan& p, int tri, const Epi& epi, void* ws, hipStream_t s) {
  if (p.total > 0x3FFFFFFF) return W4Q_EUNSUPPORTED;
  g.tm = static_cast<int>(p.tm);
  g.tn = static_cast<int>(p.tn);
  g.tri = tri;
  g.per_batch = static_cast<int>(p.per_batch);
  g.S = static_cast<int>(p.S);
  g.total = static_cast<int>(p.total);
  g.chunk = static_cast<int>(p.chunk);
  g.nblk = static_cast<int>(p.nblk);
  g.per_xcd = (g.nblk + 7) / 8;
  g.ws = static_cast<float*>(ws);
  hipLaunchKernelGGL((nt_kernel<C, Epi>), dim3(static_cast<unsigned>(8 * g.per_xcd)), dim3(C::kThreads), 0, s, g, epi);
  int rc = w4q_launch_status();
  if (rc == W4Q_OK && p.ws != 0) {
    constexpr int per_tile = C::kWaves * C::MB * C::NB / 4;
    const int64_t tiles = p.total / p.S;
    hipLaunchKernelGGL((nt_fixup_kernel<C, Epi>), dim3(static_cast<unsigned>(tiles * per_tile)), dim3(256), 0, s, g, epi);
    rc = w4q_launch_status();
  }
  return rc;
}

}  // namespace w4q
