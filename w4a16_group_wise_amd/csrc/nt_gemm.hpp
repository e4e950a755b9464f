// nt_gemm.hpp -- the tiled matrix-core product shared by the linear layer's forward and backward
// pass (linear.hip) and the Newton-Schulz products (muon.hip):
//
//   C[b][i][j] = sum_k A[b](i, k) * B[b](j, k)
//
// An operand is one 16-bit matrix (bf16, or fp16) or a split one: two fp16 parts hi + lo that hold a
// value in 22 bits, v = hi + lo with hi = RNE(v), lo = RNE(v - hi), stored with the parts of each 32
// columns side by side ([row][column / 32][hi, lo][column % 32]).  Products of the parts:
//   1 x 1: hi hi;   2 x 1: hi hi + lo hi;   2 x 2: hi lo + hi hi + lo hi
// (lo lo is below 2^-22 of the product; only the small tile adds it, where products are cheap and few
// terms average the difference out), each exact in fp32 and summed in fp32 by the matrix cores.
// What becomes of C is the epilogue's (a functor), so that no C is stored and read again.
//
// An operand lies in memory with k along its rows ("along": A[i][k], K a multiple of 32) or across
// them ("across": A[k][i], any K).  Either is copied to LDS as it lies, by buffer loads straight to
// LDS: along, 128 bytes of a row a stage (64 k, or 32 k of both parts: whole cache lines; with 64-byte
// pieces the L2 served twice the requests), 16-byte chunk c of row r at c ^ nt_swz(r), read in 16-byte
// fragments; across, rows of the tile's width with chunk c of row k at c ^ nt_tswz(k), read by the
// transposing LDS read.  Both patterns touch every bank slot once per pass.  So no operand is ever
// transposed in memory: of the gradients and of X X^T, B X and X^T X each product reads its operands
// as their producers wrote them.
//
// Mapping: BM x BN output tiles, wavefronts of WM x WN (32x32 blocks of v_mfma_f32_32x32x16).
// Two stage buffers, or three, and one barrier per stage, before the stage's last step of 16 k: there
// every wavefront holds the last fragments of the stage in registers and the next stage has landed, so
// after it the loads of the stage after next (of three: the one behind it) go into the buffer just read
// and the first fragments of the next stage are read between the products of the last step.  With two
// they have one stage to land, which on 64x64 tiles is too short: a third buffer took 0.155 to 0.12 units a
// stage there (1024x1024, five steps of 2 x 2 parts: 284 -> 200 us with the plan that follows from it); a
// fourth gained nothing, nor did a third on 128x128 tiles with two workgroups on a compute unit.
// Rows and k past an operand's end read as zeros (the buffer's bounds); columns past the end of an
// "across" row read on into the next row and only feed outputs that are never stored.
//
// Epilogue: a wavefront passes 32 rows x WN columns at a time through its share of the (then idle)
// LDS and hands the functor 8 consecutive columns of a row per lane, so that everything the epilogue
// reads and writes moves in 16-byte pieces; what it reads is loaded ahead.
//
// Bound by the matrix cores at the clocks they hold under such a load (1.4 to 1.7 GHz) and by the operands'
// way from L2 to LDS.  Measured with the epilogues: 1 x 1 parts 8192x12288x4096 1.25 PFLOP/s, 2 x 1 across
// 1.24, along and across 1.25, 2 x 2 12288x4096x4096 1.24 to 1.3; the main loop alone reaches 1.4 (the library's plain product of 8192
// cubed: 1.52).
//
// Work split: one tile per workgroup; or as many whole tiles as each of the workgroups that fit the
// device gets, and the (tile, stage) iterations of the remaining tiles on one line, cut into equal ranges,
// one per workgroup.  Partial tiles go to fp32 scratch and are summed by nt_fixup_kernel in k order (a
// fixed order: results do not depend on timing).  Ranges start at different k, so their workgroups do not
// share panels in the L2: with all 528 tiles of a symmetric 4096 cubed product in ranges it took 265 us, with 512
// of them whole and 16 in ranges about 190.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace w4q {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// position mask of a chunk of row r in an "along" tile (128-byte rows, 8 chunks).  A 16-byte LDS read
// is served in passes of 16 lanes: of each half of the wavefront, the four lane quads whose index has
// even parity, then the other four.  Rows of such a pass differ in (row / 2) % 8 or in parity, so
// with this mask they hit the 16 distinct slots of 256 bytes.
__device__ __forceinline__ int nt_swz(int r) { return (r >> 1) & 7; }
// position mask of a chunk of k row t, for rows of `bytes` bytes: a transposing read of 16 lanes
// covers 4 consecutive k x 2 chunks and one of 32 lanes 4 k x 4 chunks, which these masks spread over
// distinct slots modulo 128 and 256 bytes
template <int bytes>
__device__ __forceinline__ int nt_tswz(int t) {
  return bytes == 128 ? 2 * (t & 3) : (0xCA60 >> (4 * (t & 3))) & 15;
}

struct NtArgs {
  const uint16_t *a, *b;
  int64_t sa, sb;     // 16-bit values between the batches of A and B
  int M, N, K;        // K a multiple of 32 unless both operands lie across
  int ka, kb;         // k rows that A, B really have, where they lie across (K up to the next 32 is zero)
  int lda, ldb;       // 16-bit values per row (both parts of a split operand), multiples of 8
  int tm, tn;         // tiles along M and N
  int tri;            // 1: M == N and only tiles with row tile >= column tile
  int per_batch;      // tiles of one batch
  int S;              // stages per tile
  int whole;          // tiles a workgroup takes whole: tiles lb, lb + nblk, ...
  int rest;           // iterations of the tiles behind those, cut into ranges of `chunk`
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

template <int N>
__device__ __forceinline__ void nt_dma(uint32_t lds, v4i32 rs, const int (&vo)[N]) {
  if constexpr (N == 4)
    dma_x4(lds, rs, vo);
  else if constexpr (N == 2)
    dma_x2(lds, rs, vo[0], vo[1]);
  else
    dma_x1(lds, rs, vo[0]);
}

// An operand's tile in LDS: W rows (along) or columns (across), P parts, BK k a stage
template <int W, int P, bool kAcross, int BK, int kWaves>
struct NtOperand {
  static constexpr int kRow = kAcross ? 2 * W * P : 128;          // bytes of a row
  static constexpr int kBytes = kAcross ? BK * kRow : W * kRow;
  static constexpr int kLoads = kBytes / 1024 / kWaves;           // 1 KB loads per wave
  static_assert(kAcross || BK * P == 64, "128 bytes of a row a stage");
  static_assert(kLoads == 1 || kLoads == 2 || kLoads == 4, "loads per wave");

  // byte offset in memory of what lane `lane` brings with load u
  static __device__ __forceinline__ int load_off(int u, int lane, int ld) {
    constexpr int kChunks = kRow / 16, kRows = 64 / kChunks;  // chunks of a row, rows of a load
    const int r = u * kRows + lane / kChunks;
    const int c = (lane % kChunks) ^ (kAcross ? nt_tswz<kRow>(r) : nt_swz(r));
    return r * ld * 2 + 16 * c;
  }
  // This wavefront's loads of stage s to `dst`: loads u0 .. u0 + kLoads - 1 of the tile whose first row
  // (along) or column (across) is r0, vo their load_off.  rows: the operand's rows (along) or k rows
  // (across).  !live: empty loads, which write zeros.
  static __device__ __forceinline__ void issue(const uint16_t* base, int s, bool live, int r0, int rows, int ld, int K,
                                               uint32_t dst, int u0, int lane, const int (&vo)[kLoads]) {
    int64_t off;
    int bytes;
    if constexpr (kAcross) {
      const int left = rows - BK * s;
      const int c0 = r0 * P;
      off = static_cast<int64_t>(BK * s) * ld + c0;
      bytes = ((left < BK ? left : BK) * ld - c0) * 2;
    } else {
      const int left = rows - r0;
      off = static_cast<int64_t>(r0) * ld + 64 * s;
      bytes = ((left < W ? left : W) * ld - 64 * s) * 2;
    }
    const v4i32 rs = buffer_rsrc(base + (live ? off : 0), live ? bytes : 0);
    if (BK == 64 && !kAcross && K - 64 * s == 32) {
      // half a stage: the second 32 k of each row (chunks 4..7) lie beyond K and read as zeros
      int half[kLoads];
#pragma unroll
      for (int q = 0; q < kLoads; ++q)
        half[q] = ((lane ^ nt_swz(8 * (u0 + q) + (lane >> 3))) & 4) != 0 ? 0x7FFFFFF0 : vo[q];
      nt_dma(dst, rs, half);
    } else {
      nt_dma(dst, rs, vo);
    }
  }
  // byte offset in the tile of this lane's fragment of rows r0 .. r0 + 31, first step, first part
  static __device__ __forceinline__ int read_off(int r0, int lane) {
    if constexpr (kAcross) {
      // 16-lane group rg, lane rj in it: k 8 (rg / 2) + rj / 4 (+ 4 in the second read), values
      // 16 (rg % 2) + 4 (rj % 4); it receives value 16 (rg % 2) + rj of four consecutive k
      const int rg = lane >> 4, rj = lane & 15;
      const int t = 8 * (rg >> 1) + (rj >> 2);
      const int c = r0 / 8 * P + 2 * (rg & 1) + ((rj >> 1) & 1);
      return t * kRow + 16 * (c ^ nt_tswz<kRow>(t)) + 8 * (rj & 1);
    } else {
      const int r = r0 + (lane & 31);
      return r * 128 + 16 * ((lane >> 5) ^ nt_swz(r));
    }
  }
  static __device__ __forceinline__ u32x4 read(const uint8_t* tile, int off, int kk, int part) {
    if constexpr (kAcross) {
      const uint8_t* p = tile + (off ^ (64 * part)) + kk * 16 * kRow;
      const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)(p));
      const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)(p + 4 * kRow));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const u32x4*>(tile + (off ^ (32 * kk + 64 * part)));
    }
  }
};

template <int BM_, int BN_, int WM_, int WN_, int PA_, int PB_, bool F16_, bool AT_, bool BT_, bool LOLO_ = false, int BUFS_ = 2>
struct NtCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, PA = PA_, PB = PB_;
  static constexpr bool F16 = F16_, AT = AT_, BT = BT_, LOLO = LOLO_;  // AT, BT: operand lies across
  static constexpr int BK = PA == 1 && PB == 1 ? 64 : 32, KS = BK / 16;  // k and steps of a stage
  static constexpr int kWavesM = BM / WM, kWavesN = BN / WN, kWaves = kWavesM * kWavesN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int MB = WM / 32, NB = WN / 32;
  using OpA = NtOperand<BM, PA, AT, BK, kWaves>;
  using OpB = NtOperand<BN, PB, BT, BK, kWaves>;
  static constexpr int kOps = OpA::kLoads + OpB::kLoads;              // loads per wave and stage
  static constexpr int kStage = OpA::kBytes + OpB::kBytes;
  static constexpr int kBufs = BUFS_;                                 // stage buffers
  static constexpr int kLds = kBufs * kStage;
  static constexpr int kTileElems = BM * BN;
  static constexpr int kPitch = WN + 4;                               // floats per row of an epilogue strip
  static constexpr int kReads = PA * MB * (AT ? 2 : 1) + PB * NB * (BT ? 2 : 1);  // LDS reads per step
  static constexpr int kMma = MB * NB * (PA + PB - 1 + (LOLO ? 1 : 0));           // products per step
  static_assert(kLds <= 160 * 1024 && kLds / kWaves >= 32 * kPitch * 4, "LDS");
  static_assert(!LOLO || (PA == 2 && PB == 2), "parts");
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

// ---------------------------------------------------------------------------- epilogue strips
// A strip is 32 rows x WN columns of a wavefront's tile.  Lane l takes 8 columns from 8 (l % (WN / 8)) of
// rows l / (WN / 8) + kRows i.  The functor gives, for 8 columns of one row:
//   int word(batch)                                  a word of the tile's matrix, read before its product
//   Epi with(word)                                   the functor for that tile
//   Pre load(g, batch, row, col)                     what the epilogue reads there.  kLoads: 2 the next
//                                                    strip's before a strip is stored, 1 after, 0 a
//                                                    pass ahead, in a loop (for long epilogues, whose
//                                                    unrolled code would spill accumulators)
//   void store(g, batch, row, col, v[8], pre)        writes the outputs; leaves in v what a mirrored
//                                                    store shall write
//   bool whole()                                     false: rows are not multiples of 16 bytes, and
//   void load_rows(g, batch, row, col, x[8])         the epilogue runs on 8 rows of one column
//   void store_rows(g, batch, row, col, v[8], x[8])
//   kMirror, void store_t(g, batch, col, row, v[8])  symmetric results: 8 rows of one column
template <class C>
struct NtStrip {
  static constexpr int kLanes = C::WN / 8;     // lanes per row
  static constexpr int kRows = 64 / kLanes;    // rows per pass
  static constexpr int kPasses = 32 / kRows;
};

template <class C, class Epi>
__device__ __forceinline__ void nt_strip_load(const NtArgs& g, const Epi& epi, int batch, int row0, int col0, int lane,
                                              typename Epi::Pre (&pre)[NtStrip<C>::kPasses]) {
  using S = NtStrip<C>;
#pragma unroll
  for (int i = 0; i < S::kPasses; ++i)
    pre[i] = epi.load(g, batch, row0 + lane / S::kLanes + S::kRows * i, col0 + 8 * (lane % S::kLanes));
}

// one strip of accumulators to LDS: lane l, register r -> row 8(r/4) + 4(l/32) + r%4, column l%32
template <class C>
__device__ __forceinline__ void nt_strip_write(const f32x16 (&acc)[C::NB], int lane, float* buf) {
#pragma unroll
  for (int j = 0; j < C::NB; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      buf[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * C::kPitch + 32 * j + (lane & 31)] = acc[j][r];
}

template <class C, class Epi>
__device__ __forceinline__ void nt_strip_store(const NtArgs& g, const Epi& epi, int batch, int row0, int col0, bool diag,
                                               int lane, float* buf, const typename Epi::Pre (&pre)[NtStrip<C>::kPasses]) {
  using S = NtStrip<C>;
  asm volatile("" ::: "memory");  // the wavefront's own LDS operations stay in order
  if (!epi.whole()) {
    // rows that are not multiples of 16 bytes: a lane has one column and 8 rows at a time, so that
    // a wavefront's accesses of a row are still consecutive
    constexpr int kGroups = 4 * C::WN / 64;  // groups of 8 rows a lane has
    const int c = lane % C::WN, r0 = lane / C::WN * (8 * kGroups);
    // all that is read of the strip in flight at once (16 us of a 1531 x 2050 residual otherwise)
    float x[kGroups][8];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) epi.load_rows(g, batch, row0 + r0 + 8 * i, col0 + c, x[i]);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = buf[(r0 + 8 * i + e) * C::kPitch + c];
      if (col0 + c < g.N) epi.store_rows(g, batch, row0 + r0 + 8 * i, col0 + c, v, x[i]);
    }
    asm volatile("" ::: "memory");
    return;
  }
  auto pass = [&](int i, const typename Epi::Pre& x) {
    const int rl = lane / S::kLanes + S::kRows * i, cl = 8 * (lane % S::kLanes);
    float* p = buf + rl * C::kPitch + cl;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    epi.store(g, batch, row0 + rl, col0 + cl, v, x);
    if constexpr (Epi::kMirror) {
      *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
  };
  if constexpr (Epi::kLoads == 0) {
    auto at = [&](int i) { return epi.load(g, batch, row0 + lane / S::kLanes + S::kRows * i, col0 + 8 * (lane % S::kLanes)); };
    typename Epi::Pre x = at(0);
#pragma unroll 1
    for (int i = 0; i < S::kPasses; ++i) {
      const typename Epi::Pre next = i + 1 < S::kPasses ? at(i + 1) : x;
      pass(i, x);
      x = next;
    }
  } else {
#pragma unroll
    for (int i = 0; i < S::kPasses; ++i) pass(i, pre[i]);
  }
  if constexpr (Epi::kMirror) {
    if (!diag) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < C::WN / 16; ++i) {
        const int cl = 16 * i + (lane >> 2), rl = 8 * (lane & 3);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = buf[(rl + e) * C::kPitch + cl];
        epi.store_t(g, batch, col0 + cl, row0 + rl, v);
      }
    }
  }
  asm volatile("" ::: "memory");
}

template <class C, class Epi>
__global__ __launch_bounds__(C::kThreads) void nt_kernel(const NtArgs g, const Epi args) {
  using OpA = typename C::OpA;
  using OpB = typename C::OpB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const int lb = static_cast<int>(blockIdx.x & 7) * g.per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (lb >= g.nblk) return;
  const int whole_end = g.whole * g.S;  // iterations of the whole tiles, then of the range
  const int left = g.rest - lb * g.chunk;
  const int end = whole_end + (left < 0 ? 0 : left < g.chunk ? left : g.chunk);

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid / C::kWavesN, wn = wid % C::kWavesN;
  const uint32_t lds0 = lds_addr(lds);

  int avo[OpA::kLoads], bvo[OpB::kLoads], aro[C::MB], bro[C::NB];
#pragma unroll
  for (int q = 0; q < OpA::kLoads; ++q) avo[q] = OpA::load_off(wid * OpA::kLoads + q, lane, g.lda);
#pragma unroll
  for (int q = 0; q < OpB::kLoads; ++q) bvo[q] = OpB::load_off(wid * OpB::kLoads + q, lane, g.ldb);
#pragma unroll
  for (int i = 0; i < C::MB; ++i) aro[i] = OpA::read_off(wm * C::WM + 32 * i, lane);
#pragma unroll
  for (int j = 0; j < C::NB; ++j) bro[j] = OpB::read_off(wn * C::WN + 32 * j, lane);

  int it = 0;
  while (it < end) {
    int t, s0, s1;
    if (it < whole_end) {
      t = it / g.S * g.nblk + lb;
      s0 = 0;
      s1 = g.S;
    } else {
      const int at = lb * g.chunk + (it - whole_end);
      t = at / g.S;
      s0 = at - t * g.S;
      s1 = g.S - s0 < end - it ? g.S : s0 + (end - it);
      t += g.whole * g.nblk;
    }
    int batch, ti, tj;
    nt_tile(g, t, batch, ti, tj);
    const int m0 = ti * C::BM, n0 = tj * C::BN;
    const uint16_t* abase = g.a + batch * g.sa;
    const uint16_t* bbase = g.b + batch * g.sb;
    const int word = args.word(batch);

    // loads of stage s into buffer `buf` (past the range: empty)
    auto issue = [&](int s, int buf) {
      const uint32_t dst = lds0 + buf * C::kStage;
      OpA::issue(abase, s, s < s1, m0, C::AT ? g.ka : g.M, g.lda, g.K, dst + wid * (OpA::kLoads * 1024), wid * OpA::kLoads,
                 lane, avo);
      OpB::issue(bbase, s, s < s1, n0, C::BT ? g.kb : g.N, g.ldb, g.K, dst + OpA::kBytes + wid * (OpB::kLoads * 1024),
                 wid * OpB::kLoads, lane, bvo);
    };

    f32x16 acc[C::MB][C::NB];
#pragma unroll
    for (int i = 0; i < C::MB; ++i)
#pragma unroll
      for (int j = 0; j < C::NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    struct Frags {
      u32x4 a[C::PA][C::MB], b[C::PB][C::NB];
    };
    auto load = [&](int buf, int kk, Frags& f) {
      const uint8_t* pa = lds + buf * C::kStage;
      const uint8_t* pb = pa + OpA::kBytes;
#pragma unroll
      for (int p = C::PB - 1; p >= 0; --p)
#pragma unroll
        for (int j = 0; j < C::NB; ++j) f.b[p][j] = OpB::read(pb, bro[j], kk, p);
#pragma unroll
      for (int p = 0; p < C::PA; ++p)
#pragma unroll
        for (int i = 0; i < C::MB; ++i) f.a[p][i] = OpA::read(pa, aro[i], kk, p);
    };
    auto mma_parts = [&](const u32x4 (&a)[C::MB], const u32x4 (&b)[C::NB]) {
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int j = 0; j < C::NB; ++j) acc[i][j] = nt_mfma<C::F16>(a[i], b[j], acc[i][j]);
    };
    auto mma = [&](const Frags& f) {
      if constexpr (C::PB == 2) mma_parts(f.a[0], f.b[1]);
      mma_parts(f.a[0], f.b[0]);
      if constexpr (C::PA == 2) mma_parts(f.a[1], f.b[0]);
      if constexpr (C::LOLO) mma_parts(f.a[1], f.b[1]);
    };
    // the next step's LDS reads spread between this step's products
    auto pattern = [&]() {
      constexpr int per = C::kMma / C::kReads;
      if constexpr (per >= 1) {
#pragma unroll
        for (int i = 0; i < C::kReads; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, per, 0);  // MFMA
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    // LDS read
        }
        __builtin_amdgcn_sched_group_barrier(0x008, C::kMma - per * C::kReads, 0);
      }
    };
    // this wave's loads but the youngest n have landed and its LDS reads are done; after the barrier
    // that holds for every wave
    auto sync = [&](auto n) {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(decltype(n)::value));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    Frags f0, f1;
#pragma unroll
    for (int i = 0; i < C::kBufs; ++i) issue(s0 + i, i);
    sync(std::integral_constant<int, C::kOps * (C::kBufs - 1)>{});  // stage s0 has landed
    load(0, 0, f0);
    int buf = 0;
    for (int s = s0; s < s1; ++s) {
#pragma unroll
      for (int kk = 0; kk + 1 < C::KS; ++kk) {
        load(buf, kk + 1, (kk & 1) != 0 ? f0 : f1);
        mma((kk & 1) != 0 ? f1 : f0);
        pattern();
      }
      // stage s + 1 has landed; nobody reads buffer `buf` any more
      sync(std::integral_constant<int, C::kOps * (C::kBufs - 2)>{});
      issue(s + C::kBufs, buf);
      buf = buf + 1 == C::kBufs ? 0 : buf + 1;
      load(buf, 0, f0);  // (past the range: a buffer of zeros, never used)
      mma(f1);
      pattern();
    }
    // nothing is in flight or still being read when the buffers are used for other things
    sync(std::integral_constant<int, 0>{});

    if (s0 == 0 && s1 == g.S) {
      const Epi& epi = args.with(word);
      float* strip = reinterpret_cast<float*>(lds + wid * (C::kLds / C::kWaves));
      const int row0 = m0 + wm * C::WM, col0 = n0 + wn * C::WN;
      constexpr int kSets = Epi::kLoads == 2 ? 2 : 1;
      typename Epi::Pre pre[kSets][NtStrip<C>::kPasses];
      if (Epi::kLoads != 0) nt_strip_load<C>(g, epi, batch, row0, col0, lane, pre[0]);
#pragma unroll
      for (int i = 0; i < C::MB; ++i) {
        if (kSets == 2 && i + 1 < C::MB) nt_strip_load<C>(g, epi, batch, row0 + 32 * (i + 1), col0, lane, pre[(i + 1) % kSets]);
        nt_strip_write<C>(acc[i], lane, strip);
        nt_strip_store<C>(g, epi, batch, row0 + 32 * i, col0, ti == tj, lane, strip, pre[i % kSets]);
        if (Epi::kLoads == 1 && i + 1 < C::MB) nt_strip_load<C>(g, epi, batch, row0 + 32 * (i + 1), col0, lane, pre[0]);
      }
      if (it + (s1 - s0) < end) sync(std::integral_constant<int, 0>{});  // the next tile's loads reuse the LDS
    } else {
      float* slot = g.ws + static_cast<int64_t>(2 * lb + (it == whole_end ? 0 : 1)) * C::kTileElems;
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
// then the epilogue.  One wavefront per strip of 32 rows x WN columns.
template <class C, class Epi>
__global__ __launch_bounds__(64) void nt_fixup_kernel(const NtArgs g, const Epi args) {
  __shared__ __attribute__((aligned(16))) float strip[32 * C::kPitch];
  constexpr int kStrips = C::kWaves * C::MB;  // strips of a tile
  int t = static_cast<int>(blockIdx.x) / kStrips;
  const int64_t b0 = static_cast<int64_t>(t) * g.S;
  const int first = static_cast<int>(b0 / g.chunk);
  const int last = static_cast<int>((b0 + g.S - 1) / g.chunk);
  if (first == last) return;  // one workgroup held the whole tile
  const int lane = threadIdx.x & 63;
  const int si = static_cast<int>(blockIdx.x) % kStrips;
  const int wid = si / C::MB, i = si % C::MB;
  t += g.whole * g.nblk;
  int batch, ti, tj;
  nt_tile(g, t, batch, ti, tj);
  const int row0 = ti * C::BM + (wid / C::kWavesN) * C::WM + 32 * i;
  const int col0 = tj * C::BN + (wid % C::kWavesN) * C::WN;
  const Epi& epi = args.with(args.word(batch));
  typename Epi::Pre pre[NtStrip<C>::kPasses];
  if (Epi::kLoads != 0) nt_strip_load<C>(g, epi, batch, row0, col0, lane, pre);
  f32x16 v[C::NB];
#pragma unroll
  for (int j = 0; j < C::NB; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) v[j][r] = 0.0f;
  for (int b = first; b <= last; ++b) {
    const int slot = 2 * b + (static_cast<int64_t>(b) * g.chunk >= b0 ? 0 : 1);
    const float* p = g.ws + static_cast<int64_t>(slot) * C::kTileElems;
#pragma unroll
    for (int j = 0; j < C::NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p + nt_part_off<C>(wid, i * C::NB + j, q, lane));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][4 * q + e] += x[e];
      }
  }
  nt_strip_write<C>(v, lane, strip);
  nt_strip_store<C>(g, epi, batch, row0, col0, ti == tj, lane, strip, pre);
}

// ------------------------------------------------------------------------------- small products
// For products too small to fill the device with tiles of 64: 32x32 tiles, the stages of a tile dealt
// to the 8 wavefronts of a workgroup, each with LDS buffers of its own (no barrier until the end, all
// loads of a short sum in flight at once), the wavefronts' sums added in LDS in a fixed order.  256 x 512
// Newton-Schulz products: 8 us each on 64x64 tiles, 5.5 us here.
template <int PA_, int PB_, bool F16_, bool AT_, bool BT_, bool LOLO_ = false>
struct NtTinyCfg {
  static constexpr int BM = 32, BN = 32, WM = 32, WN = 32, PA = PA_, PB = PB_;
  static constexpr bool F16 = F16_, AT = AT_, BT = BT_, LOLO = LOLO_;
  static constexpr int BK = PA == 1 && PB == 1 ? 64 : 32, KS = BK / 16;
  static constexpr int kWaves = 8, kThreads = 64 * kWaves, MB = 1, NB = 1;
  using OpA = NtOperand<32, PA, AT, BK, 1>;
  using OpB = NtOperand<32, PB, BT, BK, 1>;
  static constexpr int kOps = OpA::kLoads + OpB::kLoads;
  static constexpr int kStage = OpA::kBytes + OpB::kBytes;
  static constexpr int kLds = 2 * kStage * kWaves;
  static constexpr int kPitch = WN + 4;
  static_assert(2 * kStage >= 32 * kPitch * 4 && kLds <= 160 * 1024, "LDS");
};

template <class C, class Epi>
__global__ __launch_bounds__(C::kThreads) void nt_tiny_kernel(const NtArgs g, const Epi args) {
  using OpA = typename C::OpA;
  using OpB = typename C::OpB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const int t = static_cast<int>(blockIdx.x & 7) * g.per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (t >= g.nblk) return;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  uint8_t* mine = lds + wid * (2 * C::kStage);
  const uint32_t lds0 = lds_addr(lds) + wid * (2 * C::kStage);
  int batch, ti, tj;
  nt_tile(g, t, batch, ti, tj);
  const int m0 = ti * 32, n0 = tj * 32;
  const uint16_t* abase = g.a + batch * g.sa;
  const uint16_t* bbase = g.b + batch * g.sb;
  int avo[OpA::kLoads], bvo[OpB::kLoads];
#pragma unroll
  for (int q = 0; q < OpA::kLoads; ++q) avo[q] = OpA::load_off(q, lane, g.lda);
#pragma unroll
  for (int q = 0; q < OpB::kLoads; ++q) bvo[q] = OpB::load_off(q, lane, g.ldb);
  const int aro = OpA::read_off(0, lane), bro = OpB::read_off(0, lane);
  auto issue = [&](int s, int buf) {
    const uint32_t dst = lds0 + buf * C::kStage;
    OpA::issue(abase, s, s < g.S, m0, C::AT ? g.ka : g.M, g.lda, g.K, dst, 0, lane, avo);
    OpB::issue(bbase, s, s < g.S, n0, C::BT ? g.kb : g.N, g.ldb, g.K, dst + OpA::kBytes, 0, lane, bvo);
  };
  // the first wavefront does the epilogue: what that reads is on its way before the operands
  const int word = args.word(batch);
  typename Epi::Pre pre[NtStrip<C>::kPasses];
  if (wid == 0 && Epi::kLoads != 0) nt_strip_load<C>(g, args, batch, m0, n0, lane, pre);
  asm volatile("" ::: "memory");
  f32x16 acc[1];
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[0][r] = 0.0f;
  issue(wid, 0);
  issue(wid + C::kWaves, 1);
  int buf = 0;
  for (int s = wid; s < g.S; s += C::kWaves) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(C::kOps));  // this stage's loads (the wavefront's own buffer)
    asm volatile("" ::: "memory");
    const uint8_t* pa = mine + buf * C::kStage;
    const uint8_t* pb = pa + OpA::kBytes;
    u32x4 a[C::KS][C::PA], b[C::KS][C::PB];
#pragma unroll
    for (int kk = 0; kk < C::KS; ++kk) {
#pragma unroll
      for (int p = 0; p < C::PA; ++p) a[kk][p] = OpA::read(pa, aro, kk, p);
#pragma unroll
      for (int p = 0; p < C::PB; ++p) b[kk][p] = OpB::read(pb, bro, kk, p);
    }
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_lgkm0());  // the buffer has been read
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(s + 2 * C::kWaves, buf);
#pragma unroll
    for (int kk = 0; kk < C::KS; ++kk) {
      if constexpr (C::LOLO) acc[0] = nt_mfma<C::F16>(a[kk][C::PA - 1], b[kk][C::PB - 1], acc[0]);
      if constexpr (C::PB == 2) acc[0] = nt_mfma<C::F16>(a[kk][0], b[kk][1], acc[0]);
      if constexpr (C::PA == 2) acc[0] = nt_mfma<C::F16>(a[kk][1], b[kk][0], acc[0]);
      acc[0] = nt_mfma<C::F16>(a[kk][0], b[kk][0], acc[0]);
    }
    buf ^= 1;
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0(0));  // nothing is on its way to the buffers
  asm volatile("" ::: "memory");
  nt_strip_write<C>(acc, lane, reinterpret_cast<float*>(mine));
  const Epi& epi = args.with(word);
  __syncthreads();
  float* strip = reinterpret_cast<float*>(lds);
  constexpr int kStride = 2 * C::kStage / 4;  // floats between the wavefronts' strips
  for (int e = threadIdx.x; e < 32 * 32; e += C::kThreads) {
    const int at = (e >> 5) * C::kPitch + (e & 31);
    float v = strip[at];
#pragma unroll
    for (int w = 1; w < C::kWaves; ++w) v += strip[w * kStride + at];
    strip[at] = v;
  }
  __syncthreads();
  if (wid == 0) nt_strip_store<C>(g, epi, batch, m0, n0, ti == tj, lane, strip, pre);
}

// ------------------------------------------------------------------------------ host side
constexpr int kNtCus = 256;
constexpr int kNtMinK = 512;  // k a range covers at least

struct NtPlan {
  int kind;  // tile: 0 256x256, 1 128x128, 2 64x64, 3 32x32 (small products)
  int64_t tm, tn, per_batch, S, total, whole, rest, chunk, nblk;
  size_t ws;  // scratch bytes (0: no tile is split)
};

// What a tile costs, in units of a 256x256 tile's stage on a fully busy device (2.4 us for 2 x 2
// parts, 2.0 for 64 k of 1 x 1, 1.8 for 2 x 1): `busy` per tile and stage when a compute unit
// always has a tile to work on, `alone` with one tile on it; measured on 4096, 2048 and 1024 cubed.
struct NtTile {
  int edge, per_cu;
  double busy, alone;
};
constexpr NtTile kNtTiles[4] = {{256, 1, 1.0, 0.70}, {128, 2, 0.265, 0.31}, {64, 3, 0.098, 0.120}, {32, 1, 0.0, 0.0}};

inline NtPlan nt_plan_tile(int kind, int64_t batch, int64_t M, int64_t N, int64_t K, bool tri, int BK) {
  NtPlan p;
  const int64_t edge = kNtTiles[kind].edge;
  p.kind = kind;
  p.tm = (M + edge - 1) / edge;
  p.tn = (N + edge - 1) / edge;
  p.per_batch = tri ? p.tm * (p.tm + 1) / 2 : p.tm * p.tn;
  p.S = (K + BK - 1) / BK;
  p.total = batch * p.per_batch * p.S;
  p.whole = 1;
  p.rest = p.chunk = 0;
  p.nblk = batch * p.per_batch;
  p.ws = 0;
  return p;
}

// The cheapest of: one tile of each size per workgroup, and (split) whole tiles with the remaining ones in
// ranges, whose partial tiles then pass through memory once more (5 us and 3 TB/s measured).  Sizes with the same
// estimate take the larger tile.  E.g. 2 x 2 parts at 2048 cubed: 112 us on 64 tiles of 256, 52 us on
// 256 of 128, 59 us on 1024 of 64; 1024 cubed: 56, 22, 12 us; 512 x 512 x 8192: 398, 143, 106 us
// whole and 42, 29, 30 us in ranges (all with two stage buffers).
inline NtPlan nt_plan(int64_t batch, int64_t M, int64_t N, int64_t K, bool tri, int BK, double unit_us, bool split,
                      bool tiny) {
  NtPlan best = {};
  double best_us = 0.0;
  for (int kind = 0; kind < 3; ++kind) {
    const NtTile& t = kNtTiles[kind];
    NtPlan p = nt_plan_tile(kind, batch, M, N, K, tri, BK);
    const int64_t tiles = p.nblk;
    const double per_cu = static_cast<double>((tiles + kNtCus - 1) / kNtCus);
    const double each = per_cu * t.busy > t.alone ? per_cu * t.busy : t.alone;
    const double us = 4.0 + unit_us * static_cast<double>(p.S) * each;
    if (kind == 0 || us < best_us) {
      best = p;
      best_us = us;
    }
    if (!split) continue;
    // as many whole tiles as every resident workgroup gets, the rest in ranges
    const int64_t slots = kNtCus * t.per_cu;
    p.whole = tiles / slots;
    p.rest = (tiles - p.whole * slots) * p.S;
    if (p.rest == 0) continue;
    p.chunk = (p.rest + slots - 1) / slots;
    if (p.chunk < kNtMinK / BK) p.chunk = kNtMinK / BK;
    const int64_t ranges = (p.rest + p.chunk - 1) / p.chunk;
    if (p.chunk % p.S == 0) continue;
    p.nblk = p.whole != 0 ? slots : ranges;
    p.ws = static_cast<size_t>(ranges) * 2 * t.edge * t.edge * sizeof(float);
    const double load = (static_cast<double>(p.whole) * t.per_cu * p.S + static_cast<double>(p.rest) / kNtCus) * t.busy;
    const double alone = static_cast<double>(p.chunk) * t.alone + static_cast<double>(p.whole) * t.per_cu * p.S * t.busy;
    const double bytes = static_cast<double>(ranges + p.rest / p.S) * t.edge * t.edge * 4.0;
    const double sus = 9.0 + unit_us * (load > alone ? load : alone) + bytes / 3e6;
    if (sus < best_us) {
      best = p;
      best_us = sus;
    }
  }
  if (tiny) {
    // a workgroup's round: a fixed 2 us and, for each of its 8 wavefronts, half a microsecond a stage
    const NtPlan p = nt_plan_tile(3, batch, M, N, K, tri, BK);
    const double us = 2.0 + static_cast<double>((p.nblk + kNtCus - 1) / kNtCus) * (2.0 + 0.5 * static_cast<double>((p.S + 7) / 8));
    if (us < best_us) best = p;
  }
  return best;
}

// Iterations in an int with room for sums of two, and workgroups whose threads (256, or 512 on tiles of
// 256 and 32, of which a plan never takes more than half as many as tiles of 64) count below 2^32.
inline bool nt_fits(const NtPlan& p) { return p.total <= 0x3FFFFFFF && p.nblk <= 0xFFFFF0; }

// one product: fills in the plan, launches the product and, where tiles were split, the fixup
inline void nt_fill(NtArgs& g, const NtPlan& p, int tri, void* ws) {
  g.tm = static_cast<int>(p.tm);
  g.tn = static_cast<int>(p.tn);
  g.tri = tri;
  g.per_batch = static_cast<int>(p.per_batch);
  g.S = static_cast<int>(p.S);
  g.whole = static_cast<int>(p.whole);
  g.rest = static_cast<int>(p.rest);
  g.chunk = static_cast<int>(p.chunk);
  g.nblk = static_cast<int>(p.nblk);
  g.per_xcd = (g.nblk + 7) / 8;
  g.ws = static_cast<float*>(ws);
}

template <class C, class Epi>
int nt_launch_tiny(NtArgs g, const NtPlan& p, int tri, const Epi& epi, hipStream_t s) {
  if (!nt_fits(p)) return W4Q_EUNSUPPORTED;
  nt_fill(g, p, tri, nullptr);
  hipLaunchKernelGGL((nt_tiny_kernel<C, Epi>), dim3(static_cast<unsigned>(8 * g.per_xcd)), dim3(C::kThreads), 0, s, g, epi);
  return w4q_launch_status();
}

template <class C, class Epi>
int nt_launch(NtArgs g, const NtPlan& p, int tri, const Epi& epi, void* ws, hipStream_t s) {
  if (!nt_fits(p)) return W4Q_EUNSUPPORTED;
  nt_fill(g, p, tri, ws);
  hipLaunchKernelGGL((nt_kernel<C, Epi>), dim3(static_cast<unsigned>(8 * g.per_xcd)), dim3(C::kThreads), 0, s, g, epi);
  int rc = w4q_launch_status();
  if (rc == W4Q_OK && p.ws != 0) {
    constexpr int per_tile = C::kWaves * C::MB;
    hipLaunchKernelGGL((nt_fixup_kernel<C, Epi>), dim3(static_cast<unsigned>(p.rest / p.S * per_tile)), dim3(64), 0, s, g, epi);
    rc = w4q_launch_status();
  }
  return rc;
}

}  // namespace w4q
