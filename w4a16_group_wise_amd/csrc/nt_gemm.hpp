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
// Two stage buffers and one barrier per stage, before the stage's last step of 16 k: there every
// wavefront holds the last fragments of the stage in registers and the next stage has landed, so after
// it the loads of the stage after next go into the buffer just read (they have a whole stage to
// land) and the first fragments of the next stage are read between the products of the last step.
// Rows and k past an operand's end read as zeros (the buffer's bounds); columns past the end of an
// "across" row read on into the next row and only feed outputs that are never stored.
//
// Epilogue: a wavefront passes 32 rows x WN columns at a time through its share of the (then idle)
// LDS and hands the functor 8 consecutive columns of a row per lane, so that everything the epilogue
// reads and writes moves in 16-byte pieces; what it reads is loaded ahead.
//
// Work split: the (tile, stage) iterations of all tiles lie on one line, cut into nblk equal
// ranges, one per workgroup.  A range that covers a whole tile ends in the epilogue; partial tiles
// go to fp32 scratch and are summed by nt_fixup_kernel in k order (a fixed order: results do not
// depend on timing).  With chunk = stages per tile this is one tile per workgroup and no scratch.
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

template <int BM_, int BN_, int WM_, int WN_, int PA_, int PB_, bool F16_, bool AT_, bool BT_, bool LOLO_ = false>
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
  static constexpr int kLds = 2 * kStage;
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
//   Pre load(g, batch, row, col)                     what the epilogue reads there (kAhead: one strip
//                                                    ahead of its use, in twice the registers)
//   void store(g, batch, row, col, v[8], pre)        writes the outputs; leaves in v what a mirrored
//                                                    store shall write
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

template <class C, class Epi>
__device__ __forceinline__ void nt_strip_store(const NtArgs& g, const Epi& epi, int batch, int row0, int col0, bool diag,
                                               const f32x16 (&acc)[C::NB], int lane, float* buf,
                                               const typename Epi::Pre (&pre)[NtStrip<C>::kPasses]) {
  using S = NtStrip<C>;
  // accumulator layout: lane l, register r -> row 8(r/4) + 4(l/32) + r%4, column l%32
#pragma unroll
  for (int j = 0; j < C::NB; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      buf[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * C::kPitch + 32 * j + (lane & 31)] = acc[j][r];
  asm volatile("" ::: "memory");  // the wavefront's own LDS operations stay in order
#pragma unroll
  for (int i = 0; i < S::kPasses; ++i) {
    const int rl = lane / S::kLanes + S::kRows * i, cl = 8 * (lane % S::kLanes);
    float* p = buf + rl * C::kPitch + cl;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    epi.store(g, batch, row0 + rl, col0 + cl, v, pre[i]);
    if constexpr (Epi::kMirror) {
      *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
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

template <int N>
__device__ __forceinline__ void nt_dma(uint32_t lds, v4i32 rs, const int (&vo)[N]) {
  if constexpr (N == 4)
    dma_x4(lds, rs, vo);
  else if constexpr (N == 2)
    dma_x2(lds, rs, vo[0], vo[1]);
  else
    dma_x1(lds, rs, vo[0]);
}

template <class C, class Epi>
__global__ __launch_bounds__(C::kThreads) void nt_kernel(const NtArgs g, const Epi epi) {
  using OpA = typename C::OpA;
  using OpB = typename C::OpB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const int lb = static_cast<int>(blockIdx.x & 7) * g.per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (lb >= g.nblk) return;
  const int it_begin = lb * g.chunk;
  const int it_end = g.total - it_begin < g.chunk ? g.total : it_begin + g.chunk;

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

  int it = it_begin;
  while (it < it_end) {
    const int t = it / g.S;
    const int s0 = it - t * g.S;
    const int s1 = g.S - s0 < it_end - it ? g.S : s0 + (it_end - it);
    int batch, ti, tj;
    nt_tile(g, t, batch, ti, tj);
    const int m0 = ti * C::BM, n0 = tj * C::BN;
    const uint16_t* abase = g.a + batch * g.sa;
    const uint16_t* bbase = g.b + batch * g.sb;

    // an operand's loads of stage s (past the range: empty loads, which write zeros)
    auto issue_op = [&](const uint16_t* base, int s, int r0, int rows, int ld, int krows, uint32_t dst, auto op, int width,
                        int parts, bool across, const auto& vo) {
      using Op = decltype(op);
      const bool live = s < s1;
      int64_t off;
      int bytes;
      if (across) {
        const int left = krows - C::BK * s;
        off = static_cast<int64_t>(C::BK * s) * ld + r0 * parts;
        bytes = ((left < C::BK ? left : C::BK) * ld - r0 * parts) * 2;
      } else {
        const int left = rows - r0;
        off = static_cast<int64_t>(r0) * ld + 64 * s;
        bytes = ((left < width ? left : width) * ld - 64 * s) * 2;
      }
      const v4i32 rs = buffer_rsrc(base + (live ? off : 0), live ? bytes : 0);
      const uint32_t to = dst + wid * (Op::kLoads * 1024);
      if (C::BK == 64 && !across && g.K - 64 * s == 32) {
        // half a stage: the second 32 k of each row (chunks 4..7) lie beyond K and read as zeros
        int half[Op::kLoads];
#pragma unroll
        for (int q = 0; q < Op::kLoads; ++q) {
          const int r = 8 * (wid * Op::kLoads + q) + (lane >> 3);
          half[q] = ((lane ^ nt_swz(r)) & 4) != 0 ? 0x7FFFFFF0 : vo[q];
        }
        nt_dma(to, rs, half);
      } else {
        nt_dma(to, rs, vo);
      }
    };
    auto issue = [&](int s, int buf) {
      const uint32_t dst = lds0 + buf * C::kStage;
      issue_op(abase, s, m0, g.M, g.lda, g.ka, dst, OpA{}, C::BM, C::PA, C::AT, avo);
      issue_op(bbase, s, n0, g.N, g.ldb, g.kb, dst + OpA::kBytes, OpB{}, C::BN, C::PB, C::BT, bvo);
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
    issue(s0, 0);
    issue(s0 + 1, 1);
    sync(std::integral_constant<int, C::kOps>{});  // stage s0 has landed
    load(0, 0, f0);
    int buf = 0;
    for (int s = s0; s < s1; ++s) {
#pragma unroll
      for (int kk = 0; kk + 1 < C::KS; ++kk) {
        load(buf, kk + 1, (kk & 1) != 0 ? f0 : f1);
        mma((kk & 1) != 0 ? f1 : f0);
        pattern();
      }
      sync(std::integral_constant<int, 0>{});  // stage s + 1 has landed; nobody reads buffer `buf` any more
      issue(s + 2, buf);
      buf ^= 1;
      load(buf, 0, f0);  // (past the range: a buffer of zeros, never used)
      mma(f1);
      pattern();
    }
    // nothing is in flight or still being read when the buffers are used for other things
    sync(std::integral_constant<int, 0>{});

    if (s0 == 0 && s1 == g.S) {
      float* strip = reinterpret_cast<float*>(lds + wid * (C::kLds / C::kWaves));
      const int row0 = m0 + wm * C::WM, col0 = n0 + wn * C::WN;
      constexpr int kSets = Epi::kAhead ? 2 : 1;
      typename Epi::Pre pre[kSets][NtStrip<C>::kPasses];
      nt_strip_load<C>(g, epi, batch, row0, col0, lane, pre[0]);
#pragma unroll
      for (int i = 0; i < C::MB; ++i) {
        if (kSets == 2 && i + 1 < C::MB) nt_strip_load<C>(g, epi, batch, row0 + 32 * (i + 1), col0, lane, pre[(i + 1) % kSets]);
        nt_strip_store<C>(g, epi, batch, row0 + 32 * i, col0, ti == tj, acc[i], lane, strip, pre[i % kSets]);
        if (kSets == 1 && i + 1 < C::MB) nt_strip_load<C>(g, epi, batch, row0 + 32 * (i + 1), col0, lane, pre[0]);
      }
      if (it + (s1 - s0) < it_end) sync(std::integral_constant<int, 0>{});  // the next tile's loads reuse the LDS
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
// then the epilogue.  One wavefront per strip of 32 rows x WN columns.
template <class C, class Epi>
__global__ __launch_bounds__(64) void nt_fixup_kernel(const NtArgs g, const Epi epi) {
  __shared__ __attribute__((aligned(16))) float strip[32 * C::kPitch];
  constexpr int kStrips = C::kWaves * C::MB;  // strips of a tile
  const int t = static_cast<int>(blockIdx.x) / kStrips;
  const int64_t b0 = static_cast<int64_t>(t) * g.S;
  const int first = static_cast<int>(b0 / g.chunk);
  const int last = static_cast<int>((b0 + g.S - 1) / g.chunk);
  if (first == last) return;  // one workgroup held the whole tile
  const int lane = threadIdx.x & 63;
  const int si = static_cast<int>(blockIdx.x) % kStrips;
  const int wid = si / C::MB, i = si % C::MB;
  int batch, ti, tj;
  nt_tile(g, t, batch, ti, tj);
  const int row0 = ti * C::BM + (wid / C::kWavesN) * C::WM + 32 * i;
  const int col0 = tj * C::BN + (wid % C::kWavesN) * C::WN;
  typename Epi::Pre pre[NtStrip<C>::kPasses];
  nt_strip_load<C>(g, epi, batch, row0, col0, lane, pre);
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
  nt_strip_store<C>(g, epi, batch, row0, col0, ti == tj, v, lane, strip, pre);
}

// ------------------------------------------------------------------------------ host side
constexpr int kNtCus = 256;
constexpr int kNtMinK = 512;  // k a range covers at least

struct NtPlan {
  int64_t tm, tn, per_batch, S, total, chunk, nblk;
  size_t ws;  // scratch bytes (0: no tile is split)
};

// The split of `batch` products of M x N x K on BM x BN tiles where `slots` workgroups run at once:
// one tile per workgroup when the tiles fill (nearly) whole rounds of the device, else equal
// ranges of stages, one per slot.
inline NtPlan nt_plan(int64_t batch, int64_t M, int64_t N, int64_t K, bool tri, int BM, int BN, int BK, int slots) {
  NtPlan p;
  p.tm = (M + BM - 1) / BM;
  p.tn = (N + BN - 1) / BN;
  p.per_batch = tri ? p.tm * (p.tm + 1) / 2 : p.tm * p.tn;
  p.S = (K + BK - 1) / BK;
  const int64_t tiles = batch * p.per_batch;
  p.total = tiles * p.S;
  p.chunk = p.S;
  const int64_t rounds = (tiles + slots - 1) / slots;
  if (tiles * 100 < rounds * slots * 85 && rounds <= 4) {
    int64_t chunk = (p.total + slots - 1) / slots;
    if (chunk < kNtMinK / BK) chunk = kNtMinK / BK;
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
    constexpr int per_tile = C::kWaves * C::MB;
    const int64_t tiles = p.total / p.S;
    hipLaunchKernelGGL((nt_fixup_kernel<C, Epi>), dim3(static_cast<unsigned>(tiles * per_tile)), dim3(64), 0, s, g, epi);
    rc = w4q_launch_status();
  }
  return rc;
}

}  // namespace w4q
