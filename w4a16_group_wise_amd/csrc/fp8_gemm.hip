// fp8_gemm.hip -- the product of two matrices held in 8-bit floating point with a scale for each block of 128
// (fp8_quant.hip), with the layer's epilogue:
//
//   z[i][j] = sum_t sa[i][t] sb[j][t] sum_{k in block t} a[i][k] b[j][k] + bias[j],  y = act(z) + residual
//
// Two kinds of product.  The matrix cores' 8-bit products are exact, but they add them in groups of 8 consecutive k
// aligned to the group's largest exponent, and what lies below 2^-13 of that is cut off (measured bit by bit on both
// 8-bit forms; between groups and with the fp32 operand the sums are fp32's).  So:
//   the codes as bf16 values (exact: 3 or 2 bits behind the point) and v_mfma_f32_16x16x32_bf16 on them, whose products
//     and sums are fp32's (kWide); written to the workspace once, or up to 64 rows made in registers, where HBM leaves the
//     time.
//   bf16 y with W4Q_FP8_SHORT, where the caller asks for it: v_mfma_f32_16x16x128_f8f6f4 on the codes as they lie (kWide
//     false), at twice the rate.  The cut is below 7 2^-13 of a group's largest product; on normal activations and weights
//     one bf16 result in 50 to 70 becomes the neighbour of the one that fp32 sums give, 3e-4 of the results' root mean
//     square (their own rounding is 1.7e-3 of it).
//
// A block's products are summed from zero, then scaled and added to the fp32 sums by the vector units, which have the
// matrix cores' time for it: 16 fused multiply-adds for 128 clocks.  b's rows are the rows of the matrix
// cores' result and a's its columns: a lane then has one row of a, so one scale, for all its 16 values, and
// where b has one scale for 128 rows the product of the two is one number.  Only where each row of b has its own
// (weight gradients) is there a second multiplication a value.
//
// Tiles: 128 bytes of k a row and stage (a block of codes, or half a block of bf16 values), so the operands' way to
// LDS and the fragments are nt_gemm.hpp's for 64 16-bit values (which 16-byte pieces of k a lane holds does not
// matter as long as both operands agree).  The stage's scales travel beside them, 4 bytes a lane.
//
// What bounds it, square scales: 8192x12288x4096 743 us (1.11 PFLOP/s; the scaling of each 64 k takes the vector units
// nearly as long as the matrix cores their products), of which about 80 for the bf16 copies at HBM's rate; short sums 405 to 455
// (the clock under this load, and the operands' way through the L2: at 12288x4096x8192 they take 371, with loads from the LDS
// alone 285).  With a scale for each row of b 12288x4096x8192 takes 881, with square blocks 815.  65 to 2048 rows: the copies
// of b and two launches, 200 rows of 4096x4096 38 us, short sums 16.  Few rows: HBM, 1x4096x12288 14 us,
// 13x12288x4096 16.
#include "epilogue.hpp"
#include "nt_gemm.hpp"
#include "w4a16q_block.h"

namespace w4q {
namespace {

typedef int v8i32 __attribute__((ext_vector_type(8)));

constexpr int kBlock = W4Q_FP8_BLOCK;

__device__ __forceinline__ v8i32 join(u32x4 lo, u32x4 hi) {
  return __builtin_bit_cast(v8i32, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
// four codes as four bf16 values (exact; NaN and infinities stay)
template <int kFmt>
__device__ __forceinline__ u32x2 widen(uint32_t codes) {
  const int c = static_cast<int>(codes);
  f32x2 lo, hi;
  if constexpr (kFmt == W4Q_FP8_E4M3) {
    lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false);
    hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
  } else {
    lo = __builtin_amdgcn_cvt_pk_f32_bf8(c, false);
    hi = __builtin_amdgcn_cvt_pk_f32_bf8(c, true);
  }
  return u32x2{__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2)),
               __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2))};
}
__device__ __forceinline__ f32x4 mfma_bf16_16(u32x4 p, u32x4 q, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c, 0, 0, 0);
}
// A stage's product of a 16 x 16 block, summed from zero: of each operand's 16 rows 128 bytes, two pieces of 16 a
// lane.  b gives the rows of the result.
template <bool kWide, int kFa, int kFb>
__device__ __forceinline__ f32x4 stage_product(const u32x4 (&b)[2], const u32x4 (&a)[2]) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (kWide)
    return mfma_bf16_16(b[1], a[1], mfma_bf16_16(b[0], a[0], zero));
  else
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(b[0], b[1]), join(a[0], a[1]), zero, kFb, kFa, 0, 0, 0, 0);
}

// a buffer load of 4 bytes per lane straight to LDS, lane l at + 4 l (see common.hpp for its kind)
__device__ __forceinline__ void dma_word(uint32_t lds, v4i32 rs, int vo) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %[sv], m0\n\t"
      "s_mov_b32 m0, %[m0]\n\t"
      "buffer_load_dword %[vo], %[rs], 0 offen lds\n\t"
      "s_mov_b32 m0, %[sv]"
      : [sv] "=&s"(saved)
      : [m0] "s"(__builtin_amdgcn_readfirstlane(lds)), [rs] "s"(rs), [vo] "v"(vo)
      : "memory", "scc");
}

template <int BM_, int BN_, int WM_, int WN_, int BUFS_>
struct Fp8Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int kWavesM = BM / WM, kWavesN = BN / WN, kWaves = kWavesM * kWavesN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int MB = WM / 16, NB = WN / 16;
  using OpA = NtOperand<BM, 1, false, 64, kWaves>;
  using OpB = NtOperand<BN, 1, false, 64, kWaves>;
  static constexpr int kParts = (OpA::kLoads + OpB::kLoads) / 2;  // of a stage's loads, two each, and the scales'
  static constexpr int kOps = 2 * kParts + 1;
  static constexpr int kScales = (BM + BN > kThreads ? BM + BN : kThreads) * 4;
  static constexpr int kStage = OpA::kBytes + OpB::kBytes + kScales;
  static constexpr int kBufs = BUFS_;
  static constexpr int kLds = kBufs * kStage;
  static constexpr int kTileElems = BM * BN;
  static constexpr int kPitch = WN + 4;
  static_assert(BM + BN <= kThreads, "a wavefront brings the scales of 64 rows");
  static_assert(BN <= 128 || BN % 128 == 0, "b's blocks of scales");
  static_assert(MB % 2 == 0, "fragments of a stage in two sets");
  static_assert(OpA::kLoads % 2 == 0 && OpA::kLoads == OpB::kLoads && kParts <= MB, "a stage's loads go out in pairs, with 16 rows each");
  static_assert(kLds <= 160 * 1024 && kLds / kWaves / 16 * 16 >= 32 * kPitch * 4, "LDS");
};

// The loads of one operand that a wavefront issues: kLoads pieces of 8 rows x 128 bytes, from row 8 kLoads wid of the tile on.
// v: this lane's offsets in the first piece, as it lies in even and in odd pieces (nt_swz alternates)
struct OperandWay {
  const uint8_t* base;  // the wavefront's first row
  int bytes;            // of its rows, 0 past the matrix
};
template <int kLoads>
__device__ __forceinline__ OperandWay operand_way(const uint16_t* p, int r0, int rows, int ld, int wid) {
  const int first = r0 + 8 * kLoads * wid;
  int left = rows - first;
  left = left < 0 ? 0 : left < 8 * kLoads ? left : 8 * kLoads;
  return {reinterpret_cast<const uint8_t*>(p) + (left == 0 ? 0 : static_cast<int64_t>(first) * ld * 2), left * ld * 2};
}
// pieces 2 pair and 2 pair + 1 of stage s
__device__ __forceinline__ void operand_issue(const OperandWay& w, int s, bool live, int pair, int ld, uint32_t dst, const int (&v)[2]) {
  const bool some = live && w.bytes != 0;
  const v4i32 rs = buffer_rsrc(w.base + (some ? 128 * static_cast<int64_t>(s) : 0), some ? w.bytes - 128 * s : 0);
  dma_x2(dst + 2048 * pair, rs, v[0] + 32 * pair * ld, v[1] + 32 * pair * ld);
}

struct Fp8Scales {
  const float *a, *b;
  int blocks;  // of 128 k
};

// This lane's way to the scale of its row of the tile (of a, behind them of b): base, bytes of the resource, offset
struct ScaleWay {
  const float* base;
  int bytes, off;
};
template <class C, bool kRowB>
__device__ __forceinline__ ScaleWay scale_way(const NtArgs& g, const Fp8Scales& sc, int m0, int n0, int wid, int lane) {
  ScaleWay w;
  int rows, row;
  const int slot = 64 * wid;
  if (slot < C::BM) {
    w.base = sc.a + static_cast<int64_t>(m0 + slot) * sc.blocks;
    rows = g.M - (m0 + slot);
    row = lane;
  } else if (kRowB) {
    const int j = n0 + slot - C::BM;
    w.base = sc.b + static_cast<int64_t>(j) * sc.blocks;
    rows = g.N - j;
    row = lane;
  } else {
    const int j = n0 + slot - C::BM;  // (64 rows of b lie in one block of 128)
    w.base = sc.b + static_cast<int64_t>(j >> 7) * sc.blocks;
    rows = j < g.N ? 1 : 0;
    row = 0;
  }
  rows = rows < 0 || slot >= C::BM + C::BN ? 0 : rows < 64 ? rows : 64;
  if (rows == 0) w.base = sc.a;
  w.bytes = rows * sc.blocks * 4;
  w.off = row * sc.blocks * 4;
  return w;
}

// The epilogue: bias, activation, residual, eight consecutive columns of a row at a time, at any address; the last ones of a
// row of other lengths one by one.  (1531x2050x1056 in short sums with gelu and a residual takes 18.6 us, without an epilogue
// 13.4: the vector units' time for gelu on the 204 compute units that have a tile.  With fp32 sums 30.6 and its copies 8.)
struct EpiFp8 {
  struct Pre {
    u32x4 r0, r1;
  };
  W4Epilogue ep;
  void* y;
  int y_dtype;
  int stream;  // y goes past the caches

  __device__ __forceinline__ Pre load(const NtArgs& g, int row, int col) const {
    Pre p = {};
    if (ep.res == nullptr || row >= g.M || col >= g.N) return p;
    const int64_t o = static_cast<int64_t>(row) * g.N + col;
    if (col + 8 <= g.N) {
      load8_any(ep.res, o, y_dtype, p.r0, p.r1);
      return p;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      if (col + e >= g.N) continue;
      if (y_dtype == 0) {
        const uint32_t v = static_cast<const uint32_t*>(ep.res)[o + e];
        e < 4 ? p.r0[e & 3] = v : p.r1[e & 3] = v;
      } else {
        p.r0[e >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(ep.res)[o + e]) << (16 * (e & 1));
      }
    }
    return p;
  }
  __device__ __forceinline__ void store(const NtArgs& g, int row, int col, float (&v)[8], const Pre& p) const {
    if (row >= g.M || col >= g.N) return;
    const int64_t o = static_cast<int64_t>(row) * g.N + col;
    if (ep.bias != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += ep.bias[col + e < g.N ? col + e : col];
    }
    switch (ep.act) {  // one branch for all eight values
      case W4Q_ACT_RELU: act8<W4Q_ACT_RELU>(v); break;
      case W4Q_ACT_GELU: act8<W4Q_ACT_GELU>(v); break;
      case W4Q_ACT_SILU: act8<W4Q_ACT_SILU>(v); break;
      default: break;
    }
    if (ep.res != nullptr) {
      float r[8];
      unpack8(p.r0, p.r1, y_dtype, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
    if (col + 8 > g.N) {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (col + e < g.N) store1(y, o + e, y_dtype, v[e]);
    } else {
      stream != 0 ? store8_stream(y, o, y_dtype, v) : store8_any(y, o, y_dtype, v);
    }
  }
  template <int kAct>
  static __device__ __forceinline__ void act8(float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_fwd(v[e], kAct);
  }
};

// 16 rows of a x WN rows of b to LDS: lane l, value e of block j -> row l % 16, column 16 j + 4 (l / 16) + e
template <class C>
__device__ __forceinline__ void fp8_strip_write(const f32x4 (&acc)[C::NB], int lane, float* buf) {
#pragma unroll
  for (int j = 0; j < C::NB; ++j) *reinterpret_cast<f32x4*>(buf + (lane & 15) * C::kPitch + 16 * j + 4 * (lane >> 4)) = acc[j];
}
// and from there through the epilogue: eight columns of a row a lane, the next rows' residual on its way meanwhile (all of
// a strip's and the next one's at once spilled on tiles of 256 and gained nothing on the others)
template <class C>
__device__ __forceinline__ void fp8_strip_store(const NtArgs& g, const EpiFp8& epi, int row0, int col0, int lane, const float* buf) {
  using S = NtStrip<C>;
  asm volatile("" ::: "memory");  // the wavefront's own LDS operations stay in order
  const int rl = lane / S::kLanes, cl = 8 * (lane % S::kLanes);
  EpiFp8::Pre x = epi.load(g, row0 + rl, col0 + cl);
#pragma unroll 1
  for (int i = 0; i < S::kPasses; ++i) {
    const EpiFp8::Pre next = i + 1 < S::kPasses ? epi.load(g, row0 + rl + S::kRows * (i + 1), col0 + cl) : x;
    const float* p = buf + (rl + S::kRows * i) * C::kPitch + cl;
    const f32x4 lo = *reinterpret_cast<const f32x4*>(p), hi = *reinterpret_cast<const f32x4*>(p + 4);
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    epi.store(g, row0 + rl + S::kRows * i, col0 + cl, v, x);
    x = next;
  }
  asm volatile("" ::: "memory");
}
// partial-tile layout: wavefront, block, lane (1 KB per store instruction)
template <class C>
__device__ __forceinline__ int64_t fp8_part_off(int w, int blk, int lane) {
  return static_cast<int64_t>((w * (C::MB * C::NB) + blk) * 256 + 4 * lane);
}

template <class C, bool kWide, int kFa, int kFb, bool kRowB>
__global__ __launch_bounds__(C::kThreads) void fp8_kernel(const NtArgs g, const Fp8Scales sc, const EpiFp8 epi) {
  using OpA = typename C::OpA;
  using OpB = typename C::OpB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  const int lb = static_cast<int>(blockIdx.x & 7) * g.per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (lb >= g.nblk) return;
  const int whole_end = g.whole * g.S;  // stages of the whole tiles, then of the range
  const int left = g.rest - lb * g.chunk;
  const int end = whole_end + (left < 0 ? 0 : left < g.chunk ? left : g.chunk);

  const int own_lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int wm = wid / C::kWavesN, wn = wid % C::kWavesN;
  const uint32_t lds0 = lds_addr(lds);

  int vo[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) vo[q] = OpA::load_off(q, own_lane, g.lda);
  int it = 0;
  while (it < end) {
    // the lane's number, asked for anew for each tile with all that is made of it: kept over the products it spilled
    int zero = 0;
    asm volatile("" : "+s"(zero));
    const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
    // where a lane's two pieces of its row lie in 16 rows of a tile: pieces l / 16 and 4 + l / 16 (with nt_swz the 16 lanes
    // that LDS serves at a time hit distinct slots; the same in every 16 rows)
    const int ro = (lane & 15) * 128 + 16 * ((lane >> 4) ^ nt_swz(lane & 15));
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
    const ScaleWay way = scale_way<C, kRowB>(g, sc, m0, n0, wid, lane);
    const OperandWay wa = operand_way<OpA::kLoads>(g.a, m0, g.M, g.lda, wid);
    const OperandWay wb = operand_way<OpB::kLoads>(g.b, n0, g.N, g.ldb, wid);

    // part `part` of the loads of stage s into buffer `buf` (past the range: empty): a's pieces, b's, two at a time, and with
    // the last the scales
    auto issue = [&](int s, int buf, int part) {
      const uint32_t dst = lds0 + buf * C::kStage;
      if (part < C::kParts / 2)
        operand_issue(wa, s, s < s1, part, g.lda, dst + wid * (OpA::kLoads * 1024), vo);
      else
        operand_issue(wb, s, s < s1, part - C::kParts / 2, g.ldb, dst + OpA::kBytes + wid * (OpB::kLoads * 1024), vo);
      if (part == C::kParts - 1)
        dma_word(dst + OpA::kBytes + OpB::kBytes + 256 * wid, buffer_rsrc(way.base, s < s1 ? way.bytes : 0),
                 way.off + 4 * (kWide ? s >> 1 : s));
    };

    f32x4 acc[C::MB][C::NB];
#pragma unroll
    for (int i = 0; i < C::MB; ++i)
#pragma unroll
      for (int j = 0; j < C::NB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

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
    auto read_a = [&](int buf, int i, u32x4 (&f)[2]) {
      const uint8_t* p = lds + (buf * C::kStage + wm * (C::WM * 128));
#pragma unroll
      for (int q = 0; q < 2; ++q) f[q] = *reinterpret_cast<const u32x4*>(p + (ro ^ (64 * q)) + 2048 * i);
    };
    auto read_b = [&](int buf, int j, u32x4 (&f)[2]) {
      const uint8_t* p = lds + (buf * C::kStage + OpA::kBytes + wn * (C::WN * 128));
#pragma unroll
      for (int q = 0; q < 2; ++q) f[q] = *reinterpret_cast<const u32x4*>(p + (ro ^ (64 * q)) + 2048 * j);
    };
    struct Factors {
      float a[C::MB];
      f32x4 b[kRowB ? C::NB : 1];  // square blocks: one for all
    };
    auto read_factors = [&](int buf, Factors& f) {
      const float* p = reinterpret_cast<const float*>(lds + buf * C::kStage + OpA::kBytes + OpB::kBytes);
#pragma unroll
      for (int i = 0; i < C::MB; ++i) f.a[i] = p[wm * C::WM + 16 * i + (lane & 15)];
      if constexpr (kRowB) {
#pragma unroll
        for (int j = 0; j < C::NB; ++j) f.b[j] = *reinterpret_cast<const f32x4*>(p + C::BM + wn * C::WN + 16 * j + 4 * (lane >> 4));
      } else {
        f.b[0][0] = p[C::BM + wn * C::WN];
      }
    };
#pragma unroll
    for (int i = 0; i < C::kBufs - 1; ++i)
#pragma unroll
      for (int part = 0; part < C::kParts; ++part) issue(s0 + i, i, part);
    issue(s0 + C::kBufs - 1, C::kBufs - 1, 0);
    sync(std::integral_constant<int, C::kOps * (C::kBufs - 2) + 2>{});  // stage s0 has landed
    // A stage: b's fragments are in registers, a's follow 16 rows at a time, one ahead.  Before the last 16 rows' products
    // every wavefront has read all of the stage and the next one has landed: there is the barrier, and the next stage's
    // first fragments are read under the products.  The loads into the buffer just read go out two at a time, the first
    // there and the others with the next stage's first rows: a wavefront waits until its loads are taken, and all
    // of them at once held up its products.
    // The vector units' part of 16 rows is left until the next 16 rows' products are on their way.
    u32x4 fa[2][2], fb[C::NB][2];
    f32x4 p[2][C::NB];
    Factors f;
    read_factors(0, f);
    read_a(0, 0, fa[0]);
#pragma unroll
    for (int j = 0; j < C::NB; ++j) read_b(0, j, fb[j]);
    auto scale = [&](int i, int j, const Factors& f) {
      const f32x4& v = p[i & 1][j];
      if constexpr (kRowB) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(v[e], f.a[i] * f.b[kRowB ? j : 0][e], acc[i][j][e]);
      } else {
        const float one = f.a[i] * f.b[0][0];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(v[e], one, acc[i][j][e]);
      }
    };
    int buf = 0, free = C::kBufs - 1;  // buffers of the stage, and of the loads going out
    for (int s = s0; s < s1; ++s) {
      Factors next;
#pragma unroll
      for (int i = 0; i < C::MB; ++i) {
        if (i + 1 < C::MB) {
          read_a(buf, i + 1, fa[(i + 1) & 1]);
        } else {
          sync(std::integral_constant<int, C::kOps * (C::kBufs - 2)>{});
          free = buf;
          buf = buf + 1 == C::kBufs ? 0 : buf + 1;
          read_a(buf, 0, fa[(i + 1) & 1]);  // (past the range: a buffer of zeros, never used)
        }
#pragma unroll
        for (int j = 0; j < C::NB; ++j) {
          p[i & 1][j] = stage_product<kWide, kFa, kFb>(fb[j], fa[i & 1]);
          if (i + 1 == C::MB) read_b(buf, j, fb[j]);
          if (i > 0) scale(i - 1, j, f);
        }
        if (i + 1 == C::MB) {
          read_factors(buf, next);
          issue(s + C::kBufs, free, 0);
        } else if (i + 1 < C::kParts) {
          issue(s + C::kBufs - 1, free, i + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < C::NB; ++j) scale(C::MB - 1, j, f);
      f = next;
    }
    // nothing is in flight or still being read when the buffers are used for other things
    sync(std::integral_constant<int, 0>{});

    if (s0 == 0 && s1 == g.S) {
      float* strip = reinterpret_cast<float*>(lds + wid * (C::kLds / C::kWaves / 16 * 16));
      const int row0 = m0 + wm * C::WM, col0 = n0 + wn * C::WN;
      // (one copy of the epilogue's code for all strips: unrolled it was fetched anew for every tile)
#pragma unroll 1
      for (int h = 0; h < C::MB / 2; ++h) {
#pragma unroll
        for (int i = 0; i < C::MB / 2; ++i)
          if (i == h) {
            fp8_strip_write<C>(acc[2 * i], lane, strip);
            fp8_strip_write<C>(acc[2 * i + 1], lane, strip + 16 * C::kPitch);
          }
        fp8_strip_store<C>(g, epi, row0 + 32 * h, col0, lane, strip);
      }
      if (it + (s1 - s0) < end) sync(std::integral_constant<int, 0>{});  // the next tile's loads reuse the LDS
    } else {
      float* slot = g.ws + static_cast<int64_t>(2 * lb + (it == whole_end ? 0 : 1)) * C::kTileElems;
#pragma unroll
      for (int i = 0; i < C::MB; ++i)
#pragma unroll
        for (int j = 0; j < C::NB; ++j) *reinterpret_cast<f32x4*>(slot + fp8_part_off<C>(wid, i * C::NB + j, lane)) = acc[i][j];
    }
    it += s1 - s0;
  }
}

// Tiles whose stages were spread over several workgroups: the partial tiles summed in k order, then the epilogue.
// One wavefront per strip of 32 rows x WN columns.
template <class C>
__global__ __launch_bounds__(64) void fp8_fixup_kernel(const NtArgs g, const EpiFp8 epi) {
  __shared__ __attribute__((aligned(16))) float strip[32 * C::kPitch];
  constexpr int kStrips = C::kWaves * C::MB / 2;
  int t = static_cast<int>(blockIdx.x) / kStrips;
  const int64_t b0 = static_cast<int64_t>(t) * g.S;
  const int first = static_cast<int>(b0 / g.chunk);
  const int last = static_cast<int>((b0 + g.S - 1) / g.chunk);
  if (first == last) return;  // one workgroup held the whole tile
  const int lane = threadIdx.x & 63;
  const int si = static_cast<int>(blockIdx.x) % kStrips;
  const int wid = si / (C::MB / 2), i = si % (C::MB / 2);
  t += g.whole * g.nblk;
  int batch, ti, tj;
  nt_tile(g, t, batch, ti, tj);
  const int row0 = ti * C::BM + (wid / C::kWavesN) * C::WM + 32 * i;
  const int col0 = tj * C::BN + (wid % C::kWavesN) * C::WN;
  f32x4 v[2][C::NB];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < C::NB; ++j) v[h][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int b = first; b <= last; ++b) {
    const int slot = 2 * b + (static_cast<int64_t>(b) * g.chunk >= b0 ? 0 : 1);
    const float* p = g.ws + static_cast<int64_t>(slot) * C::kTileElems;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < C::NB; ++j) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p + fp8_part_off<C>(wid, (2 * i + h) * C::NB + j, lane));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h][j][e] += x[e];
      }
  }
  fp8_strip_write<C>(v[0], lane, strip);
  fp8_strip_write<C>(v[1], lane, strip + 16 * C::kPitch);
  fp8_strip_store<C>(g, epi, row0, col0, lane, strip);
}

// ------------------------------------------------------------------------------- few rows
// Up to 32 or 64 rows of a: a workgroup takes 16 rows of b and deals the blocks of k to its wavefronts, whose sums are added in
// LDS in a fixed order.  A wavefront reads its 16 rows of b 64 consecutive bytes a row and load, straight to the
// matrix cores' registers, kU blocks at a time in flight, and kMT times 16 rows of a, which stay in the caches.
// kWide: the codes become bf16 in registers.  HBM bound: b's bytes.  (Six blocks in flight cost occupancy: 13x12288x4096
// 23 us, 15.7 with four; non-temporal loads 17.4.)
struct FewArgs {
  const uint8_t *a, *b;
  const float *sa, *sb;
  int m, n, k, blocks;
  W4Epilogue ep;
  void* y;
  int y_dtype;
};
template <bool kWide, int kFa, int kFb, bool kRowB, int kMT>
__global__ __launch_bounds__(1024) void fp8_few_kernel(const FewArgs f) {
  constexpr int kU = 4 / kMT;
  extern __shared__ f32x4 red[];  // [wavefront][kMT][lane]
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wid = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int n0 = 16 * static_cast<int>(blockIdx.x);
  const int l = lane & 15, part = lane >> 4;
  const int br = n0 + l < f.n ? n0 + l : f.n - 1;  // (rows past the end: the last one's, not stored)
  const uint8_t* pb = f.b + static_cast<int64_t>(br) * f.k + 16 * part;
  const uint8_t* pa[kMT];
  const float* psa[kMT];
#pragma unroll
  for (int i = 0; i < kMT; ++i) {
    const int ar = 16 * i + l < f.m ? 16 * i + l : f.m - 1;
    pa[i] = f.a + static_cast<int64_t>(ar) * f.k + 16 * part;
    psa[i] = f.sa + static_cast<int64_t>(ar) * f.blocks;
  }
  const float* psb[kRowB ? 4 : 1];
#pragma unroll
  for (int r = 0; r < (kRowB ? 4 : 1); ++r) {
    const int row = n0 + 4 * part + r;
    psb[r] = f.sb + static_cast<int64_t>(kRowB ? (row < f.n ? row : f.n - 1) : n0 >> 7) * f.blocks;
  }
  f32x4 acc[kMT];
#pragma unroll
  for (int i = 0; i < kMT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int t0 = wid; t0 < f.blocks; t0 += kU * waves) {
    u32x4 a[kU][kMT][2], b[kU][2];
    float sa[kU][kMT], sb[kU][kRowB ? 4 : 1];
    // a and the scales first: loads come back in order, and b's take longest
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int t = t0 + u * waves < f.blocks ? t0 + u * waves : t0;  // (past the end: loaded and not used)
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
#pragma unroll
        for (int q = 0; q < 2; ++q) a[u][i][q] = *reinterpret_cast<const u32x4*>(pa[i] + t * kBlock + 64 * q);
        sa[u][i] = psa[i][t];
      }
#pragma unroll
      for (int r = 0; r < (kRowB ? 4 : 1); ++r) sb[u][r] = psb[r][t];
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int t = t0 + u * waves < f.blocks ? t0 + u * waves : t0;
#pragma unroll
      for (int q = 0; q < 2; ++q) b[u][q] = *reinterpret_cast<const u32x4*>(pb + t * kBlock + 64 * q);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (t0 + u * waves >= f.blocks) break;
      u32x4 wb[4];
      if constexpr (kWide) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const u32x2 lo = widen<kFb>(b[u][q >> 1][2 * (q & 1)]), hi = widen<kFb>(b[u][q >> 1][2 * (q & 1) + 1]);
          wb[q] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (kWide) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x2 lo = widen<kFa>(a[u][i][q >> 1][2 * (q & 1)]), hi = widen<kFa>(a[u][i][q >> 1][2 * (q & 1) + 1]);
            p = mfma_bf16_16(wb[q], u32x4{lo[0], lo[1], hi[0], hi[1]}, p);
          }
        } else {
          p = stage_product<false, kFa, kFb>(b[u], a[u][i]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(p[r], sa[u][i] * sb[u][kRowB ? r : 0], acc[i][r]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kMT; ++i) red[(wid * kMT + i) * 64 + lane] = acc[i];
  __syncthreads();
  for (int o = threadIdx.x; o < 256 * kMT; o += blockDim.x) {
    const int row = o >> 4, c = o & 15;
    if (row >= f.m || n0 + c >= f.n) continue;
    float v = 0.0f;
    for (int w = 0; w < waves; ++w) v += red[(w * kMT + (row >> 4)) * 64 + (row & 15) + 16 * (c >> 2)][c & 3];
    store1(f.y, static_cast<int64_t>(row) * f.n + n0 + c, f.y_dtype, apply_epilogue(f.ep, v, row, n0 + c, f.n, f.y_dtype));
  }
}
// rows up to which it is taken, against tiles (us).  bf16 values: 64 rows of 4096x4096 16 to 28, of 12288x4096 41 to 56, of
// 4096x12288 42 to 60: on tiles all of b is first written out.  Codes: 32 rows 10 to 13, 25 to 21, 25 to 24 (17 rows 8 to
// 13, 18 to 21, 18 to 23; 64 rows of 12288x4096 would be 40 to 21).
constexpr int few_rows(bool wide) { return wide ? 64 : 32; }

// Both operands' codes as bf16 values: 16 codes a thread and step.  HBM bound: 3 B a code.
struct WidenArgs {
  const uint8_t* src[2];
  uint16_t* dst[2];
  int64_t n16[2];
  int blocks;  // workgroups on the first operand; those behind them have the second
};
template <int kFmt>
__device__ __forceinline__ void widen_part(const uint8_t* __restrict__ src, uint16_t* __restrict__ dst, int64_t n16, int block, int blocks) {
#pragma unroll 2
  for (int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x; i < n16; i += static_cast<int64_t>(blocks) * 256) {
    const u32x4 c = reinterpret_cast<const u32x4*>(src)[i];
    const u32x2 v0 = widen<kFmt>(c[0]), v1 = widen<kFmt>(c[1]), v2 = widen<kFmt>(c[2]), v3 = widen<kFmt>(c[3]);
    reinterpret_cast<u32x4*>(dst)[2 * i] = u32x4{v0[0], v0[1], v1[0], v1[1]};
    reinterpret_cast<u32x4*>(dst)[2 * i + 1] = u32x4{v2[0], v2[1], v3[0], v3[1]};
  }
}
template <int kFa, int kFb>
__global__ __launch_bounds__(256) void fp8_widen_kernel(const WidenArgs w) {
  const int b = blockIdx.x;
  if (b < w.blocks)
    widen_part<kFa>(w.src[0], w.dst[0], w.n16[0], b, w.blocks);
  else
    widen_part<kFb>(w.src[1], w.dst[1], w.n16[1], b - w.blocks, gridDim.x - w.blocks);
}

// ------------------------------------------------------------------------------ host side
// Tiles: 256 x 256; 128 x 128, two workgroups on a compute unit or one, with more stages in flight (for codes, eight
// wavefronts then, two on each SIMD: 1024x4096x4096 29.4 -> 27.8 us; bf16 values take longer that way, 61 -> 68); 64 x 64.
using Big = Fp8Cfg<256, 256, 128, 64, 2>;
using Mid = Fp8Cfg<128, 128, 64, 64, 2>;
template <bool kWide>
using MidAlone = Fp8Cfg<128, 128, 64, kWide ? 64 : 32, kWide ? 3 : 4>;
using Small = Fp8Cfg<64, 64, 32, 32, 3>;

inline size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// What a tile costs (us): `busy` a stage when its compute unit always has a tile to work on, `alone` a stage with one tile
// on it, `ends` its first loads and its epilogue; per_cu workgroups fit a compute unit.  Measured on 4096 x 4096 codes
// times 64 to 4096 rows, and within a tenth on bf16 values, whose stages hold half the k.
struct Fp8Tile {
  int edge, per_cu;
  double busy, alone, ends;
};
constexpr Fp8Tile kFp8Tiles[3] = {{256, 1, 1.75, 1.55, 5.0}, {128, 2, 0.62, 0.70, 1.5}, {64, 3, 0.22, 0.36, 0.5}};

// The cheapest of: one tile of each size per workgroup, and whole tiles with the remaining ones' stages in ranges,
// whose partial tiles then pass through memory once more.  k16: 16-bit values of a row (half the codes, or the
// bf16 values).  Measured whole: 64 rows of 4096x4096 codes 16 us on tiles of 64, 26 on 128, 52 on 256; 1024 rows 38, 28,
// 57; 2048 rows 62, 46, 58; 4096 rows 122, 86, 66.  As bf16 values, with their copies: 200 rows 38, 61, 115; 1024 rows 76, 65,
// 118; 2048 rows of 12288x4096 370, 277, 250.  Over 65 to 2048 rows of 4096x4096, 2050x1152 and 12288x4096 no other tile or
// split took less than 0.91 of the chosen one's time.
NtPlan fp8_plan(int64_t M, int64_t N, int64_t k16) {
  NtPlan best = {};
  double best_us = 0.0;
  for (int kind = 0; kind < 3; ++kind) {
    const Fp8Tile& t = kFp8Tiles[kind];
    NtPlan p = nt_plan_tile(kind, 1, M, N, k16, false, 64);
    const int64_t tiles = p.nblk, slots = kNtCus * t.per_cu;
    const double per_cu = static_cast<double>((tiles + kNtCus - 1) / kNtCus);
    const double each = per_cu * t.busy > t.alone ? per_cu * t.busy : t.alone;
    const double us = 4.0 + static_cast<double>(p.S) * each + per_cu * t.ends;
    if (kind == 0 || us < best_us) {
      best = p;
      best_us = us;
    }
    p.whole = tiles / slots;
    p.rest = (tiles - p.whole * slots) * p.S;
    if (p.rest == 0) continue;
    p.chunk = (p.rest + slots - 1) / slots;
    if (p.chunk < kNtMinK / 64) p.chunk = kNtMinK / 64;
    const int64_t ranges = (p.rest + p.chunk - 1) / p.chunk;
    if (p.chunk % p.S == 0) continue;
    p.nblk = p.whole != 0 ? slots : ranges;
    p.ws = static_cast<size_t>(ranges) * 2 * t.edge * t.edge * sizeof(float);
    const double whole = static_cast<double>(p.whole) * t.per_cu * (p.S * t.busy + t.ends);
    // (ranges start at different k and share no panels in the L2: 300 rows of 4096x12288 took 58 us in ranges, 52 whole)
    const double load = whole + static_cast<double>(p.rest) / kNtCus * t.busy * 2.0;
    const double alone = whole + static_cast<double>(p.chunk) * t.alone;
    const double bytes = static_cast<double>(ranges + p.rest / p.S) * t.edge * t.edge * 4.0;
    const double sus = 9.0 + (load > alone ? load : alone) + t.ends + bytes / 3e6;
    if (sus < best_us) {
      best = p;
      best_us = sus;
    }
  }
  return best;
}

template <class C, bool kWide, int kFa, int kFb, bool kRowB>
int fp8_launch(NtArgs g, const Fp8Scales& sc, const NtPlan& p, const EpiFp8& epi, void* ws, hipStream_t s) {
  if (!nt_fits(p)) return W4Q_EUNSUPPORTED;
  nt_fill(g, p, 0, ws);
  fp8_kernel<C, kWide, kFa, kFb, kRowB><<<dim3(static_cast<unsigned>(8 * g.per_xcd)), dim3(C::kThreads), 0, s>>>(g, sc, epi);
  int rc = w4q_launch_status();
  if (rc == W4Q_OK && p.ws != 0) {
    fp8_fixup_kernel<C><<<dim3(static_cast<unsigned>(p.rest / p.S * (C::kWaves * C::MB / 2))), dim3(64), 0, s>>>(g, epi);
    rc = w4q_launch_status();
  }
  return rc;
}

template <bool kWide, int kFa, int kFb, bool kRowB>
int fp8_product(const NtArgs& g, const Fp8Scales& sc, const NtPlan& p, const EpiFp8& epi, void* ws, hipStream_t s) {
  if (p.kind == 0) return fp8_launch<Big, kWide, kFa, kFb, kRowB>(g, sc, p, epi, ws, s);
  if (p.kind == 1 && p.nblk <= kNtCus) return fp8_launch<MidAlone<kWide>, kWide, kFa, kFb, kRowB>(g, sc, p, epi, ws, s);
  if (p.kind == 1) return fp8_launch<Mid, kWide, kFa, kFb, kRowB>(g, sc, p, epi, ws, s);
  return fp8_launch<Small, kWide, kFa, kFb, kRowB>(g, sc, p, epi, ws, s);
}

template <bool kWide, int kFa, int kFb, bool kRowB>
int fp8_few(const FewArgs& f, hipStream_t s) {
  // wavefronts that deal the blocks of k: at least four blocks each, or what 16 leave
  int waves = 1;
  while (waves < 16 && 4 * waves < f.blocks) waves *= 2;
  const dim3 grid(static_cast<unsigned>((f.n + 15) / 16)), block(64 * waves);
  const unsigned lds = static_cast<unsigned>(waves * 64 * sizeof(f32x4));
  if (f.m <= 16)
    fp8_few_kernel<kWide, kFa, kFb, kRowB, 1><<<grid, block, lds, s>>>(f);
  else if (f.m <= 32)
    fp8_few_kernel<kWide, kFa, kFb, kRowB, 2><<<grid, block, 2 * lds, s>>>(f);
  else if constexpr (kWide)
    fp8_few_kernel<kWide, kFa, kFb, kRowB, 4><<<grid, block, 4 * lds, s>>>(f);
  return w4q_launch_status();
}

template <int kFa, int kFb>
int fp8_gemm_of(const uint8_t* a, const float* sa, int64_t m, const uint8_t* b, const float* sb, bool row_b, int64_t n, int64_t k,
                const W4Epilogue& ep, void* y, int y_dtype, bool wide, void* ws, hipStream_t s) {
  if (m <= few_rows(wide)) {
    const FewArgs f = {a, b, sa, sb, static_cast<int>(m), static_cast<int>(n), static_cast<int>(k), static_cast<int>(k / kBlock), ep, y, y_dtype};
    if (wide) return row_b ? fp8_few<true, kFa, kFb, true>(f, s) : fp8_few<true, kFa, kFb, false>(f, s);
    return row_b ? fp8_few<false, kFa, kFb, true>(f, s) : fp8_few<false, kFa, kFb, false>(f, s);
  }
  const int64_t k16 = wide ? k : k / 2;
  const NtPlan p = fp8_plan(m, n, k16);
  NtArgs g = {};
  g.a = reinterpret_cast<const uint16_t*>(a);
  g.b = reinterpret_cast<const uint16_t*>(b);
  g.M = static_cast<int>(m);
  g.N = static_cast<int>(n);
  g.K = static_cast<int>(k16);
  g.lda = g.ldb = g.K;
  // past the caches, where rows are whole 16-byte pieces (8192x12288x4096 450 -> 405 us: bursts of 33 MB push the
  // operands out of the L2)
  const bool stream = p.kind == 0 && n % 8 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0;
  const EpiFp8 epi = {ep, y, y_dtype, stream ? 1 : 0};
  const Fp8Scales sc = {sa, sb, static_cast<int>(k / kBlock)};
  if (!wide) return row_b ? fp8_product<false, kFa, kFb, true>(g, sc, p, epi, ws, s) : fp8_product<false, kFa, kFb, false>(g, sc, p, epi, ws, s);
  uint16_t* wa = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + up256(p.ws));
  uint16_t* wb = wa + up256(static_cast<size_t>(2) * m * k) / 2;
  const int64_t na = m * k / 16, nb = n * k / 16;
  const int64_t ba = na / 1024 < 1 ? 1 : na / 1024 < 4096 ? na / 1024 : 4096, bb = nb / 1024 < 1 ? 1 : nb / 1024 < 4096 ? nb / 1024 : 4096;
  const WidenArgs w = {{a, b}, {wa, wb}, {na, nb}, static_cast<int>(ba)};
  fp8_widen_kernel<kFa, kFb><<<dim3(static_cast<unsigned>(ba + bb)), dim3(256), 0, s>>>(w);
  const int rc = w4q_launch_status();
  if (rc != W4Q_OK) return rc;
  g.a = wa;
  g.b = wb;
  return row_b ? fp8_product<true, 0, 0, true>(g, sc, p, epi, ws, s) : fp8_product<true, 0, 0, false>(g, sc, p, epi, ws, s);
}

}  // namespace
}  // namespace w4q

using namespace w4q;

bool w4q_fp8_fits(int64_t m, int64_t n, int64_t k) { return nt_fits(nt_plan_tile(2, 1, m, n, k, false, 64)); }

size_t w4q_fp8_gemm_workspace(int64_t m, int64_t n, int64_t k, int y_dtype) {
  const bool wide = (y_dtype & W4Q_FP8_SHORT) == 0;
  if (m <= few_rows(wide)) return 0;
  if (!wide) return fp8_plan(m, n, k / 2).ws;
  return up256(fp8_plan(m, n, k).ws) + up256(static_cast<size_t>(2) * m * k) + up256(static_cast<size_t>(2) * n * k);
}

int w4q_launch_fp8_gemm(const uint8_t* a, int a_fmt, const float* sa, int64_t m, const uint8_t* b, int b_fmt, const float* sb,
                        int b_square, int64_t n, int64_t k, const W4Epilogue& ep, void* y, int y_dtype, void* ws, hipStream_t s) {
  auto go = [&](auto fa, auto fb) {
    return fp8_gemm_of<decltype(fa)::value, decltype(fb)::value>(a, sa, m, b, sb, b_square == 0, n, k, ep, y, y_dtype & ~W4Q_FP8_SHORT,
                                                              (y_dtype & W4Q_FP8_SHORT) == 0, ws, s);
  };
  using E4 = std::integral_constant<int, W4Q_FP8_E4M3>;
  using E5 = std::integral_constant<int, W4Q_FP8_E5M2>;
  if (a_fmt == W4Q_FP8_E4M3) return b_fmt == W4Q_FP8_E4M3 ? go(E4{}, E4{}) : go(E4{}, E5{});
  return b_fmt == W4Q_FP8_E4M3 ? go(E5{}, E4{}) : go(E5{}, E5{});
}
