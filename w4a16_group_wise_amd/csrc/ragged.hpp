// ragged.hpp -- which elements an epilogue reads where the rows of its matrices are not multiples of
// 16 bytes: a lane has one column and groups of 8 rows of a tile, and the last tiles reach past the matrix,
// with whole groups too.  Everything such a group reads goes through ragged8, so that the bounds
// hold in one place.  Plain C++ as well, for a check of the bounds on the host.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define W4Q_HD __host__ __device__ __forceinline__
#else
#define W4Q_HD inline
#endif

namespace w4q {

// get(e, row, col) for the 8 rows from `row` on of column `col`: rows past the matrix are its last and columns
// past it its first, read and not used (clamped rather than branched over, so that the loads overlap)
template <class Get>
W4Q_HD void ragged8(int row, int rows, int col, int cols, Get get) {
#ifdef __HIPCC__
#pragma unroll
#endif
  for (int e = 0; e < 8; ++e) get(e, row + e < rows ? row + e : rows - 1, col < cols ? col : 0);
}

// element of [batch][rows][cols]
W4Q_HD int64_t element_at(int64_t batch, int64_t row, int64_t rows, int64_t col, int64_t cols) {
  return (batch * rows + row) * cols + col;
}

// hi part of an element of a split matrix (nt_gemm.hpp): rows of ld columns, the parts of 32 columns side by side,
// `stride` 16-bit values between batches; the lo part is 32 further
W4Q_HD int64_t split_at(int64_t batch, int64_t stride, int64_t row, int ld, int col) {
  return batch * stride + row * (2 * ld) + (col >> 5) * 64 + (col & 31);
}

}  // namespace w4q
