// Walks every 8-row group that a ragged epilogue may be handed (all tiles of a matrix, whole ones past its
// last row and column too) and counts the elements it would read outside its buffers.  Prints that
// count for the reads as they are, and for a read whose base is built from the unclamped row (the
// mistake this guards against), which must be caught.
#include <cstdio>
#include <initializer_list>

#include "ragged.hpp"

int main() {
  const int edges[] = {32, 64, 128, 256};
  const int sizes[] = {1, 2, 7, 8, 9, 31, 33, 63, 65, 66, 127, 129, 130, 250, 255, 257, 300, 321, 520, 777};
  long long bad = 0, caught = 0, wrong = 0;
  for (int edge : edges)
    for (int rows : sizes)
      for (int cols : sizes)
        for (int batches : {1, 3}) {
          const int64_t total = int64_t(batches) * rows * cols;
          const int ld = (cols + 31) / 32 * 32;
          const int64_t stride = 2 * int64_t(rows) * ld, split = batches * stride;
          const int tm = (rows + edge - 1) / edge, tn = (cols + edge - 1) / edge;
          for (int batch = 0; batch < batches; ++batch)
            for (int row = 0; row < tm * edge; row += 8)
              for (int col = 0; col < tn * edge; ++col) {
                w4q::ragged8(row, rows, col, cols, [&](int e, int r, int c) {
                  const int64_t at = w4q::element_at(batch, r, rows, c, cols);
                  if (at < 0 || at >= total) ++bad;
                  // what is inside the matrix is the element itself
                  if (row + e < rows && col < cols && at != (int64_t(batch) * rows + row + e) * cols + col) ++wrong;
                });
                w4q::ragged8(row, rows, col, ld, [&](int e, int r, int c) {
                  const int64_t at = w4q::split_at(batch, stride, r, ld, c);
                  if (at < 0 || at + 32 >= split) ++bad;
                  if (row + e < rows && col < ld &&
                      at != batch * stride + int64_t(row + e) * 2 * ld + col / 32 * 64 + col % 32) ++wrong;
                });
                if (col < cols)
                  for (int e = 0; e < 8; ++e) {
                    const int64_t o = (int64_t(batch) * rows + row) * cols + col;
                    if (o + (row + e < rows ? int64_t(e) * cols : 0) >= total) ++caught;
                  }
              }
        }
  std::printf("%lld %lld %lld\n", bad, wrong, caught);
  return 0;
}
