// fa_rows.h -- do output rows lie on one another? Plain C++: no CUDA header, so the logic is tested
// on its own with a host compiler.
//
// A tensor of `heads` x `rows` rows of `d` contiguous elements has row i of head h at
// h * st_h + i * st_r (elements, strides not negative).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace fa {

struct RowGrid {
  int64_t heads, rows, st_h, st_r;
};

// Whether a row of the grid and a row of the same grid moved by `offset` elements share one: some
// |i| < heads, |j| < rows have |i st_h + j st_r + offset| < d. (offset 0: rows other than the same,
// so (i, j) is not (0, 0).) For each i only the two j around -(i st_h + offset) / st_r can do;
// 2 * heads steps.
inline bool rows_meet(const RowGrid& g, int64_t offset, int64_t d) {
  if (g.heads <= 0 || g.rows <= 0) return false;
  for (int64_t i = 1 - g.heads; i < g.heads; ++i) {
    const int64_t at = i * g.st_h + offset;
    int64_t near = 0;
    if (g.st_r > 0) near = std::clamp(-at / g.st_r, 1 - g.rows, g.rows - 1);
    for (int64_t j = std::max(near - 1, 1 - g.rows); j <= std::min(near + 1, g.rows - 1); ++j) {
      if (offset == 0 && i == 0 && j == 0) continue;
      const int64_t x = at + j * g.st_r;
      if (x > -d && x < d) return true;
    }
  }
  return false;
}

// Whether the rows of two such tensors, `offset` elements from a's first to b's, may be written by
// one call: neither's own lie on one another, nor a's on b's. Where the two have different strides
// (those of dimensions of one element do not count) only a's and b's first rows are compared.
inline bool rows_apart(RowGrid a, RowGrid b, int64_t offset, int64_t d) {
  for (RowGrid* g : {&a, &b}) {
    if (g->heads == 1) g->st_h = 0;
    if (g->rows == 1) g->st_r = 0;
  }
  for (const RowGrid* g : {&a, &b})  // no memory has as many elements (and nothing below overflows)
    if ((double)g->heads * (double)g->st_h + (double)g->rows * (double)g->st_r > 1e15) return false;
  if (rows_meet(a, 0, d) || rows_meet(b, 0, d)) return false;
  if (a.heads <= 0 || a.rows <= 0) return true;
  if (a.st_h != b.st_h || a.st_r != b.st_r) return offset <= -d || offset >= d;
  return offset != 0 && !rows_meet(a, offset, d);
}

}  // namespace fa
