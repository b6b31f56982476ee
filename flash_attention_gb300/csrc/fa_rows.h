// fa_rows.h -- do rows lie on one another? Plain C++: no CUDA header, so the logic is tested on its own
// with a host compiler.
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

// Rows of d contiguous elements, row i of head h of sequence b at b st[0] + h st[1] + i st[2]
// (extents of at least 1, strides not negative, no tensor of more than 10^15 elements).
struct RowBox {
  int64_t n[3], st[3];
};

// A number of steps: x * s for lo <= x <= hi.
struct RowStep {
  int64_t s, lo, hi;
};

// Whether some sum of one number of each of the n steps, which descend, lies less than d from `at`.
// `budget` counts the sums of the larger steps that are looked at; yes where it is used up.
inline bool steps_reach(const RowStep* step, int n, int64_t at, int64_t d, int& budget) {
  if (n == 0) return at > -d && at < d;
  int64_t lo = 0, hi = 0;  // what the smaller steps can add
  for (int i = 1; i < n; ++i) {
    lo += step[i].s * step[i].lo;
    hi += step[i].s * step[i].hi;
  }
  auto down = [](int64_t x, int64_t s) { return x / s - (x % s < 0); };  // x / s, rounded down
  const int64_t s = step[0].s;
  const int64_t x0 = std::max(step[0].lo, -down(hi + d - 1 - at, s));
  const int64_t x1 = std::min(step[0].hi, down(at - lo + d - 1, s));
  if (n == 1) return x0 <= x1;
  for (int64_t x = x0; x <= x1; ++x)
    if (--budget < 0 || steps_reach(step + 1, n - 1, at - x * s, d, budget)) return true;
  return false;
}

// Whether a row of a and a row of b, whose first row lies `offset` elements behind a's, share an
// element. Of dimensions with the same stride only the difference of the two indexes counts; where
// strides nest, each step leaves two or three numbers for the next, so that views of one tensor take
// some ten steps.
inline bool boxes_meet(const RowBox& a, const RowBox& b, int64_t offset, int64_t d) {
  RowStep step[6];
  int n = 0;
  auto add = [&](int64_t s, int64_t lo, int64_t hi) {
    if (s != 0 && lo != hi) step[n++] = {s, lo, hi};
  };
  for (int k = 0; k < 3; ++k) {
    if (a.st[k] == b.st[k] || a.n[k] == 1 || b.n[k] == 1) {
      add(a.n[k] == 1 ? b.st[k] : a.st[k], 1 - b.n[k], a.n[k] - 1);
    } else {
      add(a.st[k], 0, a.n[k] - 1);
      add(b.st[k], 1 - b.n[k], 0);
    }
  }
  std::sort(step, step + n, [](const RowStep& x, const RowStep& y) { return x.s > y.s; });
  int budget = 4096;
  return steps_reach(step, n, offset, d, budget);
}

}  // namespace fa
