// Whether two strided tensors of token rows share a byte.  Host code.
#pragma once

#include <cstdint>

namespace pagedkv {

// n rows of `row` bytes from `at` on, `stride` >= row bytes apart.
struct TokenRows {
  uintptr_t at;
  int64_t row, stride;
};

inline bool rows_overlap(const TokenRows& a, const TokenRows& b, int64_t n) {
  using Wide = __int128;
  if (n <= 0 || a.row <= 0 || b.row <= 0) return false;
  const Wide a0 = a.at, b0 = b.at;
  if (a0 + Wide(n - 1) * a.stride + a.row <= b0 || b0 + Wide(n - 1) * b.stride + b.row <= a0) return false;
  if (a.stride == b.stride) {
    // row i of a meets row j of b iff (i - j) stride lies inside (b0 - a0 - a.row, b0 - a0 + b.row)
    const Wide s = a.stride, lo = b0 - a0 - a.row, hi = b0 - a0 + b.row;
    Wide k = lo / s - (lo % s < 0 ? 1 : 0) + 1;  // the first multiple above lo
    if (k <= -Wide(n)) k = -Wide(n) + 1;
    return k < Wide(n) && k * s < hi;
  }
  // rows in order of address, the earlier end steps on
  for (int64_t i = 0, j = 0; i < n && j < n;) {
    const Wide ai = a0 + Wide(i) * a.stride, bj = b0 + Wide(j) * b.stride;
    if (ai < bj + b.row && bj < ai + a.row) return true;
    if (ai + a.row <= bj + b.row) ++i;
    else ++j;
  }
  return false;
}

}  // namespace pagedkv
