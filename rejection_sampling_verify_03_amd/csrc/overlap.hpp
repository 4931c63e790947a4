// overlap.hpp -- whether rows of memory, given by their strides, have a place in
// common (host code: what a call must not write twice, or read and write).
#pragma once

#include <stdint.h>

namespace specv {

// n x m rows of len bytes, row (i, j) at base + i * outer + j * inner (strides >= 0).
struct MemRows {
  uintptr_t base;
  int64_t n, outer, m, inner, len;
};
using wide_t = __int128;  // (strides may be any)

// The bytes from the first row's beginning to the last one's end.
inline wide_t rows_span(const MemRows& r) { return (wide_t)(r.n - 1) * r.outer + (wide_t)(r.m - 1) * r.inner + r.len; }

// Whether d + i * step, for some i in [lo, hi], lies within (-a, b).
inline bool some_within(wide_t d, wide_t step, int64_t lo, int64_t hi, int64_t a, int64_t b) {
  int64_t i = lo;
  if (step > 0) {  // the first multiple above -a
    const wide_t need = -(wide_t)a + 1 - d;
    const wide_t k = need > 0 ? (need + step - 1) / step : -(-need / step);
    if (k > hi) return false;
    if (k > lo) i = (int64_t)k;
  }
  const wide_t x = d + i * step;
  return x > -(wide_t)a && x < b;
}

// Whether two rows of r share a byte.
inline bool rows_share(const MemRows& r) {
  if (r.n > 1 && r.outer < r.len) return true;
  if (r.m > 1 && r.inner < r.len) return true;
  if (r.n == 1 || r.m == 1) return false;
  if (r.outer >= (wide_t)(r.m - 1) * r.inner + r.len || r.inner >= (wide_t)(r.n - 1) * r.outer + r.len) return false;
  for (int64_t j = 1; j < r.m; ++j)
    if (some_within(-(wide_t)j * r.inner, r.outer, 0, r.n - 1, r.len, r.len)) return true;
  return false;
}

// Whether a row of a and one of b share a byte; b's rows do not share any among
// themselves.  (True also where strides differ and b's rows stand neither in the
// order of i, j nor in that of j, i, unless all of b lies in front of a or behind.)
inline bool rows_meet(const MemRows& a, const MemRows& b) {
  const wide_t d = (wide_t)b.base - (wide_t)a.base;  // row (0, 0) of b behind that of a
  if (d >= rows_span(a) || -d >= rows_span(b)) return false;
  if (a.n == b.n && (a.n == 1 || a.outer == b.outer)) {
    const int64_t n = a.n, T = n == 1 ? 0 : a.outer;
    // (parts of the same rows: one behind the other in each)
    const wide_t ea = (wide_t)(a.m - 1) * a.inner + a.len, eb = (wide_t)(b.m - 1) * b.inner + b.len;
    if (T > 0) {
      const wide_t r = (d % T + T) % T;
      if (r >= ea && r + eb <= T) return false;
    }
    const bool same = a.inner == b.inner;  // (then the difference of the two j counts)
    for (int64_t j = same ? 1 - a.m : 0; j < b.m; ++j)
      for (int64_t k = 0; k < (same ? 1 : a.m); ++k)
        if (some_within(d + (wide_t)j * b.inner - (wide_t)k * a.inner, T, 1 - n, n - 1, b.len, a.len)) return true;
    return false;
  }
  const bool by_n = b.outer >= (wide_t)(b.m - 1) * b.inner + b.len || b.n == 1;
  if (!by_n && b.m > 1 && b.inner < (wide_t)(b.n - 1) * b.outer + b.len) return true;  // (not told apart)
  const int64_t n = by_n ? b.n : b.m, m = by_n ? b.m : b.n, outer = by_n ? b.outer : b.inner,
                inner = by_n ? b.inner : b.outer;
  for (int64_t i = 0; i < a.n; ++i)
    for (int64_t j = 0; j < a.m; ++j) {
      // the last row of b that begins in front of the end of a's row (i, j)
      const wide_t x = (wide_t)i * a.outer + (wide_t)j * a.inner - d, last = x + a.len - 1;
      if (last < 0) continue;
      wide_t p = outer > 0 ? last / outer : 0;
      p = p < n ? p : n - 1;
      wide_t q = inner > 0 ? (last - p * outer) / inner : 0;
      q = q < m ? q : m - 1;
      if (p * outer + q * inner + b.len > x) return true;
    }
  return false;
}

}  // namespace specv
