// wq_checks.hpp -- host-side checks of arguments that several entry points share.
#pragma once
#include <stdint.h>

#include "../../include/wq.h"

namespace wq {

inline bool power_of_two(int v) { return v > 0 && (v & (v - 1)) == 0; }

// Row matrices [rows][width] with a row stride: 16-byte loads.
inline wq_status check_rows(const void* p, int64_t ld, int rows, int width) {
  if (!p) return WQ_EINVAL;
  if (rows > 1 && ld < width) return WQ_EINVAL;
  if (((uintptr_t)p & 15) || (rows > 1 && ld % 8 != 0)) return WQ_EUNSUPPORTED;
  return WQ_OK;
}

// Whether two matrices of `rows` rows of wa and wb elements share one.  The rows
// of one may lie between those of the other (slices of one buffer).
inline bool rows_meet(const void* a, int64_t ld_a, int wa, const void* b, int64_t ld_b, int wb, int rows) {
  typedef __int128 Z;  // (any stride)
  if (rows == 1) {
    ld_a = wa;
    ld_b = wb;
  }
  const Z d = ((Z)(uintptr_t)b - (Z)(uintptr_t)a) / 2;  // both are 16-byte aligned
  if (d >= (rows - 1) * (Z)ld_a + wa || -d >= (rows - 1) * (Z)ld_b + wb) return false;
  // rows of a from the first that ends behind b's beginning on; for each the
  // first row of b that ends behind its beginning
  for (Z i = d < wa ? 0 : (d - wa) / ld_a + 1; i < rows; ++i) {
    const Z at = i * ld_a - d;  // from b's beginning
    const Z j = at < wb ? 0 : (at - wb) / ld_b + 1;
    if (j >= rows) return false;
    if (j * ld_b < at + wa) return true;
    if (ld_a == ld_b && at >= wb) return false;  // the same for every further row
  }
  return false;
}

// Whether two byte ranges share one.
inline bool bytes_meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && na && nb && (x < y ? y - x < na : x - y < nb);
}

}  // namespace wq
