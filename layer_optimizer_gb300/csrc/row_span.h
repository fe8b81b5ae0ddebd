// Which bytes of a matrix row a bulk copy brings.  A copy starts and ends on
// 16 bytes; a row that starts off a unit of eight columns seldom does.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SF_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SF_HOST_DEVICE inline
#endif

namespace sf {

// Bytes [begin, end), counted from the unit (8 * size bytes, aligned) that
// holds the row's first column, which is column m of it.
struct CopySpan {
  uint32_t begin, end;
};

// The 16-byte units that hold any of the row.  `last`: of the matrix's last
// row, those that the row fills to their end, since past it the matrix ends:
// the columns from `end` on come with ordinary loads.  (Row 0 starts on a unit, so
// no row's first unit reaches before the matrix.)
SF_HOST_DEVICE CopySpan copy_span(uint32_t m, uint32_t cols, uint32_t size, bool last) {
  return CopySpan{(m * size) & ~15u, ((m + cols) * size + (last ? 0u : 15u)) & ~15u};
}

}  // namespace sf
