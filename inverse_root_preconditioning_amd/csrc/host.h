// Host-side checks that the entry points of the layers share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/shampoo.h"

namespace shp {

// A launch has fewer than 2^32 threads along x.
constexpr int64_t kMaxThreads = 0xffffffff;
constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxCols = (int64_t)1 << 29;  // byte offsets within a row have 32 bits

inline int check_launch() { return hipGetLastError() == hipSuccess ? SHAMPOO_OK : SHAMPOO_EHIP; }
inline bool valid_type(int64_t t) { return t == SHAMPOO_T_F32 || t == SHAMPOO_T_BF16; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool valid_mx8(const void* codes, const void* scales) {
  return codes != nullptr && scales != nullptr && aligned16(codes) && aligned16(scales);
}
inline int check_sides(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return SHAMPOO_EINVAL;
  return rows > kMaxRows || cols > kMaxCols ? SHAMPOO_EUNSUPPORTED : SHAMPOO_OK;
}

// Lanes (a power of two, 16 to 256) that take a row of pieces of `elems`, and
// how many such stretches a row has.
inline void row_shape(int64_t padded, int64_t elems, int* lanes_log2, int64_t* col_blocks) {
  int k = 4;
  while (k < 8 && (elems << k) < padded) ++k;
  *lanes_log2 = k;
  *col_blocks = (padded + (elems << k) - 1) / (elems << k);
}

}  // namespace shp
