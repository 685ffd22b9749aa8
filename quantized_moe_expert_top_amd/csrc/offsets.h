// Byte offsets of buffer accesses by the lanes.  Plain C++ for host and device.
#pragma once
#include <stdint.h>

namespace moe {

constexpr uint32_t kOut = ~0u;  // past any buffer: a load gives zero

// off + add, and kOut where off is: the plain sum would wrap around to the buffer's first bytes.
constexpr uint32_t offset_sum(uint32_t off, uint32_t add) { return off == kOut ? kOut : off + add; }

// Column `col` of row `row` of 16-bit numbers [rows][ld] of less than 4 GiB; kOut for a row past
// them (whose plain product may pass 2^32, with long rows).
constexpr uint32_t row_offset(uint32_t row, uint32_t rows, uint32_t ld, uint32_t col) {
  return row < rows ? (row * ld + col) * 2 : kOut;
}

}  // namespace moe
