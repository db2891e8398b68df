// Which rows the ring takes by bulk copies and which bytes these read: plain C++ as
// well, so that it can be checked without a GPU.
//
// Rows that do not lie on 16-byte boundaries are copied with the whole 16-byte words
// that hold their ends, up to 15 bytes more on either side, which belong to the rows
// beside them; the first and last rows of all, whose words may reach in front of the
// matrix or behind it, are read in place.
#pragma once

#include <stdint.h>

#ifndef Q4_HOST_DEVICE
#ifdef __CUDACC__
#define Q4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define Q4_HOST_DEVICE inline
#endif
#endif

namespace q4 {
namespace {

// Rows at either end that are read in place: 15 bytes of neighbours (whose pitch is
// no less than a row).
Q4_HOST_DEVICE constexpr int edge_rows(uint32_t row_bytes) { return (int)((15 + row_bytes - 1) / row_bytes); }
// (rows >= 2 edge)
Q4_HOST_DEVICE bool read_in_place(int64_t row, int64_t rows, int edge) {
  return (uint64_t)(row - edge) >= (uint64_t)(rows - 2 * edge);
}

// Of the per_block rows from `base` on, `begin` .. `end` - 1 are copied.
struct CopiedRows {
  int begin, end;
};
Q4_HOST_DEVICE CopiedRows copied_rows(int64_t base, int per_block, int64_t rows, int edge) {
  const int64_t left = rows - edge - base;
  return {base < edge ? (int)(edge - base) : 0, left < per_block ? (int)left : per_block};
}

// The words that hold row_bytes bytes at `at`.
struct Window {
  uintptr_t begin;
  uint32_t size;
};
Q4_HOST_DEVICE Window window_of(uintptr_t at, uint32_t row_bytes) {
  const uintptr_t begin = at & ~uintptr_t(15);
  return {begin, (uint32_t)(((at + row_bytes + 15) & ~uintptr_t(15)) - begin)};
}
// Room for a window of any alignment.
Q4_HOST_DEVICE constexpr uint32_t window_bytes(uint32_t row_bytes) { return (row_bytes + 30) / 16 * 16; }

}  // namespace
}  // namespace q4
