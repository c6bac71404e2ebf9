// Argument checks that the host files of the C ABI share (host code, header-only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace {

inline int status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }
inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool float_type(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
inline unsigned size_of(int32_t t) { return t == MOE_BF16 ? 2u : 4u; }

// Rows of `bytes` bytes, `step` bytes from one to the next, in memory.
struct Rows {
  const void* p;
  long long rows;
  unsigned long long bytes, step;
};
inline Rows flat(const void* p, unsigned long long bytes) { return {p, 1, bytes, bytes}; }
inline Rows float_rows(const void* p, int32_t type, int64_t ld, int64_t rows, int64_t n) {
  return {p, rows, (unsigned long long)n * size_of(type), (unsigned long long)ld * size_of(type)};
}

// Whether [y, y + n) holds a byte of one of those rows (128 bits: rows may reach past any address).
inline bool overlaps(const void* y, unsigned long long n, const Rows& r) {
  typedef unsigned __int128 wide;
  if (!y || !r.p || n == 0 || r.rows < 1 || r.bytes == 0) return false;
  const wide lo = reinterpret_cast<uintptr_t>(y), hi = lo + n, first = reinterpret_cast<uintptr_t>(r.p);
  if (hi <= first || lo >= first + (wide)(r.rows - 1) * r.step + r.bytes) return false;
  // the last row that starts at or before y, and the one after it
  const wide at = lo > first ? (lo - first) / r.step : 0;
  for (wide i = at; i < at + 2 && i < (wide)r.rows; ++i)
    if (lo < first + i * r.step + r.bytes && first + i * r.step < hi) return true;
  return false;
}

}  // namespace
