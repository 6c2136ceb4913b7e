// Host-side checks of a call's arguments.
#pragma once

#include <stdint.h>

namespace mla {

// Given, and on a boundary of `a` bytes (a power of two).
inline bool aligned_to(const void* p, uintptr_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }
inline bool ok4(const void* p) { return aligned_to(p, 4); }

struct Range {
  const void* at;
  int64_t bytes;          // 0: not used
};
inline bool overlap(const Range& a, const Range& b) {
  const char *x = (const char*)a.at, *y = (const char*)b.at;
  return a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}

}  // namespace mla
