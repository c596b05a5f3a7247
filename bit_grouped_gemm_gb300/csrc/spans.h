// spans.h -- host-side checks of the address ranges that a call is given.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

struct Span {
  const void* p;   // may be NULL: the argument is absent
  size_t n;        // bytes
};

inline bool clash(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && x < y + b.n && y < x + a.n;
}

inline bool is_aligned(const void* p, unsigned a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace moe
