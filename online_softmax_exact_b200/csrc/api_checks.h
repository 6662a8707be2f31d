// api_checks.h - helpers of the C ABI's argument checks (host only; no CUDA call).
#pragma once

#include <cstdint>

namespace osx {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

struct Span {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Span span(const void* p, uint64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + static_cast<uintptr_t>(bytes)};
}

inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// The status injected by attn_debug_inject for this call (ATTN_OK: none).
int take_injected();

}  // namespace osx
