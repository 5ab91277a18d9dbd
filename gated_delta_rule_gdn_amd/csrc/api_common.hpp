// api_common.hpp -- argument-checking helpers shared by the C ABI layers
// (gdn_api.cpp, attn_api.cpp).
#pragma once

#include <cstdint>

#include "gdn.h"
#include "gdn_kernels.hpp"

namespace gdn {

struct Span {
  uintptr_t lo, hi;  // [lo, hi)
  bool valid() const { return hi > lo; }
};

inline Span span(const void* p, int64_t elems, int64_t elem_bytes) {
  Span s{0, 0};
  if (p && elems > 0) {
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + static_cast<uintptr_t>(elems * elem_bytes);
  }
  return s;
}

inline bool overlaps(const Span& a, const Span& b) {
  return a.valid() && b.valid() && a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int64_t dtype_bytes(int32_t d) { return d == GDN_F32 ? 4 : 2; }

inline DType to_dtype(int32_t d) { return d == GDN_F32 ? DType::F32 : DType::BF16; }

}  // namespace gdn
