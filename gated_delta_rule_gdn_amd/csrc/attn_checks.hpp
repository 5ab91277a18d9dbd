// attn_checks.hpp -- argument checks shared by the C ABI layers of the attention
// operators (attn_api.cpp, hybrid_api.cpp).
#pragma once

#include <cmath>
#include <cstdint>

#include "api_common.hpp"
#include "gdn_attn.h"

namespace gdn {

constexpr double kMaxElems = 2.0e15;                 // of any tensor
constexpr double kMaxThreads = 4294967295.0;         // of a grid

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline gdn_status check_head(int32_t d, int32_t io) {
  if (io != GDN_F32 && io != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (d < 1) return GDN_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// A strided operand of `rows` rows of H heads.
inline gdn_status check_rows(int64_t rows, int64_t ld, int32_t H, int32_t d) {
  const int64_t cols = (int64_t)H * d;
  if (cols > (int64_t(1) << 22)) return GDN_ERR_UNSUPPORTED;
  if (ld < cols || ld % 8 != 0 || ld > (int64_t(1) << 24)) return GDN_ERR_INVALID_ARG;
  if ((double)rows * (double)ld > kMaxElems) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

inline Span rows_span(const void* p, int64_t rows, int64_t ld, int32_t H, int32_t d, int32_t io) {
  return rows > 0 ? span(p, (rows - 1) * ld + (int64_t)H * d, dtype_bytes(io)) : Span{0, 0};
}

inline gdn_status check_rope(int32_t dim, int32_t mode, float factor, float eps, int32_t d) {
  if (dim < 0 || dim > d || dim % 16 != 0) return GDN_ERR_INVALID_ARG;
  if (mode != GDN_ROPE_HALF && mode != GDN_ROPE_INTERLEAVED) return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(factor) || !std::isfinite(eps) || eps < 0.f) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

// No output overlaps an input or another output.
template <size_t I, size_t O>
bool apart(const Span (&ins)[I], const Span (&outs)[O]) {
  for (size_t o = 0; o < O; ++o) {
    for (const Span& in : ins)
      if (overlaps(outs[o], in)) return false;
    for (size_t i = 0; i < o; ++i)
      if (overlaps(outs[o], outs[i])) return false;
  }
  return true;
}

// Two outputs of rows `w` bytes wide, `ld` bytes from one to the next, share no byte:
// apart as wholes, or column blocks of one buffer.
inline bool blocks_apart(const Span& a, int64_t lda, int64_t wa, const Span& b, int64_t ldb, int64_t wb) {
  if (!overlaps(a, b)) return true;
  if (lda != ldb) return false;
  const int64_t gap = a.lo < b.lo ? (int64_t)(b.lo - a.lo) : (int64_t)(a.lo - b.lo);
  const int64_t at = gap % lda, first = a.lo < b.lo ? wa : wb, second = a.lo < b.lo ? wb : wa;
  return at >= first && at + second <= lda;
}

}  // namespace gdn
