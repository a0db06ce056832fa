// Argument checks shared by the C entry points: descriptors, alignment, early returns.
#pragma once

#include <stdint.h>

#include <initializer_list>

#include "../../include/fp8lin.h"

namespace fp8lin {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Scales, maxima and offsets (any may be null) are read and written word by word at least.
inline bool word_aligned(std::initializer_list<const fp8_tensor*> ts) {
  for (const fp8_tensor* t : ts)
    if (t && (reinterpret_cast<uintptr_t>(t->ptr) & 3u) != 0) return false;
  return true;
}
inline bool is_fp8(int dt) { return dt == FP8_DT_E4M3 || dt == FP8_DT_E5M2; }
inline bool is_out(int dt) { return dt == FP8_DT_BF16 || dt == FP8_DT_F32; }
inline int64_t numel(const fp8_tensor* t) {
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
  return n;
}
inline bool valid_desc(const fp8_tensor* t) {
  if (!t || t->ndim < 1 || t->ndim > 3) return false;
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] < 0) return false;
  return t->ptr != nullptr || numel(t) == 0;
}
inline bool shape_is(const fp8_tensor* t, int nd, int64_t a, int64_t b = -1, int64_t c = -1) {
  if (t->ndim != nd) return false;
  const int64_t s[3] = {a, b, c};
  for (int i = 0; i < nd; ++i)
    if (t->shape[i] != s[i]) return false;
  return true;
}
inline int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

}  // namespace fp8lin

#define FP8_CHECK(cond, code) \
  do {                        \
    if (!(cond)) return (code); \
  } while (0)
#define FP8_TRY(expr)        \
  do {                       \
    int rc_ = (expr);        \
    if (rc_ != FP8_OK) return rc_; \
  } while (0)
