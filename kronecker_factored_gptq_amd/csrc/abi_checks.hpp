// Checks of arguments that the calls beside the solve share. Host only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "bakron.h"

namespace bk {

inline size_t type_size(int t) { return t == BAKRON_F32 ? 4 : t == BAKRON_BF16 || t == BAKRON_F16 ? 2 : 0; }
inline bool type_ok(int t) { return type_size(t) != 0; }

// whether a matrix of `rows` x `cols` elements of `es` bytes can be addressed
inline bool matrix_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
  if (rows == 0 || cols == 0) return true;
  return p && ld >= cols && ld <= (INT64_MAX / 8) / rows && (uintptr_t)p % es == 0;
}
// whether two matrices' byte ranges intersect
inline bool overlap(const void* a, int64_t arows, int64_t acols, int64_t lda, size_t ea,
                    const void* b, int64_t brows, int64_t bcols, int64_t ldb, size_t eb) {
  if (!a || !b || arows == 0 || acols == 0 || brows == 0 || bcols == 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  const uintptr_t a1 = a0 + ((uintptr_t)(arows - 1) * (uintptr_t)lda + (uintptr_t)acols) * ea;
  const uintptr_t b1 = b0 + ((uintptr_t)(brows - 1) * (uintptr_t)ldb + (uintptr_t)bcols) * eb;
  return a0 < b1 && b0 < a1;
}
inline int status(hipError_t e) { return e == hipSuccess ? BAKRON_OK : BAKRON_EHIP; }

// A launch holds fewer than 2^32 threads: 2^24 - 1 workgroups of 256.
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;
// whether tiles of 128 x 128 over an a x b output fit one launch
inline bool tiles_ok(int64_t a, int64_t b) {
  return ((a + 127) / 128) * ((b + 127) / 128) <= kMaxGroups;
}
// the workgroups that lay out `rows` rows of 16-bit planes, eight elements a thread
inline int64_t plane_groups(int64_t rows, int64_t cols) { return rows * (cols + 64) / 2048 + 1; }

constexpr size_t kAlign = 256;
// Rows of planes short enough for the tile product's 32-bit offsets.
constexpr int64_t kMaxPlaneCols = (int64_t)1 << 20;

}  // namespace bk
