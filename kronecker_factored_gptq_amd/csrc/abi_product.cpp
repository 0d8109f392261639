// C ABI of the calls beside the solve (declared in include/bakron.h): the
// 8-bit product of quantised tokens with a layer's codes, and the cross entropy
// over a vocabulary. Host side only: argument checks and the choice of types;
// nothing here touches data.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "bakron.h"
#include "launch.hpp"
#include "tile_product.hpp"

namespace {

using namespace bk;

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

// the largest n whose int8 sums fit int32: 128 * 128 * 131071 < 2^31
constexpr int64_t kMaxInt8Sum = 131071;
// A launch holds fewer than 2^32 threads: 2^24 - 1 workgroups of 256.
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;
// whether tiles of 128 x 128 over an a x b output fit one launch
inline bool tiles_ok(int64_t a, int64_t b) {
  return ((a + 127) / 128) * ((b + 127) / 128) <= kMaxGroups;
}
// the workgroups that lay out `rows` rows of 16-bit planes, eight elements a thread
inline int64_t plane_groups(int64_t rows, int64_t cols) { return rows * (cols + 64) / 2048 + 1; }

inline bool int8_sizes_ok(int64_t T, int64_t m, int64_t n) {
  return T >= 0 && m >= 0 && n >= 0 && T <= kMaxGroups && m <= kMaxGroups && n <= kMaxInt8Sum &&
         tiles_ok(T, m) && (T + m) * (n + 128) / 4096 < kMaxGroups;  // rows laid out, 16 bytes a thread
}

constexpr size_t kAlign = 256;

// Sizes of the input gradient: rows of planes short enough for the tile
// product's 32-bit offsets.
constexpr int64_t kMaxPlaneCols = (int64_t)1 << 20;
inline bool grad_sizes_ok(int t, int64_t T, int64_t m, int64_t n) {
  return type_ok(t) && T >= 0 && m >= 0 && n >= 0 && T <= kMaxGroups && m <= kMaxPlaneCols &&
         n <= kMaxPlaneCols && tiles_ok(T, n) &&
         T + plane_groups(T, m) + plane_groups(m, n) <= kMaxGroups;
}

inline bool entropy_sizes_ok(int t, int64_t T, int64_t d, int64_t V) {
  return type_ok(t) && T >= 0 && d >= 0 && V >= 1 && T <= kMaxPlaneCols && d <= kMaxPlaneCols &&
         V <= kMaxGroups && tiles_ok(T, V) && tiles_ok(d, V) && tiles_ok(T, d) &&
         plane_groups(T, d) <= kMaxGroups &&
         plane_groups(V < kMaxPlaneCols ? V : kMaxPlaneCols, d) <= kMaxGroups;
}

}  // namespace

extern "C" {

int bakron_quantize_tokens(int xtype, int64_t T, int64_t n, const void* X, int64_t ldx,
                           const float* channel, int8_t* Xq, int64_t ldq, float* sx, void* stream) {
  if (!type_ok(xtype) || T < 0 || n < 0 || T > kMaxGroups) return BAKRON_EINVAL;
  if (T == 0) return BAKRON_OK;
  if (!matrix_ok(X, T, n, ldx, type_size(xtype)) || !matrix_ok(Xq, T, n, ldq, 1)) return BAKRON_EINVAL;
  if (!sx || (uintptr_t)sx % 4 || (uintptr_t)channel % 4) return BAKRON_EINVAL;
  const size_t es = type_size(xtype);
  if (overlap(Xq, T, n, ldq, 1, X, T, n, ldx, es) || overlap(Xq, T, n, ldq, 1, sx, 1, T, T, 4) ||
      overlap(sx, 1, T, T, 4, X, T, n, ldx, es) || overlap(Xq, T, n, ldq, 1, channel, 1, n, n, 4) ||
      overlap(sx, 1, T, T, 4, channel, 1, n, n, 4))
    return BAKRON_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (xtype == BAKRON_F32)
    return status(launch_quantize_tokens(T, n, (const float*)X, ldx, channel, Xq, ldq, sx, s));
  if (xtype == BAKRON_BF16)
    return status(launch_quantize_tokens(T, n, (const BF16*)X, ldx, channel, Xq, ldq, sx, s));
  return status(launch_quantize_tokens(T, n, (const F16*)X, ldx, channel, Xq, ldq, sx, s));
}

size_t bakron_matmul_int8_workspace_bytes(int64_t T, int64_t m, int64_t n) {
  if (!int8_sizes_ok(T, m, n)) return 0;
  const size_t b = matmul_int8_bytes(T, m, n);
  return b ? b + kAlign : 0;
}

int bakron_matmul_int8(int ytype, int64_t T, int64_t m, int64_t n, const int8_t* Xq, int64_t ldx,
                       const float* sx, const int8_t* Vq, int64_t ldv, const float* sv, void* Y,
                       int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (!type_ok(ytype) || !int8_sizes_ok(T, m, n)) return BAKRON_EINVAL;
  if (T == 0 || m == 0) return BAKRON_OK;
  const size_t es = type_size(ytype);
  const size_t need = matmul_int8_bytes(T, m, n);
  if (need && (!workspace || (uintptr_t)workspace % kAlign || workspace_bytes < need))
    return BAKRON_EINVAL;
  if (!matrix_ok(Xq, T, n, ldx, 1) || !matrix_ok(Vq, m, n, ldv, 1) ||
      !matrix_ok(Y, T, m, ldy, es))
    return BAKRON_EINVAL;
  if (!sx || (uintptr_t)sx % 4 || (uintptr_t)sv % 4) return BAKRON_EINVAL;
  if (overlap(Y, T, m, ldy, es, Xq, T, n, ldx, 1) || overlap(Y, T, m, ldy, es, Vq, m, n, ldv, 1) ||
      overlap(Y, T, m, ldy, es, sx, 1, T, T, 4) || overlap(Y, T, m, ldy, es, sv, 1, m, m, 4))
    return BAKRON_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (ytype == BAKRON_F32)
    return status(launch_matmul_int8(T, m, n, Xq, ldx, sx, Vq, ldv, sv, (float*)Y, ldy, workspace, s));
  if (ytype == BAKRON_BF16)
    return status(launch_matmul_int8(T, m, n, Xq, ldx, sx, Vq, ldv, sv, (BF16*)Y, ldy, workspace, s));
  return status(launch_matmul_int8(T, m, n, Xq, ldx, sx, Vq, ldv, sv, (F16*)Y, ldy, workspace, s));
}

size_t bakron_matmul_int8_grad_workspace_bytes(int gtype, int64_t T, int64_t m, int64_t n) {
  if (!grad_sizes_ok(gtype, T, m, n)) return 0;
  return matmul_int8_grad_bytes((int)type_size(gtype), T, m, n) + kAlign;
}

int bakron_matmul_int8_grad(int gtype, int64_t T, int64_t m, int64_t n, const void* G, int64_t ldg,
                            const int8_t* Vq, int64_t ldv, const float* sv, const float* channel,
                            void* dX, int64_t ldx, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (!grad_sizes_ok(gtype, T, m, n)) return BAKRON_EINVAL;
  if (T == 0 || n == 0) return BAKRON_OK;
  const size_t es = type_size(gtype);
  if (!matrix_ok(G, T, m, ldg, es) || !matrix_ok(Vq, m, n, ldv, 1) ||
      !matrix_ok(dX, T, n, ldx, es))
    return BAKRON_EINVAL;
  if ((uintptr_t)sv % 4 || (uintptr_t)channel % 4) return BAKRON_EINVAL;
  if (!workspace || (uintptr_t)workspace % kAlign ||
      workspace_bytes < matmul_int8_grad_bytes((int)type_size(gtype), T, m, n))
    return BAKRON_EINVAL;
  if (overlap(dX, T, n, ldx, es, G, T, m, ldg, es) || overlap(dX, T, n, ldx, es, Vq, m, n, ldv, 1) ||
      overlap(dX, T, n, ldx, es, sv, 1, m, m, 4) || overlap(dX, T, n, ldx, es, channel, 1, n, n, 4))
    return BAKRON_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (gtype == BAKRON_F32)
    return status(launch_matmul_int8_grad(T, m, n, (const float*)G, ldg, Vq, ldv, sv, channel,
                                          (float*)dX, ldx, workspace, s));
  if (gtype == BAKRON_BF16)
    return status(launch_matmul_int8_grad(T, m, n, (const BF16*)G, ldg, Vq, ldv, sv, channel,
                                          (BF16*)dX, ldx, workspace, s));
  return status(launch_matmul_int8_grad(T, m, n, (const F16*)G, ldg, Vq, ldv, sv, channel, (F16*)dX,
                                        ldx, workspace, s));
}

size_t bakron_cross_entropy_workspace_bytes(int xtype, int64_t T, int64_t d, int64_t V) {
  if (!entropy_sizes_ok(xtype, T, d, V)) return 0;
  return entropy_bytes((int)type_size(xtype), T, d, V) + kAlign;
}

int bakron_cross_entropy(int xtype, int64_t T, int64_t d, int64_t V, const void* X, int64_t ldx,
                         const void* W, int64_t ldw, const int64_t* targets, float* loss,
                         float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!entropy_sizes_ok(xtype, T, d, V)) return BAKRON_EINVAL;
  if (T == 0) return BAKRON_OK;
  const size_t es = type_size(xtype);
  if (!matrix_ok(X, T, d, ldx, es) || !matrix_ok(W, V, d, ldw, es)) return BAKRON_EINVAL;
  if (!targets || !loss || !lse || (uintptr_t)targets % 8 || (uintptr_t)loss % 4 || (uintptr_t)lse % 4)
    return BAKRON_EINVAL;
  if (!workspace || (uintptr_t)workspace % kAlign ||
      workspace_bytes < entropy_bytes((int)es, T, d, V))
    return BAKRON_EINVAL;
  for (const float* o : {loss, lse})
    if (overlap(o, 1, T, T, 4, X, T, d, ldx, es) || overlap(o, 1, T, T, 4, W, V, d, ldw, es) ||
        overlap(o, 1, T, T, 4, targets, 1, T, T, 8))
      return BAKRON_EINVAL;
  if (overlap(loss, 1, T, T, 4, lse, 1, T, T, 4)) return BAKRON_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (xtype == BAKRON_F32)
    return status(launch_entropy(T, d, V, (const float*)X, ldx, (const float*)W, ldw, targets, loss,
                                 lse, workspace, s));
  if (xtype == BAKRON_BF16)
    return status(launch_entropy(T, d, V, (const BF16*)X, ldx, (const BF16*)W, ldw, targets, loss,
                                 lse, workspace, s));
  return status(launch_entropy(T, d, V, (const F16*)X, ldx, (const F16*)W, ldw, targets, loss, lse,
                               workspace, s));
}

size_t bakron_cross_entropy_grad_workspace_bytes(int xtype, int64_t T, int64_t d, int64_t V) {
  if (!entropy_sizes_ok(xtype, T, d, V)) return 0;
  return entropy_grad_bytes((int)type_size(xtype), T, d, V) + kAlign;
}

int bakron_cross_entropy_grad(int xtype, int64_t T, int64_t d, int64_t V, const void* X,
                              int64_t ldx, const void* W, int64_t ldw, const int64_t* targets,
                              const float* lse, const float* g, void* dX, int64_t lddx, void* dW,
                              int64_t lddw, void* workspace, size_t workspace_bytes, void* stream) {
  if (!entropy_sizes_ok(xtype, T, d, V)) return BAKRON_EINVAL;
  if (d == 0 || (!dX && !dW) || (T == 0 && !dW)) return BAKRON_OK;
  const size_t es = type_size(xtype);
  if (!matrix_ok(X, T, d, ldx, es) || !matrix_ok(W, V, d, ldw, es)) return BAKRON_EINVAL;
  if ((dX && !matrix_ok(dX, T, d, lddx, es)) || (dW && !matrix_ok(dW, V, d, lddw, es)))
    return BAKRON_EINVAL;
  if (T > 0 && (!targets || !lse || !g || (uintptr_t)targets % 8 || (uintptr_t)lse % 4 ||
                (uintptr_t)g % 4))
    return BAKRON_EINVAL;
  if (!workspace || (uintptr_t)workspace % kAlign ||
      workspace_bytes < entropy_grad_bytes((int)es, T, d, V))
    return BAKRON_EINVAL;
  const struct {
    const void* p;
    int64_t rows, ld;
  } outs[2] = {{dX, T, lddx}, {dW, V, lddw}};
  for (const auto& o : outs)
    if (overlap(o.p, o.rows, d, o.ld, es, X, T, d, ldx, es) ||
        overlap(o.p, o.rows, d, o.ld, es, W, V, d, ldw, es) ||
        overlap(o.p, o.rows, d, o.ld, es, targets, 1, T, T, 8) ||
        overlap(o.p, o.rows, d, o.ld, es, lse, 1, T, T, 4) ||
        overlap(o.p, o.rows, d, o.ld, es, g, 1, T, T, 4))
      return BAKRON_EINVAL;
  if (overlap(dX, T, d, lddx, es, dW, V, d, lddw, es)) return BAKRON_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (xtype == BAKRON_F32)
    return status(launch_entropy_grad(T, d, V, (const float*)X, ldx, (const float*)W, ldw, targets,
                                      lse, g, (float*)dX, lddx, (float*)dW, lddw, workspace, s));
  if (xtype == BAKRON_BF16)
    return status(launch_entropy_grad(T, d, V, (const BF16*)X, ldx, (const BF16*)W, ldw, targets,
                                      lse, g, (BF16*)dX, lddx, (BF16*)dW, lddw, workspace, s));
  return status(launch_entropy_grad(T, d, V, (const F16*)X, ldx, (const F16*)W, ldw, targets, lse, g,
                                    (F16*)dX, lddx, (F16*)dW, lddw, workspace, s));
}

double bakron_debug_plan(int64_t M, int64_t N, int64_t steps, int pairs, int kmajor, int may_split,
                         int32_t* tile, int32_t* splits) {
  if (M < 1 || N < 1 || steps < 0 || pairs < 1 || !tile || !splits) return __builtin_inf();
  if (*tile == 0) {
    const TilePlan p = plan_tiles(M, N, steps, pairs, kmajor, may_split);
    *tile = p.tile;
    *splits = p.splits;
  }
  if (*tile == 256) return 0;
  if ((*tile != 128 && *tile != 64) || *splits < 1 ||
      !plan_allowed(M, N, steps * pairs, pairs, may_split, *tile, *splits))
    return __builtin_inf();
  return plan_us(M, N, steps * pairs, pairs, kmajor, *tile, *splits);
}

}  // extern "C"
