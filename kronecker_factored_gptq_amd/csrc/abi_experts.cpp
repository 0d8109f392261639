// C ABI of 8-bit floating point and of the tokens of experts (declared in
// include/bakron.h). Host side only: argument checks and the choice of types;
// nothing here touches data.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "abi_checks.hpp"
#include "bakron.h"
#include "launch.hpp"
#include "tile_product.hpp"

namespace {

using namespace bk;

constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxRoutes = INT32_MAX - 4096;
inline int64_t blocks(int64_t n) { return (n + 127) / 128; }

// whether `batch` matrices `stride` elements apart can be addressed
inline bool batch_ok(const void* p, int64_t batch, int64_t stride, int64_t rows, int64_t cols,
                     int64_t ld, size_t es) {
  if (batch == 0 || rows == 0 || cols == 0) return true;
  return matrix_ok(p, rows, cols, ld, es) && stride >= 0 && stride <= (INT64_MAX / 8) / batch;
}
// whether rows x cols floats, any non-negative strides apart, can be addressed
inline bool strided_ok(const float* p, int64_t rows, int64_t srow, int64_t cols, int64_t scol) {
  if (rows == 0 || cols == 0) return true;
  return p && (uintptr_t)p % 4 == 0 && srow >= 0 && scol >= 0 && srow <= (INT64_MAX / 16) / rows &&
         scol <= (INT64_MAX / 16) / cols;
}
// An array as the bytes from its first element to its last; overlap of two.
struct Span {
  uintptr_t a, b;
};
inline Span span(const void* p, size_t es, int64_t n0, int64_t s0, int64_t n1 = 1, int64_t s1 = 0,
                 int64_t n2 = 1, int64_t s2 = 0) {
  if (!p || n0 <= 0 || n1 <= 0 || n2 <= 0) return {0, 0};
  const uintptr_t a = (uintptr_t)p;
  return {a, a + ((uintptr_t)((n0 - 1) * s0) + (uintptr_t)((n1 - 1) * s1) +
                  (uintptr_t)((n2 - 1) * s2) + 1) * es};
}
inline bool meets(const Span& x, std::initializer_list<Span> others) {
  for (const Span& y : others)
    if (x.a < y.b && y.a < x.b) return true;
  return false;
}

inline bool fp8_sizes_ok(int64_t T, int64_t R, int64_t experts, int64_t m, int64_t n) {
  if (T < 0 || R < 0 || m < 0 || n < 0 || experts < 1 || experts > kMaxExperts) return false;
  if (T > kMaxGroups || R > kMaxGroups || m > kMaxPlaneCols || n > kMaxPlaneCols) return false;
  return (m + 63) / 64 * (R / 64 + experts + 1) <= kMaxGroups &&
         (T + experts * m) * (n + 128) / 4096 < kMaxGroups;  // rows laid out, 16 bytes a thread
}
inline bool fp8_grad_sizes_ok(int t, int64_t R, int64_t experts, int64_t m, int64_t n) {
  return type_ok(t) && fp8_sizes_ok(0, R, experts, m, n) &&
         (n + 63) / 64 * (R / 64 + experts + 1) <= kMaxGroups &&
         R + plane_groups(R, m) + plane_groups(experts * m, n) <= kMaxGroups;
}

// a query's answer: room to align what the call needs, nothing for nothing
inline size_t with_slack(size_t b) { return b ? b + kAlign : 0; }
inline size_t fp8_query(int t, int64_t T, int64_t R, int64_t experts, int64_t m, int64_t n, bool aligned) {
  if (!type_ok(t) || !fp8_sizes_ok(T, R, experts, m, n)) return 0;
  return with_slack(matmul_fp8_bytes((int)type_size(t), T, R, experts, m, n, aligned));
}
inline size_t fp8_grad_query(int t, int64_t R, int64_t experts, int64_t m, int64_t n, bool aligned) {
  if (!fp8_grad_sizes_ok(t, R, experts, m, n)) return 0;
  return with_slack(matmul_fp8_grad_bytes((int)type_size(t), R, experts, m, n, aligned));
}

template <typename F> int by_type(int t, F f) {
  if (t == BAKRON_F32) return status(f((float*)nullptr));
  if (t == BAKRON_BF16) return status(f((BF16*)nullptr));
  return status(f((F16*)nullptr));
}

}  // namespace

extern "C" {

int bakron_quantize_fp8(int xtype, int64_t batch, int64_t rows, int64_t n, const void* X, int64_t ldx,
                        int64_t stride_x, int block_rows, uint8_t* Xq, int64_t ldq, int64_t stride_q,
                        float* s, int64_t s_row, int64_t s_block, int64_t stride_s, void* stream) {
  if (!type_ok(xtype) || batch < 0 || rows < 0 || n < 0 || (block_rows != 1 && block_rows != 128))
    return BAKRON_EINVAL;
  if (batch > 65535 || rows > kMaxGroups || n > INT64_MAX / 16) return BAKRON_EINVAL;
  if (batch == 0 || rows == 0 || n == 0) return BAKRON_OK;
  const size_t es = type_size(xtype);
  const int64_t na = block_rows == 1 ? rows : blocks(rows), nb = blocks(n);
  // a workgroup takes 16 rows of four blocks, or one block of 128 rows
  const int64_t down = block_rows == 1 ? (rows + 15) / 16 : na, across = block_rows == 1 ? (nb + 3) / 4 : nb;
  if (down > kMaxGroups / across) return BAKRON_EINVAL;
  if (!batch_ok(X, batch, stride_x, rows, n, ldx, es) || !batch_ok(Xq, batch, stride_q, rows, n, ldq, 1) ||
      !strided_ok(s, na, s_row, nb, s_block) || stride_s < 0 || stride_s > (INT64_MAX / 16) / batch)
    return BAKRON_EINVAL;
  // every output in a place of its own
  if (batch > 1 && (stride_q < (rows - 1) * ldq + n || stride_s < (na - 1) * s_row + (nb - 1) * s_block + 1))
    return BAKRON_EINVAL;
  if ((na > 1 && s_row < 1) || (nb > 1 && s_block < 1) ||
      (na > 1 && nb > 1 && s_row < (nb - 1) * s_block + 1 && s_block < (na - 1) * s_row + 1))
    return BAKRON_EINVAL;
  const Span x = span(X, es, batch, stride_x, rows, ldx, n, 1);
  const Span q = span(Xq, 1, batch, stride_q, rows, ldq, n, 1);
  const Span c = span(s, 4, batch, stride_s, na, s_row, nb, s_block);
  if (meets(q, {x, c}) || meets(c, {x})) return BAKRON_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_type(xtype, [&](auto* t) {
    return launch_quantize_fp8(batch, rows, n, (decltype(t))X, ldx, stride_x, block_rows, Xq, ldq,
                               stride_q, s, s_row, s_block, stride_s, st);
  });
}

size_t bakron_matmul_fp8_workspace_bytes(int ytype, int64_t T, int64_t R, int64_t experts, int64_t m,
                                         int64_t n) {
  return fp8_query(ytype, T, R, experts, m, n, false);
}
size_t bakron_matmul_fp8_aligned_workspace_bytes(int ytype, int64_t T, int64_t R, int64_t experts,
                                                 int64_t m, int64_t n) {
  return fp8_query(ytype, T, R, experts, m, n, true);
}

int bakron_matmul_fp8(int ytype, int64_t T, int64_t R, int64_t experts, int64_t m, int64_t n,
                      const uint8_t* Xq, int64_t ldx, const float* sx, int64_t sx_token,
                      int64_t sx_block, const uint8_t* Wq, int64_t ldw, int64_t stride_w,
                      const float* sw, int64_t ldsw, int64_t stride_sw, const int32_t* offsets,
                      const int32_t* order, int64_t per_token, void* Y, int64_t ldy, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!type_ok(ytype) || !fp8_sizes_ok(T, R, experts, m, n)) return BAKRON_EINVAL;
  if ((!offsets && experts != 1) || (!order && R != T) || per_token < 1 || per_token > kMaxRoutes ||
      T > kMaxRoutes / per_token)
    return BAKRON_EINVAL;
  if (R == 0 || m == 0) return BAKRON_OK;
  const size_t es = type_size(ytype);
  const int64_t nb = blocks(n), mb = blocks(m);
  const bool aligned = (T == 0 || fp8_rows_on_16(Xq, T > 1 ? ldx : 0, 0)) &&
                       fp8_weights_on_16(Wq, experts, stride_w, m, ldw);
  const size_t need = matmul_fp8_bytes((int)es, T, R, experts, m, n, aligned);
  if (need && (!workspace || (uintptr_t)workspace % kAlign || workspace_bytes < need))
    return BAKRON_EINVAL;
  if (!matrix_ok(Xq, T, n, ldx, 1) || !strided_ok(sx, T, sx_token, nb, sx_block) ||
      !batch_ok(Wq, experts, stride_w, m, n, ldw, 1) ||
      !batch_ok(sw, experts, stride_sw, mb, nb, ldsw, 4) || !matrix_ok(Y, R, m, ldy, es))
    return BAKRON_EINVAL;
  if ((uintptr_t)offsets % 4 || (uintptr_t)order % 4) return BAKRON_EINVAL;
  if (meets(span(Y, es, R, ldy, m, 1),
            {span(Xq, 1, T, ldx, n, 1), span(sx, 4, T, sx_token, nb, sx_block),
             span(Wq, 1, experts, stride_w, m, ldw, n, 1), span(sw, 4, experts, stride_sw, mb, ldsw, nb, 1),
             span(offsets, 4, experts + 1, 1), span(order, 4, R, 1)}))
    return BAKRON_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_type(ytype, [&](auto* t) {
    return launch_matmul_fp8(T, R, experts, m, n, Xq, ldx, sx, sx_token, sx_block, Wq, ldw, stride_w, sw,
                             ldsw, stride_sw, offsets, order, per_token, (decltype(t))Y, ldy, workspace,
                             st);
  });
}

size_t bakron_matmul_fp8_grad_workspace_bytes(int gtype, int64_t R, int64_t experts, int64_t m,
                                              int64_t n) {
  return fp8_grad_query(gtype, R, experts, m, n, false);
}
size_t bakron_matmul_fp8_grad_aligned_workspace_bytes(int gtype, int64_t R, int64_t experts, int64_t m,
                                                      int64_t n) {
  return fp8_grad_query(gtype, R, experts, m, n, true);
}

int bakron_matmul_fp8_grad(int gtype, int64_t R, int64_t experts, int64_t m, int64_t n, const void* G,
                           int64_t ldg, const uint8_t* Wq, int64_t ldw, int64_t stride_w,
                           const float* sw, int64_t ldsw, int64_t stride_sw, const int32_t* offsets,
                           void* dX, int64_t ldx, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!fp8_grad_sizes_ok(gtype, R, experts, m, n) || (!offsets && experts != 1)) return BAKRON_EINVAL;
  if (R == 0 || n == 0) return BAKRON_OK;
  const size_t es = type_size(gtype);
  const int64_t nb = blocks(n), mb = blocks(m);
  const size_t need = matmul_fp8_grad_bytes((int)es, R, experts, m, n,
                                            fp8_weights_on_16(Wq, experts, stride_w, m, ldw));
  if (need && (!workspace || (uintptr_t)workspace % kAlign || workspace_bytes < need))
    return BAKRON_EINVAL;
  if (!matrix_ok(G, R, m, ldg, es) || !batch_ok(Wq, experts, stride_w, m, n, ldw, 1) ||
      !batch_ok(sw, experts, stride_sw, mb, nb, ldsw, 4) || !matrix_ok(dX, R, n, ldx, es) ||
      (uintptr_t)offsets % 4)
    return BAKRON_EINVAL;
  if (meets(span(dX, es, R, ldx, n, 1),
            {span(G, es, R, ldg, m, 1), span(Wq, 1, experts, stride_w, m, ldw, n, 1),
             span(sw, 4, experts, stride_sw, mb, ldsw, nb, 1), span(offsets, 4, experts + 1, 1)}))
    return BAKRON_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_type(gtype, [&](auto* t) {
    return launch_matmul_fp8_grad(R, experts, m, n, (decltype(t))G, ldg, Wq, ldw, stride_w, sw, ldsw,
                                  stride_sw, offsets, (decltype(t))dX, ldx, workspace, st);
  });
}

size_t bakron_sort_tokens_workspace_bytes(int64_t T, int64_t k, int64_t experts) {
  if (T < 0 || k < 1 || T > kMaxRoutes / k || experts < 1 || experts > kMaxExperts) return 0;
  return with_slack(sort_tokens_bytes(T * k, experts));
}

int bakron_sort_tokens(int64_t T, int64_t k, int64_t experts, const int64_t* ids, int64_t ld,
                       int32_t* order, int32_t* slots, int32_t* offsets, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (T < 0 || k < 1 || T > kMaxRoutes / k || experts < 1 || experts > kMaxExperts) return BAKRON_EINVAL;
  const int64_t N = T * k;
  const size_t need = sort_tokens_bytes(N, experts);
  if (need && (!workspace || (uintptr_t)workspace % kAlign || workspace_bytes < need))
    return BAKRON_EINVAL;
  if (!matrix_ok(ids, T, k, ld, 8) || !matrix_ok(order, 1, N, N, 4) || !matrix_ok(slots, 1, N, N, 4) ||
      !matrix_ok(offsets, 1, experts + 1, experts + 1, 4))
    return BAKRON_EINVAL;
  const Span i = span(ids, 8, T, ld, k, 1), o = span(order, 4, N, 1), l = span(slots, 4, N, 1),
             f = span(offsets, 4, experts + 1, 1);
  if (meets(o, {i, l, f}) || meets(l, {i, f}) || meets(f, {i})) return BAKRON_EINVAL;
  return status(launch_sort_tokens(T, k, experts, ids, ld, order, slots, offsets, workspace,
                                   static_cast<hipStream_t>(stream)));
}

int bakron_gather_tokens(int xtype, int64_t T, int64_t n, const void* X, int64_t ldx,
                         int64_t per_token, int64_t R, const int32_t* order, void* Xs, int64_t ldxs,
                         void* stream) {
  if (!type_ok(xtype) || T < 0 || n < 0 || R < 0 || per_token < 1 || T > kMaxRoutes ||
      R > kMaxRoutes || (R + 3) / 4 > kMaxGroups)
    return BAKRON_EINVAL;
  if (R == 0 || n == 0) return BAKRON_OK;
  const size_t es = type_size(xtype);
  if (!matrix_ok(X, T, n, ldx, es) || !matrix_ok(Xs, R, n, ldxs, es) || !matrix_ok(order, 1, R, R, 4))
    return BAKRON_EINVAL;
  if (meets(span(Xs, es, R, ldxs, n, 1), {span(X, es, T, ldx, n, 1), span(order, 4, R, 1)}))
    return BAKRON_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_type(xtype, [&](auto* t) {
    return launch_gather_tokens(T, n, (decltype(t))X, ldx, per_token, R, order, (decltype(t))Xs, ldxs, st);
  });
}

int bakron_combine_tokens(int ytype, int64_t T, int64_t k, int64_t n, int64_t R, const void* Ys,
                          int64_t ldys, const int32_t* slots, const float* weights, void* Y,
                          int64_t ldy, void* stream) {
  if (!type_ok(ytype) || T < 0 || k < 0 || n < 0 || R < 0 || R > kMaxRoutes || T > kMaxGroups ||
      (k > 0 && T > kMaxRoutes / k) || n > INT64_MAX / 16)
    return BAKRON_EINVAL;
  if (T == 0 || n == 0) return BAKRON_OK;
  if ((n + 2047) / 2048 > kMaxGroups / T) return BAKRON_EINVAL;
  const size_t es = type_size(ytype);
  if (!matrix_ok(Ys, R, n, ldys, es) || !matrix_ok(slots, 1, T * k, T * k, 4) ||
      (weights && !matrix_ok(weights, 1, T * k, T * k, 4)) || !matrix_ok(Y, T, n, ldy, es))
    return BAKRON_EINVAL;
  if (meets(span(Y, es, T, ldy, n, 1), {span(Ys, es, R, ldys, n, 1), span(slots, 4, T * k, 1),
                                        span(weights, 4, T * k, 1)}))
    return BAKRON_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_type(ytype, [&](auto* t) {
    return launch_combine_tokens(T, k, n, R, (decltype(t))Ys, ldys, slots, weights, (decltype(t))Y, ldy,
                                 st);
  });
}

int bakron_combine_tokens_grad(int ytype, int64_t T, int64_t k, int64_t n, int64_t R, const void* G,
                               int64_t ldg, const void* Ys, int64_t ldys, const int32_t* slots,
                               const float* weights, void* dYs, int64_t lddys, float* dweights,
                               void* stream) {
  if (!type_ok(ytype) || T < 0 || k < 0 || n < 0 || R < 0 || R > kMaxRoutes || T > kMaxGroups ||
      (k > 0 && T > kMaxRoutes / k) || n > INT64_MAX / 16)
    return BAKRON_EINVAL;
  if (T == 0 || k == 0 || (!dYs && !dweights)) return BAKRON_OK;
  if ((k + 3) / 4 > kMaxGroups / T) return BAKRON_EINVAL;
  const size_t es = type_size(ytype);
  if (!matrix_ok(G, T, n, ldg, es) || (dweights && !matrix_ok(Ys, R, n, ldys, es)) ||
      !matrix_ok(slots, 1, T * k, T * k, 4) || (weights && !matrix_ok(weights, 1, T * k, T * k, 4)) ||
      (dYs && !matrix_ok(dYs, R, n, lddys, es)) || (uintptr_t)dweights % 4)
    return BAKRON_EINVAL;
  const Span g = span(G, es, T, ldg, n, 1), y = dweights ? span(Ys, es, R, ldys, n, 1) : Span{0, 0},
             l = span(slots, 4, T * k, 1), w = span(weights, 4, T * k, 1),
             d = span(dYs, es, R, lddys, n, 1), dw = span(dweights, 4, T * k, 1);
  if (meets(d, {g, y, l, w, dw}) || meets(dw, {g, y, l, w})) return BAKRON_EINVAL;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return by_type(ytype, [&](auto* t) {
    return launch_combine_tokens_grad(T, k, n, R, (decltype(t))G, ldg, (decltype(t))Ys, ldys, slots,
                                      weights, (decltype(t))dYs, lddys, dweights, st);
  });
}

}  // extern "C"
