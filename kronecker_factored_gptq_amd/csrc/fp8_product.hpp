// What the products with block scales share: the matrix instructions of one block
// of k, and where a group (an expert) of sorted rows lies.
#pragma once

#include "tile_product.hpp"

namespace bk {

constexpr int kBlock = 128;  // k (and rows of weights) under one scale

// A product of one step (128 bytes of k; a lane holds two chunks of 16 of each
// operand's row), from zero, so that the block's scale can be applied before it is
// added to the rest. Both operands have the same k in the same place, so the order of k
// inside does not matter.
//
// e4m3 codes on their own instruction: groups of eight neighbouring products are
// added after each was cut to 2^-13 of the largest of the eight, the groups in
// float32 (measured by planting one large and one small product; the older instruction of
// 32 k does the same at half the rate). Sums of Gaussian codes are off by 1.5e-5 in the
// 2-norm, a sixteenth of a float16's rounding and less of a bfloat16's.
struct MulFP8 {
  static constexpr bool kTransposed = false;
  static constexpr int kPlanes = 1;
  __device__ static inline f32x4 block(v4i a0, v4i a1, v4i b0, v4i b1) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7),
        __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7), f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0,
        0);
  }
};
// e4m3 codes as float16 (exact: 4 of its 11 bits, 2^-9 to 448) on the float16 instructions,
// whose products are exact and whose sums are float32: for float32 results, which the
// other would leave at 1.5e-5, and for few rows, which wait for memory. Half its rate.
__device__ inline v8h fp8_to_f16(int lo, int hi) {
  typedef _Float16 v2h __attribute__((ext_vector_type(2)));
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return v8h{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ inline v8bf fp8_to_bf16(int lo, int hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
struct MulFP8Exact {
  static constexpr bool kTransposed = false;
  static constexpr int kPlanes = 1;
  __device__ static inline f32x4 block(v4i a0, v4i a1, v4i b0, v4i b1) {
    f32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(fp8_to_f16(a0[i], a0[i + 1]),
                                                 fp8_to_f16(b0[i], b0[i + 1]), c, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(fp8_to_f16(a1[i], a1[i + 1]),
                                                 fp8_to_f16(b1[i], b1[i + 1]), c, 0, 0, 0);
    return c;
  }
};

// e4m3 codes, made 16-bit where they are used, times 16-bit values: 64 k, eight neighbouring
// ones to a lane and instruction. Exact in either type (e4m3 has 4 bits, and its exponents lie
// in both types' normal range). PLANES: of the values (three bfloat16 hold a float32).
template <class M, int PLANES>
struct MulWide {
  static constexpr bool kTransposed = true;
  static constexpr int kPlanes = PLANES;
  __device__ static inline void widen(v4i codes, v4i& a, v4i& b) {
    if (std::is_same<M, MmaF16>::value) {
      a = __builtin_bit_cast(v4i, fp8_to_f16(codes[0], codes[1]));
      b = __builtin_bit_cast(v4i, fp8_to_f16(codes[2], codes[3]));
    } else {
      a = __builtin_bit_cast(v4i, fp8_to_bf16(codes[0], codes[1]));
      b = __builtin_bit_cast(v4i, fp8_to_bf16(codes[2], codes[3]));
    }
  }
  __device__ static inline f32x4 first(v4i a, v4i b) { return M::mma(a, b, f32x4{0, 0, 0, 0}); }
  __device__ static inline f32x4 second(v4i a, v4i b, f32x4 c) { return M::mma(a, b, c); }
  __device__ static inline f32x4 block(v4i a0, v4i a1, v4i b0, v4i b1) {
    return second(a1, b1, first(a0, b0));
  }
};

// Groups of sorted rows: group e holds rows [offsets[e], offsets[e + 1]) of R; without
// offsets the one group of all rows. Offsets are held inside [0, R], and one below an earlier
// one counts as it, so that whatever they hold the groups lie apart and inside the rows.
struct Groups {
  const int* offsets;
  int64_t count, R;
  __device__ inline int offset(int64_t e) const {
    const int64_t a = offsets ? offsets[e] : e == 0 ? 0 : R;
    return (int)(a < 0 ? 0 : a > R ? R : a);
  }
  __device__ static inline int lane_of(int x, int l) { return __builtin_amdgcn_readlane(x, l); }
  // Groups e0 to e0 + 63, one to a lane: first rows and numbers of rows (0 past the last group).
  // `before`: the largest offset before e0 (uniform), which is brought up to date.
  __device__ inline void ranges(int64_t e0, int& before, int& first, int& rows) const {
    const int lane = threadIdx.x & 63;
    const bool has = e0 + lane < count;
    int a = has ? offset(e0 + lane) : 0, b = has ? offset(e0 + lane + 1) : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(a, o, 64);
      a = lane >= o && u > a ? u : a;
    }
    a = a > before ? a : before;
    first = a;
    rows = has && b > a ? b - a : 0;
    before = lane_of(a, 63);
  }
  // The group that tile number `at` belongs to when every group is cut into tiles of B
  // rows: its number (uniform over the wave), the tile's first row and the rows from there to
  // its group's end. Every wave looks through all groups, 64 at a time. False past the last
  // tile.
  template <int B>
  __device__ inline bool tile(int64_t at, int64_t& group, int64_t& first, int64_t& rows) const {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int64_t e0 = 0; e0 < count; e0 += 64) {
      int a, n;
      ranges(e0, before, a, n);
      const int tiles = (n + B - 1) / B;
      int sum = tiles;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(sum, o, 64);
        sum += lane >= o ? u : 0;
      }
      const uint64_t past = __ballot((int64_t)sum > at);
      if (past) {
        const int l = __builtin_ctzll(past);
        group = e0 + l;
        const int skip = ((int)at - (lane_of(sum, l) - lane_of(tiles, l))) * B;
        first = lane_of(a, l) + skip;
        rows = lane_of(n, l) - skip;
        return true;
      }
      at -= lane_of(sum, 63);
    }
    return false;
  }
  // the number of all tiles
  template <int B> __device__ inline int64_t tiles() const {
    int64_t all = 0;
    int before = 0;
    for (int64_t e0 = 0; e0 < count; e0 += 64) {
      int a, n;
      ranges(e0, before, a, n);
      int sum = (n + B - 1) / B;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
      all += lane_of(sum, 0);
    }
    return all;
  }
  // the most tiles of B rows that any offsets can give
  int64_t most(int64_t B) const {
    if (!offsets) return (R + B - 1) / B;
    return R / B + (count < R ? count : R);
  }
};

// The operands of bakron_matmul_fp8.
struct Fp8Tokens {  // tokens' codes and scales; row r of a product is token `order[r] / per_token`
  const char* p;
  int64_t ld, T;
  const float* s;
  int64_t st, sb;
  const int* order;
  int64_t per;
  // the token of sorted row r, -1 if none
  __device__ inline int64_t token(int64_t r) const {
    if (!order) return r;
    const int64_t p = order[r];
    return p >= 0 && p < per * T ? p / per : -1;
  }
};
struct Fp8Weights {
  const char* p;
  int64_t ld, stride, m;
  const float* s;
  int64_t lds, strides;
};

}  // namespace bk
