// The product of tile_product.hpp for few columns (single tokens to a few
// dozen), bound by reading R once:
//   D[r][c] = sum_k R[r][k] C[c][k],  c < 16 NT.
//
// A workgroup of 8 waves takes 16 RT rows of R and all columns; its waves
// divide k between them in blocks of 64 U bytes, so that one workgroup has all
// of its rows' bytes in flight at once, straight from memory to registers (a
// lane's 16 bytes are its operand: LDS would add a trip). The next block is on
// its way while one is multiplied (U = 4 and one block ahead: 14336 x 4096 int8,
// one column, 13.5 us; U = 8 without: 14.4). C comes from the caches, as often as
// there are workgroups, which is what bounds more than a few columns. The waves'
// sums meet in LDS.
#pragma once

#include "tile_product.hpp"

namespace bk {

template <class M, int RT, int NT, int U, bool ANY>
struct SkinnyProduct {
  typedef typename M::acc_t acc_t;
  static constexpr int kWaves = 8, kThreads = 512;
  static constexpr int kRows = 16 * RT, kCols = 16 * NT;
  static constexpr int kTiles = RT * NT;
  static constexpr int kLds = kWaves * kTiles * 1024;
  static_assert(kTiles <= kWaves, "a wave to each tile");

  __device__ static inline v4i load(const char* row, int64_t k, int64_t kbytes) {
    if (ANY) return load_any<M::kElem>(row, k, kbytes);
    return k < kbytes ? *(const v4i*)(row + k) : v4i{0, 0, 0, 0};
  }

  // This wave's 16 x 16 tile, if it has one: its first row and column, with the
  // lane's first element's.
  __device__ static inline bool has_tile() { return (int)(threadIdx.x >> 6) < kTiles; }
  __device__ static inline int tile_r() {
    return (threadIdx.x >> 6) / NT * 16 + 4 * ((threadIdx.x & 63) >> 4);
  }
  __device__ static inline int tile_c() { return (threadIdx.x >> 6) % NT * 16 + (threadIdx.x & 15); }

  // f(sums) for every 16 x 16 tile, by one wave each, a lane's sums
  // D[tile_r() + e][tile_c()]. Rows past the operands' last are their last's.
  template <typename F>
  __device__ static inline void run(const TileOperand& R, const TileOperand& C, int64_t kbytes,
                                    int64_t r0, char* lds, F f) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const char* pr[RT];
    const char* pc[NT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int64_t r = r0 + 16 * i + r16;
      pr[i] = R.p + (r < R.rows ? r : R.rows - 1) * R.ld;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t c = 16 * j + r16;
      pc[j] = C.p + (c < C.rows ? c : C.rows - 1) * C.ld;
    }
    acc_t acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = acc_t{0, 0, 0, 0};
    struct Block {
      v4i a[RT][U], b[NT][U];
    };
    auto read = [&](Block& t, int64_t k) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < RT; ++i) t.a[i][u] = load(pr[i], k + 64 * u + 16 * q, kbytes);
#pragma unroll
        for (int j = 0; j < NT; ++j) t.b[j][u] = load(pc[j], k + 64 * u + 16 * q, kbytes);
      }
    };
    auto multiply = [&](const Block& t) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[i][j] = M::mma(t.a[i][u], t.b[j][u], acc[i][j]);
    };
    constexpr int64_t kStride = kWaves * 64 * U;
    int64_t k = (int64_t)wave * 64 * U;
    if (k < kbytes) {
      Block x, y;
      read(x, k);
      while (k + kStride < kbytes) {
        read(y, k + kStride);
        multiply(x);
        k += kStride;
        if (k + kStride >= kbytes) {
          x = y;
          break;
        }
        read(x, k + kStride);
        multiply(y);
        k += kStride;
      }
      multiply(x);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        ((acc_t*)lds)[(wave * kTiles + i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    if (wave < kTiles) {
      acc_t sum = ((acc_t*)lds)[wave * 64 + lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += ((acc_t*)lds)[(w * kTiles + wave) * 64 + lane];
      f(sum);
    }
  }
};

}  // namespace bk
