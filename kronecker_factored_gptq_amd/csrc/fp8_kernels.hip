// 8-bit floating point on gfx950: matrices quantised to e4m3 codes with a float32
// scale for each block of 1 x 128 or 128 x 128, and the product of such tokens with
// such weights, for one layer or for groups of tokens with weights of their own.
#include "fp8_product.hpp"
#include "launch.hpp"

namespace bk {

// ---------------------------------------------------------------------------
// Blocks to e4m3: s = max |x| / 448 (448 = the largest code), at least 2^-126, 1 for an
// all-zero block; code = x / s rounded to nearest even, the division correctly
// rounded. The maximum is taken over the bits of |x|, in which a NaN is larger than
// infinity: a block with either gets it as its scale.
// ---------------------------------------------------------------------------
__device__ inline float block_scale(unsigned top) {
  if (top == 0) return 1.0f;
  const float s = __uint_as_float(top) / 448.0f;
  return s < 0x1p-126f ? 0x1p-126f : s;
}
template <typename X> __device__ inline unsigned top8(const Eight<X>& t) {
  unsigned top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned a = __float_as_uint(to_f32(t.v[e])) & 0x7fffffffu;
    top = a > top ? a : top;
  }
  return top;
}
__device__ inline unsigned max_of_16(unsigned top) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const unsigned u = __shfl_xor(top, o, 64);
    top = u > top ? u : top;
  }
  return top;
}
// eight codes of a row from column c on
template <typename X>
__device__ inline void store_codes(char* row, int64_t c, int64_t n, const Eight<X>& t, float s,
                                   bool vec) {
  int w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = to_f32(t.v[4 * i]) / s, b = to_f32(t.v[4 * i + 1]) / s;
    const float d = to_f32(t.v[4 * i + 2]) / s, e = to_f32(t.v[4 * i + 3]) / s;
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(d, e, w[i], true);
  }
  if (vec && c + 8 <= n) {
    *(int2*)(row + c) = int2{w[0], w[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = (char)(w[e / 4] >> 8 * (e % 4));
  }
}

// Blocks of 1 x 128: 16 lanes to kRun neighbouring blocks of a row, neighbouring groups of
// lanes on neighbouring rows, so that their scales are stored side by side where the
// scales' rows are. Bound by memory.
constexpr int kRun = 4;
template <typename X>
__global__ __launch_bounds__(256) void quantize_rows_kernel(
    int64_t rows, int64_t n, int64_t runs, const X* __restrict__ x, int64_t ldx, int64_t sX,
    char* __restrict__ q, int64_t ldq, int64_t sQ, float* __restrict__ s, int64_t srow,
    int64_t sblock, int64_t sS, bool vec, bool vecq) {
  const int64_t at = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (at >= rows * runs) return;  // whole groups of 16 lanes
  const int l = threadIdx.x & 15;
  const int64_t run = at / rows, r = at - run * rows;
  x += blockIdx.y * sX + r * ldx;
  q += blockIdx.y * sQ + r * ldq;
  s += blockIdx.y * sS + r * srow;
  Eight<X> t[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) t[i] = load8(x, (run * kRun + i) * kBlock + 8 * l, n, vec);
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int64_t b = run * kRun + i;
    if (b * kBlock >= n) break;
    const float f = block_scale(max_of_16(top8(t[i])));
    if (l == 0) s[b * sblock] = f;
    store_codes(q, b * kBlock + 8 * l, n, t[i], f, vecq);
  }
}

// Blocks of 128 x 128, a workgroup each, held in registers between the maximum and the codes.
template <typename X>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(
    int64_t rows, int64_t n, unsigned across, const X* __restrict__ x, int64_t ldx, int64_t sX,
    char* __restrict__ q, int64_t ldq, int64_t sQ, float* __restrict__ s, int64_t srow,
    int64_t sblock, int64_t sS, bool vec, bool vecq) {
  __shared__ unsigned red[4];
  const int64_t a = blockIdx.x / across, b = blockIdx.x - a * across;
  const int64_t c = b * kBlock + 8 * (threadIdx.x & 15);
  x += blockIdx.y * sX;
  q += blockIdx.y * sQ;
  Eight<X> t[8];
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = a * kBlock + 16 * i + (threadIdx.x >> 4);
    t[i] = load8(x + (r < rows ? r : rows - 1) * ldx, c, n, vec);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned u = top8(t[i]);  // rows past the last count as it, columns past n as zero
    top = u > top ? u : top;
  }
  const float f = block_scale(max_of_256(top, red));
  if (threadIdx.x == 0) s[blockIdx.y * sS + a * srow + b * sblock] = f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = a * kBlock + 16 * i + (threadIdx.x >> 4);
    if (r < rows) store_codes(q + r * ldq, c, n, t[i], f, vecq);
  }
}

template <typename X>
hipError_t launch_quantize_fp8(int64_t batch, int64_t rows, int64_t n, const X* x, int64_t ldx,
                               int64_t sX, int block_rows, uint8_t* q, int64_t ldq, int64_t sQ,
                               float* s, int64_t srow, int64_t sblock, int64_t sS,
                               hipStream_t st) {
  if (batch <= 0 || rows <= 0 || n <= 0) return hipSuccess;
  const bool vec = load8_ok(x, ldx) && load8_ok(x, sX), vecq = ((uintptr_t)q | ldq | sQ) % 8 == 0;
  const int64_t nb = (n + kBlock - 1) / kBlock;
  if (block_rows == 1) {
    const int64_t runs = (nb + kRun - 1) / kRun;
    hipLaunchKernelGGL(quantize_rows_kernel<X>,
                       dim3((unsigned)((rows * runs + 15) / 16), (unsigned)batch), dim3(256), 0, st,
                       rows, n, runs, x, ldx, sX, (char*)q, ldq, sQ, s, srow, sblock, sS, vec, vecq);
  } else {
    const int64_t na = (rows + kBlock - 1) / kBlock;
    hipLaunchKernelGGL(quantize_blocks_kernel<X>, dim3((unsigned)(na * nb), (unsigned)batch),
                       dim3(256), 0, st, rows, n, (unsigned)nb, x, ldx, sX, (char*)q, ldq, sQ, s,
                       srow, sblock, sS, vec, vecq);
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Y[r][i] = sum over blocks b of k of sx[t][b] sw[i / 128][b] sum_{j in b} Xq[t][j] Wq[i][j],
// t the token of row r, W its group's. Tiles of 64 channels x 64 rows, a block of k a
// step, read to registers while the step before is computed.
// ---------------------------------------------------------------------------
template <class Mul, typename O>
__global__ __launch_bounds__(256) void matmul_fp8_kernel(Groups groups, Fp8Tokens X, Fp8Weights W,
                                                         int64_t n, O* __restrict__ Y, int64_t ldy) {
  constexpr int B = 64, F = 2;  // four waves of 32 x 32
  __shared__ __attribute__((aligned(16))) char lds[2 * 2 * B * kBlock];
  const unsigned nr = (unsigned)((W.m + B - 1) / B);
  const unsigned nc = (unsigned)groups.tiles<B>();
  if (blockIdx.x >= nr * nc) return;
  int tr, tc;
  tile_of(blockIdx.x, nr, nc, tr, tc);
  int64_t group, c0, cols;
  if (!groups.tile<B>(tc, group, c0, cols)) return;
  const int64_t r0 = (int64_t)tr * B;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r16 = lane & 15, q = lane >> 4;
  const int wr = (wave >> 1) * 32, wc = (wave & 1) * 32;
  const char* w = W.p + group * W.stride;
  const float* sw = W.s + group * W.strides + r0 / kBlock * W.lds;
  const char *pw[2], *px[2];  // this thread's chunks: of rows tid / 8 and 32 further
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t e = u * 32 + (tid >> 3), i = r0 + e;
    pw[u] = w + (i < W.m ? i : W.m - 1) * W.ld;
    const int64_t t = X.token(c0 + (e < cols ? e : cols - 1));
    px[u] = t < 0 ? nullptr : X.p + t * X.ld;
  }
  const float* ps[F];
#pragma unroll
  for (int j = 0; j < F; ++j) {
    const int64_t e = wc + j * 16 + r16, t = X.token(c0 + (e < cols ? e : cols - 1));
    ps[j] = t < 0 ? nullptr : X.s + t * X.st;
  }
  f32x4 acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  auto at = [&](int row, int chunk) { return row * kBlock + (chunk ^ ((row >> 1) & 7)) * 16; };
  const int64_t nb = (n + kBlock - 1) / kBlock;
  v4i vw[2], vx[2];
  auto read = [&](int64_t b) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      vw[u] = load_any<1>(pw[u], b * kBlock + (tid & 7) * 16, n);
      vx[u] = px[u] ? load_any<1>(px[u], b * kBlock + (tid & 7) * 16, n) : v4i{0, 0, 0, 0};
    }
  };
  auto write = [&](int slot) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      *(v4i*)(lds + slot * 2 * B * kBlock + at(u * 32 + (tid >> 3), tid & 7)) = vw[u];
      *(v4i*)(lds + (slot * 2 + 1) * B * kBlock + at(u * 32 + (tid >> 3), tid & 7)) = vx[u];
    }
  };
  if (nb > 0) {
    read(0);
    write(0);
  }
  __syncthreads();
  for (int64_t b = 0; b < nb; ++b) {
    if (b + 1 < nb) read(b + 1);
    const char *lw = lds + (b & 1) * 2 * B * kBlock, *lx = lw + B * kBlock;
    const float fw = sw[b];
    v4i x[F][2], y[F][2];
    float f[F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[i][h] = *(const v4i*)(lw + at(wr + i * 16 + r16, h * 4 + q));
        y[i][h] = *(const v4i*)(lx + at(wc + i * 16 + r16, h * 4 + q));
      }
#pragma unroll
    for (int j = 0; j < F; ++j) f[j] = ps[j] ? ps[j][b * X.sb] * fw : 0.0f;
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        const f32x4 p = Mul::block(x[i][0], x[i][1], y[j][0], y[j][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], f[j], acc[i][j][e]);
      }
    if (b + 1 < nb) write((b + 1) & 1);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < F; ++j)
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t c = wc + j * 16 + r16, r = r0 + wr + i * 16 + 4 * q + e;
        if (c < cols && r < W.m) Y[(c0 + c) * ldy + r] = from_f32<O>(acc[i][j][e]);
      }
}

size_t matmul_fp8_bytes(int, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

template <typename O>
hipError_t launch_matmul_fp8(int64_t T, int64_t R, int64_t experts, int64_t m, int64_t n,
                             const uint8_t* Xq, int64_t ldx, const float* sx, int64_t sx_token,
                             int64_t sx_block, const uint8_t* Wq, int64_t ldw, int64_t stride_w,
                             const float* sw, int64_t ldsw, int64_t stride_sw,
                             const int32_t* offsets, const int32_t* order, int64_t per_token, O* Y,
                             int64_t ldy, void*, hipStream_t s) {
  if (R <= 0 || m <= 0) return hipSuccess;
  const Groups groups = {offsets, experts, R};
  const Fp8Tokens X = {(const char*)Xq, ldx, T, sx, sx_token, sx_block, order, per_token};
  const Fp8Weights W = {(const char*)Wq, ldw, stride_w, m, sw, ldsw, stride_sw};
  typedef typename std::conditional<sizeof(O) == 4, MulFP8Exact, MulFP8>::type Mul;
  const int64_t tiles = (m + 63) / 64 * groups.most(64);
  hipLaunchKernelGGL((matmul_fp8_kernel<Mul, O>), dim3((unsigned)tiles), dim3(256), 0, s, groups, X,
                     W, n, Y, ldy);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// dX[r][j] = sum_i G[r][i] sw[i / 128][j / 128] Wq[i][j]: a thread to an output, its sum
// over the channels in order.
// ---------------------------------------------------------------------------
template <typename G>
__global__ __launch_bounds__(256) void matmul_fp8_grad_kernel(Groups groups, int64_t m, int64_t n,
                                                              const G* __restrict__ g, int64_t ldg,
                                                              Fp8Weights W, G* __restrict__ dX,
                                                              int64_t ldx) {
  const int64_t per = (n + 255) / 256, r = blockIdx.x / per;
  const int64_t j = (blockIdx.x - r * per) * 256 + threadIdx.x;
  int64_t e = 0, first = 0;
  for (; e < groups.count; ++e) {
    const int64_t a = groups.offset(e);
    first = a > first ? a : first;
    if (r >= first && r < groups.offset(e + 1)) break;
  }
  if (e == groups.count) return;
  if (j >= n) return;
  const unsigned char* w = (const unsigned char*)W.p + e * W.stride + j;
  const float* sw = W.s + e * W.strides + j / kBlock;
  float sum = 0.0f;
  for (int64_t i0 = 0; i0 < m; i0 += kBlock) {
    float part = 0.0f;
    for (int64_t i = i0; i < i0 + kBlock && i < m; ++i)
      part = __builtin_fmaf(to_f32(g[r * ldg + i]),
                            __builtin_amdgcn_cvt_f32_fp8((int)w[i * W.ld], 0), part);
    sum = __builtin_fmaf(part, sw[i0 / kBlock * W.lds], sum);
  }
  dX[r * ldx + j] = from_f32<G>(sum);
}

size_t matmul_fp8_grad_bytes(int, int64_t, int64_t, int64_t, int64_t) { return 0; }

template <typename G>
hipError_t launch_matmul_fp8_grad(int64_t R, int64_t experts, int64_t m, int64_t n, const G* g,
                                  int64_t ldg, const uint8_t* Wq, int64_t ldw, int64_t stride_w,
                                  const float* sw, int64_t ldsw, int64_t stride_sw,
                                  const int32_t* offsets, G* dX, int64_t ldx, void*,
                                  hipStream_t s) {
  if (R <= 0 || n <= 0) return hipSuccess;
  const Groups groups = {offsets, experts, R};
  const Fp8Weights W = {(const char*)Wq, ldw, stride_w, m, sw, ldsw, stride_sw};
  hipLaunchKernelGGL(matmul_fp8_grad_kernel<G>, dim3((unsigned)(R * ((n + 255) / 256))), dim3(256),
                     0, s, groups, m, n, g, ldg, W, dX, ldx);
  return hipGetLastError();
}

#define BK_INST(X)                                                                               \
  template hipError_t launch_quantize_fp8<X>(int64_t, int64_t, int64_t, const X*, int64_t,       \
                                             int64_t, int, uint8_t*, int64_t, int64_t, float*,   \
                                             int64_t, int64_t, int64_t, hipStream_t);            \
  template hipError_t launch_matmul_fp8<X>(                                                      \
      int64_t, int64_t, int64_t, int64_t, int64_t, const uint8_t*, int64_t, const float*,        \
      int64_t, int64_t, const uint8_t*, int64_t, int64_t, const float*, int64_t, int64_t,        \
      const int32_t*, const int32_t*, int64_t, X*, int64_t, void*, hipStream_t);                 \
  template hipError_t launch_matmul_fp8_grad<X>(                                                 \
      int64_t, int64_t, int64_t, int64_t, const X*, int64_t, const uint8_t*, int64_t, int64_t,   \
      const float*, int64_t, int64_t, const int32_t*, X*, int64_t, void*, hipStream_t);
BK_INST(float)
BK_INST(BF16)
BK_INST(F16)
#undef BK_INST

}  // namespace bk
