// Operands laid out as 16-bit planes, and the tiled products of them
// (tile_product.hpp): the products whose operands are not already k-contiguous
// rows of one 16-bit type.
#include "launch.hpp"
#include "tile_product.hpp"

namespace bk {

struct I8 {
  signed char v;
};
__device__ inline float to_f32(I8 x) { return (float)x.v; }

// Eight columns of one row per thread, one 16-byte store per plane.
template <typename X, int KIND>
__global__ __launch_bounds__(256) void planes_kernel(int64_t rows, int64_t cols,
                                                     const X* __restrict__ x, int64_t ldx,
                                                     const float* __restrict__ cs, Planes out) {
  constexpr int NP = kPlanes[KIND];
  const int64_t per = out.ld / 16;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= rows * per) return;
  const int64_t r = at / per, c0 = (at - r * per) * 8;
  unsigned short w[NP][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t c = c0 + e;
    float v = 0.0f;
    if (c < cols) v = to_f32(x[r * ldx + c]) * (cs ? cs[c] : 1.0f);
    unsigned short t[NP];
    split16<KIND>(v, t);
#pragma unroll
    for (int p = 0; p < NP; ++p) w[p][e] = t[p];
  }
#pragma unroll
  for (int p = 0; p < NP; ++p)
    *(v4i*)(out.w + p * out.plane + r * out.ld + c0 * 2) = __builtin_bit_cast(v4i, w[p]);
}

// The transpose by tiles of 64 x 64 through LDS, both sides in full lines.
template <typename X, int KIND>
__global__ __launch_bounds__(256) void planes_t_kernel(int64_t rows, int64_t cols,
                                                       const X* __restrict__ x, int64_t ldx,
                                                       const float* __restrict__ rs, Planes out) {
  constexpr int NP = kPlanes[KIND];
  __shared__ float tile[64][65];
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int64_t r = r0 + u * 4 + ty, c = c0 + tx;
    float v = r < rows && c < cols ? to_f32(x[r * ldx + c]) : 0.0f;
    if (rs && r < rows) v = rs[r] == 0.0f ? 0.0f : v * rs[r];
    tile[u * 4 + ty][tx] = v;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e = u * 256 + threadIdx.x, c = e >> 3, k = (e & 7) * 8;
    if (c0 + c >= cols) continue;
    unsigned short w[NP][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      unsigned short t[NP];
      split16<KIND>(tile[k + i][c], t);
#pragma unroll
      for (int p = 0; p < NP; ++p) w[p][i] = t[p];
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
      *(v4i*)(out.w + p * out.plane + (c0 + c) * out.ld + (r0 + k) * 2) =
          __builtin_bit_cast(v4i, w[p]);
  }
}

template <class M, typename O, int BR, int BC, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) void plane_product_kernel(
    TileOperand R, TileOperand C, int64_t kbytes, PlanePairs pairs, PlaneEpilogue ep,
    O* __restrict__ Y, int64_t ldy, bool vec, unsigned nr, unsigned nc) {
  typedef TileProduct<M, BR, BC, WR, WC> TP;
  extern __shared__ char lds[];
  int tr, tc;
  tile_of(blockIdx.x, nr, nc, tr, tc);
  const int64_t r0 = (int64_t)tr * BR, c0 = (int64_t)tc * BC;
  TP tp;
  tp.zero();
  tp.run(R, C, kbytes, pairs, r0, c0, lds);
  const int lane = threadIdx.x & 63;
  const int64_t rb = r0 + tp.wave_r() + 4 * (lane >> 4), cb = c0 + tp.wave_c() + (lane & 15);
  const float all = (ep.alpha ? *ep.alpha : 1.0f) * ep.beta;
  float sr[TP::FR][4], sc[TP::FC];
#pragma unroll
  for (int i = 0; i < TP::FR; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sr[i][e] = all;
  if (ep.row_scale) {
#pragma unroll
    for (int i = 0; i < TP::FR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t r = rb + i * 16 + e;
        sr[i][e] = ep.row_scale[r < R.rows ? r : R.rows - 1] * all;
      }
  }
#pragma unroll
  for (int j = 0; j < TP::FC; ++j) {
    const int64_t c = cb + j * 16;
    sc[j] = ep.col_scale ? ep.col_scale[c < C.rows ? c : C.rows - 1] : 1.0f;
  }
  if (ep.prev) {  // rows of whole groups of four: its columns are padded
#pragma unroll
    for (int j = 0; j < TP::FC; ++j) {
      const int64_t c = cb + j * 16;
      if (c >= C.rows) continue;
#pragma unroll
      for (int i = 0; i < TP::FR; ++i)
        if (rb + i * 16 < R.rows)
          tp.acc[i][j] += *(const f32x4*)(ep.prev + c * ep.ldprev + rb + i * 16);
    }
  }
  store_tile(tp, r0, c0, R.rows, C.rows, Y, ldy, vec,
             [&](float a, int i, int j, int e) { return a * sr[i][e] * sc[j]; });
}

template <class M, typename O, int BR, int BC, int WR, int WC>
static hipError_t start_plane_product(const TileOperand& R, const TileOperand& C, int64_t kbytes,
                                      const PlanePairs& pairs, const PlaneEpilogue& ep, O* Y,
                                      int64_t ldy, hipStream_t s) {
  typedef TileProduct<M, BR, BC, WR, WC> TP;
  auto* k = plane_product_kernel<M, O, BR, BC, WR, WC>;
  if (TP::kLds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, TP::kLds);
    if (e != hipSuccess) return e;
  }
  const int64_t nr = (R.rows + BR - 1) / BR, nc = (C.rows + BC - 1) / BC;
  hipLaunchKernelGGL(k, dim3((unsigned)(nr * nc)), dim3(TP::kThreads), TP::kLds, s, R, C, kbytes,
                     pairs, ep, Y, ldy, vec4_ok(Y, ldy), (unsigned)nr, (unsigned)nc);
  return hipGetLastError();
}

template <typename O, bool F16P>
hipError_t launch_plane_product(int64_t M, int64_t N, int64_t K, Planes R, Planes C,
                                const PlanePairs& pairs, const PlaneEpilogue& ep, O* Y,
                                int64_t ldy, hipStream_t s) {
  typedef typename std::conditional<F16P, MmaF16, MmaBF16>::type Mma;
  if (M <= 0 || N <= 0) return hipSuccess;
  const TileOperand r = {R.w, R.ld, R.plane, M}, c = {C.w, C.ld, C.plane, N};
  const int64_t kbytes = (K + 7) / 8 * 16;  // whole 16-byte chunks: the planes' padding is zero
  const int64_t big = ((M + 255) / 256) * ((N + 255) / 256);
  if (big >= 192)
    return start_plane_product<Mma, O, 256, 256, 2, 4>(r, c, kbytes, pairs, ep, Y, ldy, s);
  return start_plane_product<Mma, O, 128, 128, 2, 2>(r, c, kbytes, pairs, ep, Y, ldy, s);
}

template <typename X, int KIND>
hipError_t launch_planes(int64_t rows, int64_t cols, const X* x, int64_t ldx,
                         const float* col_scale, Planes out, hipStream_t s) {
  const int64_t n = rows * (out.ld / 16);
  if (n <= 0) return hipSuccess;
  hipLaunchKernelGGL((planes_kernel<X, KIND>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                     rows, cols, x, ldx, col_scale, out);
  return hipGetLastError();
}

template <typename X, int KIND>
hipError_t launch_planes_t(int64_t rows, int64_t cols, const X* x, int64_t ldx,
                           const float* row_scale, Planes out, hipStream_t s) {
  if (rows <= 0 || cols <= 0) return hipSuccess;
  hipLaunchKernelGGL((planes_t_kernel<X, KIND>),
                     dim3((unsigned)((rows + 63) / 64), (unsigned)((cols + 63) / 64)), dim3(256), 0,
                     s, rows, cols, x, ldx, row_scale, out);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Input gradient of the 8-bit product: dX[t][j] = channel[j] sum_i (G[t][i]
// sv[i]) Vq[i][j]. The codes are exact in bfloat16, so the product runs on
// the bfloat16 instructions with Vq's transpose as one plane and G sv as as
// many planes as its type has bits: one for bfloat16 (its rounding is as large
// as the output's own), two for float16 (2^-16 against the output's 2^-11), three
// for float32 (all 24 bits).
// ---------------------------------------------------------------------------
template <typename G> struct GradSplit;
template <> struct GradSplit<float> { static constexpr int kind = kBF16x3; };
template <> struct GradSplit<BF16> { static constexpr int kind = kBF16x1; };
template <> struct GradSplit<F16> { static constexpr int kind = kBF16x2; };

size_t matmul_int8_grad_bytes(int planes, int64_t T, int64_t m, int64_t n) {
  return (size_t)plane_ld(m) * (size_t)(n + planes * T);
}

template <typename G>
hipError_t launch_matmul_int8_grad(int64_t T, int64_t m, int64_t n, const G* g, int64_t ldg,
                                   const int8_t* Vq, int64_t ldv, const float* sv,
                                   const float* channel, G* dX, int64_t ldx, void* ws,
                                   hipStream_t s) {
  constexpr int kind = GradSplit<G>::kind;
  if (T <= 0 || n <= 0) return hipSuccess;
  const int64_t ld = plane_ld(m);
  const Planes v = {(char*)ws, ld, 0}, gp = {(char*)ws + n * ld, ld, T * ld};
  hipError_t e = launch_planes_t<I8, kBF16x1>(m, n, (const I8*)Vq, ldv, nullptr, v, s);
  if (e != hipSuccess) return e;
  if ((e = launch_planes<G, kind>(T, m, g, ldg, sv, gp, s)) != hipSuccess) return e;
  const PlanePairs pairs = {kPlanes[kind], {0, 0, 0}, {0, 1, 2}};
  const PlaneEpilogue ep = {channel, nullptr, nullptr, 1.0f, nullptr, 0};
  return launch_plane_product<G, false>(n, T, m, v, gp, pairs, ep, dX, ldx, s);
}

#define BK_INST_P(X, KIND)                                                                  \
  template hipError_t launch_planes<X, KIND>(int64_t, int64_t, const X*, int64_t,           \
                                             const float*, Planes, hipStream_t);            \
  template hipError_t launch_planes_t<X, KIND>(int64_t, int64_t, const X*, int64_t,         \
                                               const float*, Planes, hipStream_t);
BK_INST_P(float, kBF16x3)
BK_INST_P(BF16, kBF16x1)
BK_INST_P(F16, kF16x1)
#undef BK_INST_P
#define BK_INST_Y(O, F)                                                                     \
  template hipError_t launch_plane_product<O, F>(int64_t, int64_t, int64_t, Planes, Planes, \
                                                 const PlanePairs&, const PlaneEpilogue&,   \
                                                 O*, int64_t, hipStream_t);
BK_INST_Y(float, false)
BK_INST_Y(float, true)
BK_INST_Y(BF16, false)
BK_INST_Y(F16, true)
#undef BK_INST_Y
#define BK_INST(G)                                                                            \
  template hipError_t launch_matmul_int8_grad<G>(int64_t, int64_t, int64_t, const G*,         \
                                                 int64_t, const int8_t*, int64_t,             \
                                                 const float*, const float*, G*, int64_t,     \
                                                 void*, hipStream_t);
BK_INST(float)
BK_INST(BF16)
BK_INST(F16)
#undef BK_INST

}  // namespace bk
