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

// Eight columns of one row, one 16-byte store per plane: group `at` of all rows.
template <typename X, int KIND>
__device__ inline void planes_group(int64_t at, int64_t rows, int64_t cols, const X* x, int64_t ldx,
                                    const float* rs, const float* cs, const Planes& out, bool vec) {
  constexpr int NP = kPlanes[KIND];
  const int64_t per = out.ld / 16;
  if (at >= rows * per) return;
  const int64_t r = at / per, c0 = (at - r * per) * 8;
  const Eight<X> t8 = load8(x + r * ldx, c0, cols, vec);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = to_f32(t8.v[e]);
  if (cs) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= cs[c0 + e < cols ? c0 + e : cols - 1];
  }
  if (rs) {
    const float f = rs[r];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f == 0.0f ? 0.0f : v[e] * f;
  }
  unsigned short w[NP][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    unsigned short t[NP];
    split16<KIND>(v[e], t);
#pragma unroll
    for (int p = 0; p < NP; ++p) w[p][e] = t[p];
  }
#pragma unroll
  for (int p = 0; p < NP; ++p)
    *(v4i*)(out.w + p * out.plane + r * out.ld + c0 * 2) = __builtin_bit_cast(v4i, w[p]);
}
template <typename X, int KIND>
__global__ __launch_bounds__(256) void planes_kernel(int64_t rows, int64_t cols,
                                                     const X* __restrict__ x, int64_t ldx,
                                                     const float* __restrict__ rs,
                                                     const float* __restrict__ cs, Planes out,
                                                     bool vec) {
  planes_group<X, KIND>((int64_t)blockIdx.x * 256 + threadIdx.x, rows, cols, x, ldx, rs, cs, out,
                        vec);
}

template <typename X, int KIND>
hipError_t launch_planes(int64_t rows, int64_t cols, const X* x, int64_t ldx,
                         const float* row_scale, const float* col_scale, Planes out,
                         hipStream_t s) {
  const int64_t n = rows * (out.ld / 16);
  if (n <= 0) return hipSuccess;
  hipLaunchKernelGGL((planes_kernel<X, KIND>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                     rows, cols, x, ldx, row_scale, col_scale, out, load8_ok(x, ldx));
  return hipGetLastError();
}

// ---- products -----------------------------------------------------------------

// A tiled product of planes, R k-major. 4096 x 4096 with k = 32768 in bfloat16: 750 to
// 800 us, 1.37 to 1.47 PFLOP/s (a library's large product reaches 1.48 here); with k =
// 4096 over eight rounds of tiles 1.2, the ring's filling and the stores
// standing between tiles.
//
// Workgroup b: tile b % (nr nc), of `splits` equal ranges of the steps number
// b / (nr nc). With more than one range the sums go to parts[range][c][r]
// (rows ldp apart, ranges `stride`) and the epilogue to plane_join_kernel.
template <class M, typename O, int BR, int BC, int WR, int WC, bool CK>
__global__ __launch_bounds__(64 * WR * WC) void plane_product_kernel(
    TileOperand R, TileOperand C, int64_t kbytes, PlanePairs pairs, PlaneEpilogue ep,
    O* __restrict__ Y, int64_t ldy, bool vec, unsigned nr, unsigned nc, int splits,
    float* __restrict__ parts, int64_t ldp, int64_t stride) {
  typedef TileProduct<M, BR, BC, WR, WC, true, CK> TP;
  extern __shared__ char lds[];
  const unsigned tiles = nr * nc;
  const int range = blockIdx.x / tiles;
  int tr, tc;
  tile_of(blockIdx.x - range * tiles, nr, nc, tr, tc);
  const int64_t r0 = (int64_t)tr * BR, c0 = (int64_t)tc * BC;
  const int total = TP::steps(kbytes, pairs);
  TP tp;
  tp.zero();
  tp.run(R, C, kbytes, pairs, r0, c0, (int)((int64_t)total * range / splits),
         (int)((int64_t)total * (range + 1) / splits), lds);
  const int lane = threadIdx.x & 63;
  const int64_t rb = r0 + tp.wave_r() + 4 * (lane >> 4), cb = c0 + tp.wave_c() + (lane & 15);
  if (splits > 1) {
    store_sums(tp, r0, c0, C.rows, parts + range * stride, ldp);
    return;
  }
  const float all = (ep.alpha ? *ep.alpha : 1.0f) * ep.beta;
  float sc[TP::FC];
#pragma unroll
  for (int j = 0; j < TP::FC; ++j) {
    const int64_t c = cb + j * 16;
    sc[j] = (ep.col_scale ? ep.col_scale[c < C.rows ? c : C.rows - 1] : 1.0f) * all;
  }
  if (ep.prev) {  // rows of whole groups of four: its columns are padded
#pragma unroll
    for (int j = 0; j < TP::FC; ++j) {
      const int64_t c = cb + j * 16;
      if (c < C.rows) {
#pragma unroll
        for (int i = 0; i < TP::FR; ++i)
          if (rb + i * 16 < R.rows)
            tp.acc[i][j] += *(const f32x4*)(ep.prev + c * ep.ldprev + rb + i * 16);
      }
      __builtin_amdgcn_sched_barrier(0);  // one column's loads at a time: registers
    }
  }
  if (ep.row_scale) {
#pragma unroll
    for (int i = 0; i < TP::FR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t r = rb + i * 16 + e;
        const float f = ep.row_scale[r < R.rows ? r : R.rows - 1];
#pragma unroll
        for (int j = 0; j < TP::FC; ++j) tp.acc[i][j][e] *= f;
      }
  }
  store_tile(tp, r0, c0, R.rows, C.rows, Y, ldy, vec,
             [&](float a, int, int j, int) { return a * sc[j]; });
}

// The ranges' sums in order, and the epilogue; four columns of one row a thread
// (join_ranges).
template <typename O, int S>
__global__ __launch_bounds__(256) void plane_join_kernel(int64_t M, int64_t N, int splits,
                                                         const float* __restrict__ parts,
                                                         int64_t ldp, int64_t stride,
                                                         PlaneEpilogue ep, O* __restrict__ Y,
                                                         int64_t ldy, bool vec) {
  __shared__ f32x4 red[S > 1 ? 256 : 1];
  const int64_t per = ldp / 4, at = JoinAt<S>::at();
  const int64_t c = at / per, r = (at - c * per) * 4;
  f32x4 a;
  if (!join_ranges<S>(parts + c * ldp + r, stride, splits, at < N * per, a, red)) return;
  if (ep.prev) a += *(const f32x4*)(ep.prev + c * ep.ldprev + r);
  const float all = (ep.alpha ? *ep.alpha : 1.0f) * ep.beta;
  const float sc = (ep.col_scale ? ep.col_scale[c] : 1.0f) * all;
  O t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float sr = ep.row_scale ? ep.row_scale[r + e < M ? r + e : M - 1] : 1.0f;
    t[e] = from_f32<O>(a[e] * sr * sc);
  }
  if (vec && r + 4 <= M) {
    *(typename Vec4<O>::type*)(Y + c * ldy + r) = __builtin_bit_cast(typename Vec4<O>::type, t);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r + e < M) Y[c * ldy + r + e] = t[e];
  }
}

static TilePlan plane_plan(int64_t M, int64_t N, int64_t K, int npairs) {
  return plan_tiles(M, N, (K + 63) / 64, npairs, true, true);
}
size_t plane_product_bytes(int64_t M, int64_t N, int64_t K, int npairs) {
  return (size_t)split_words(M, N, plane_plan(M, N, K, npairs).splits) * 4;
}

template <class M, typename O, int BR, int BC, int WR, int WC, bool CK>
static hipError_t start_plane_product(const TileOperand& R, const TileOperand& C, int64_t kbytes,
                                      const PlanePairs& pairs, const PlaneEpilogue& ep, O* Y,
                                      int64_t ldy, int splits, float* parts, hipStream_t s) {
  typedef TileProduct<M, BR, BC, WR, WC, true, CK> TP;
  auto* k = plane_product_kernel<M, O, BR, BC, WR, WC, CK>;
  if (TP::kLds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, TP::kLds);
    if (e != hipSuccess) return e;
  }
  const int64_t nr = (R.rows + BR - 1) / BR, nc = (C.rows + BC - 1) / BC;
  const int64_t ldp = (R.rows + 3) / 4 * 4, stride = C.rows * ldp;
  const bool vec = vec4_ok(Y, ldy);
  hipLaunchKernelGGL(k, dim3((unsigned)(nr * nc * splits)), dim3(TP::kThreads), TP::kLds, s, R, C,
                     kbytes, pairs, ep, Y, ldy, vec, (unsigned)nr, (unsigned)nc, splits, parts, ldp,
                     stride);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
#define BK_JOIN(S)                                                                               \
  hipLaunchKernelGGL((plane_join_kernel<O, S>),                                                  \
                     dim3((unsigned)((stride / 4 + 256 / S - 1) / (256 / S))), dim3(256), 0, s,  \
                     R.rows, C.rows, splits, parts, ldp, stride, ep, Y, ldy, vec)
  if (join_slices(splits) == 1) BK_JOIN(1);
  else BK_JOIN(8);
#undef BK_JOIN
  return hipGetLastError();
}

template <typename O, bool F16P, bool CK>
hipError_t launch_plane_product(int64_t M, int64_t N, int64_t K, Planes R, Planes C,
                                const PlanePairs& pairs, const PlaneEpilogue& ep, O* Y,
                                int64_t ldy, float* parts, hipStream_t s) {
  typedef typename std::conditional<F16P, MmaF16, MmaBF16>::type Mma;
  if (M <= 0 || N <= 0) return hipSuccess;
  const TileOperand r = {R.w, R.ld, R.plane, M, K}, c = {C.w, C.ld, C.plane, N, K};
  const int64_t kbytes = (K + 7) / 8 * 16;  // whole 16-byte chunks: the planes' padding is zero
  const TilePlan plan = plane_plan(M, N, K, pairs.n);
  if (plan.tile == 256)
    return start_plane_product<Mma, O, 256, 256, 2, 4, CK>(r, c, kbytes, pairs, ep, Y, ldy, 1, parts,
                                                           s);
  if (plan.tile == 128)
    return start_plane_product<Mma, O, 128, 128, 2, 2, CK>(r, c, kbytes, pairs, ep, Y, ldy,
                                                           plan.splits, parts, s);
  return start_plane_product<Mma, O, 64, 64, 2, 2, CK>(r, c, kbytes, pairs, ep, Y, ldy, plan.splits,
                                                       parts, s);
}

// ---------------------------------------------------------------------------
// Input gradient of the 8-bit product: dX[t][j] = channel[j] sum_i (G[t][i]
// sv[i]) Vq[i][j]. The codes are exact in 16-bit floats, so the product runs on
// those instructions with Vq as one k-major plane. For a 16-bit G the other
// operand is one float16 plane of G sv times a power of two for each token,
// which brings the token's largest to [2^14, 2^15): 11 bits, which values down to
// 2^-28 of the largest keep. (One bfloat16 plane would keep 8 bits, as coarse as
// a bfloat16 output, at the same cost; more bits cost a second product.) A
// float32 G is three bfloat16 planes, all 24 bits.
// 8192 x 4096 x 14336 bfloat16: 775 to 815 us, of them 56 to 60 for the two operands (bound
// by memory); 512 x 1024 x 2048 float32: 26 us in three kernels.
// ---------------------------------------------------------------------------
// The codes as one plane, m x n: the part of both operands' launch that both
// types of G share.
struct GradCodes {
  const I8* v;
  int64_t ld, m, n;
  Planes out;
  bool vec;
};
template <int KIND>
__device__ inline void grad_codes(int64_t block, const GradCodes& c) {
  planes_group<I8, KIND>(block * 256 + threadIdx.x, c.m, c.n, c.v, c.ld, nullptr, nullptr, c.out,
                         c.vec);
}
__global__ __launch_bounds__(256) void grad_planes_kernel(int64_t T, int64_t m,
                                                          const float* __restrict__ g, int64_t ldg,
                                                          const float* __restrict__ sv, Planes out,
                                                          bool vec, int64_t blocks, GradCodes c) {
  if ((int64_t)blockIdx.x < blocks)
    planes_group<float, kBF16x3>((int64_t)blockIdx.x * 256 + threadIdx.x, T, m, g, ldg, nullptr, sv,
                                 out, vec);
  else
    grad_codes<kBF16x1>(blockIdx.x - blocks, c);
}
template <typename G, int NV>
__global__ __launch_bounds__(256) void grad_tokens_kernel(int64_t T, int64_t m,
                                                          const G* __restrict__ g, int64_t ldg,
                                                          const float* __restrict__ sv, Planes out,
                                                          float* __restrict__ unscale, bool vec,
                                                          bool vecs, GradCodes codes) {
  if ((int64_t)blockIdx.x >= T) {
    grad_codes<kF16x1>(blockIdx.x - T, codes);
    return;
  }
  __shared__ unsigned red[4];
  const RowOf<G, NV> row(g + (int64_t)blockIdx.x * ldg, m, vec);
  auto values = [&](int64_t c, const Eight<G>& t, float* v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(t.v[e]);
    if (sv) {
      float f[8];
      factors8(sv, c, m, vecs, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= f[e];
    }
  };
  unsigned top = 0;
  row.each(m, [&](int64_t c, const Eight<G>& t) {
    float v[8];
    values(c, t, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // what lies past m was read as zero
      const unsigned a = __float_as_uint(v[e]) & 0x7fffffffu;
      top = a > top ? a : top;
    }
  });
  top = max_of_256(top, red);
  // 2^k with 2^(14 - k) <= the largest < 2^(15 - k); an infinity or NaN counts as
  // 2^127 (finite values beside it stay finite), small ones as 2^-112 (2^k stays normal)
  const int e = (int)(top >> 23) - 127;
  const int k = e > 127 ? -113 : e < -112 ? 126 : 14 - e;
  const float scale = __uint_as_float((unsigned)(k + 127) << 23);
  if (threadIdx.x == 0) unscale[blockIdx.x] = __uint_as_float((unsigned)(127 - k) << 23);
  row.each(out.ld / 2, [&](int64_t c, const Eight<G>& t) {
    float v[8];
    values(c, t, v);
    _Float16 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (_Float16)(v[i] * scale);
    *(v4i*)(out.w + (int64_t)blockIdx.x * out.ld + c * 2) = __builtin_bit_cast(v4i, w);
  });
}

// Both operands in one launch: G's tokens, and behind them the codes.
template <typename G>
static hipError_t launch_grad_operands(int64_t T, int64_t m, const G* g, int64_t ldg,
                                       const float* sv, Planes out, float* unscale,
                                       const GradCodes& c, hipStream_t s) {
  const int64_t blocks = (c.m * (c.out.ld / 16) + 255) / 256;
  const bool vec = load8_ok(g, ldg), vecs = load8_ok(sv, 0);
  if constexpr (sizeof(G) == 4) {
    const int64_t own = (T * (out.ld / 16) + 255) / 256;
    if (own + blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(grad_planes_kernel, dim3((unsigned)(own + blocks)), dim3(256), 0, s, T, m, g,
                       ldg, sv, out, vec, own, c);
  } else {
#define BK_ROWS(NV)                                                                             \
  hipLaunchKernelGGL((grad_tokens_kernel<G, NV>), dim3((unsigned)(T + blocks)), dim3(256), 0, s, \
                     T, m, g, ldg, sv, out, unscale, vec, vecs, c)
    switch (row_groups(out.ld / 2)) {
      case 1: BK_ROWS(1); break;
      case 2: BK_ROWS(2); break;
      case 4: BK_ROWS(4); break;
      case 8: BK_ROWS(8); break;
      default: BK_ROWS(0);
    }
#undef BK_ROWS
  }
  return hipGetLastError();
}

static inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
struct GradOffsets {
  size_t v, g, unscale, parts, total;
};
static GradOffsets grad_offsets(int es, int64_t T, int64_t m, int64_t n) {
  GradOffsets o;
  o.v = 0;
  o.g = o.v + up256((size_t)(m * plane_ld(n)));
  o.unscale = o.g + up256((size_t)((es == 4 ? 3 : 1) * T * plane_ld(m)));
  o.parts = o.unscale + up256((size_t)T * 4);
  o.total = o.parts + plane_product_bytes(n, T, m, es == 4 ? 3 : 1);
  return o;
}
size_t matmul_int8_grad_bytes(int es, int64_t T, int64_t m, int64_t n) {
  return grad_offsets(es, T, m, n).total;
}

template <typename G>
hipError_t launch_matmul_int8_grad(int64_t T, int64_t m, int64_t n, const G* g, int64_t ldg,
                                   const int8_t* Vq, int64_t ldv, const float* sv,
                                   const float* channel, G* dX, int64_t ldx, void* ws,
                                   hipStream_t s) {
  constexpr bool wide = sizeof(G) == 4;
  if (T <= 0 || n <= 0) return hipSuccess;
  const GradOffsets o = grad_offsets(sizeof(G), T, m, n);
  char* b = (char*)ws;
  const Planes v = {b + o.v, plane_ld(n), 0}, gp = {b + o.g, plane_ld(m), T * plane_ld(m)};
  float* unscale = (float*)(b + o.unscale);
  const GradCodes codes = {(const I8*)Vq, ldv, m, n, v, load8_ok((const I8*)Vq, ldv)};
  const hipError_t e = launch_grad_operands(T, m, g, ldg, sv, gp, unscale, codes, s);
  if (e != hipSuccess) return e;
  const PlanePairs pairs = wide ? PlanePairs{3, 0x000, 0x210} : PlanePairs{1, 0, 0};
  const PlaneEpilogue ep = {channel, wide ? nullptr : unscale, nullptr, 1.0f, nullptr, 0};
  return launch_plane_product<G, !wide, false>(n, T, m, v, gp, pairs, ep, dX, ldx,
                                               (float*)(b + o.parts), s);
}

#define BK_INST_P(X, KIND)                                                                 \
  template hipError_t launch_planes<X, KIND>(int64_t, int64_t, const X*, int64_t,          \
                                             const float*, const float*, Planes, hipStream_t);
BK_INST_P(float, kBF16x3)
BK_INST_P(BF16, kBF16x1)
BK_INST_P(F16, kF16x1)
#undef BK_INST_P
#define BK_INST_Y(O, F, CK)                                                                \
  template hipError_t launch_plane_product<O, F, CK>(int64_t, int64_t, int64_t, Planes,    \
                                                     Planes, const PlanePairs&,            \
                                                     const PlaneEpilogue&, O*, int64_t,    \
                                                     float*, hipStream_t);
BK_INST_Y(float, false, false)
BK_INST_Y(float, true, false)
BK_INST_Y(BF16, false, false)
BK_INST_Y(F16, true, false)
BK_INST_Y(float, false, true)
BK_INST_Y(BF16, false, true)
BK_INST_Y(F16, true, true)
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
