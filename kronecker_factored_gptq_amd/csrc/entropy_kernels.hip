// Softmax cross entropy over a large vocabulary on gfx950, the logits z = X W^T
// never stored, and its gradient.
//
// Forward: a tiled product (tile_product.hpp; rows = vocabulary, columns =
// tokens) whose epilogue keeps, per token and wave, the largest logit m and
// sum exp(z - m) of its rows, and the target's logit; a second kernel joins
// these to lse and the loss.
//
// Gradient: with D[t][v] = exp(z - lse_t) - [v = y_t] (0 for a token without a
// target), dX = g (.) (D W) and dW = D^T (g (.) X). The vocabulary goes by in
// pieces: a piece's logits are formed again, D is written as 16-bit planes, and
// the two products are formed from it, W, X and (for dW) D read k-major; dX is
// summed over the pieces in float32.
//
// float32 operands are three bfloat16 planes each (exact), and a product the six
// pairs of planes whose terms reach float32's precision.
//
// 4096 tokens, d = 4096, 128256 words, bfloat16: forward 3.15 to 3.25 ms (1.32 to 1.37
// PFLOP/s in 256 x 256 tiles; a tile's epilogue, 65536 exponentials, takes its share
// of what is missing to a plain product), gradient 10.1 to 10.7 ms (1.21 to 1.28): D
// 0.91 ms a piece, D W 0.78, D^T X 0.90. One token, d = 2048, 50257 words, float16:
// 45 us (4.5 TB/s). 333 x 1000 x 10007 float32, gradient: 211 to 220 us, of them 16 for W's
// planes and 183 for six plane products in each of the three products.
#include <initializer_list>

#include "launch.hpp"
#include "skinny_product.hpp"
#include "tile_product.hpp"

namespace bk {

namespace {

template <typename X> struct Kind;
template <> struct Kind<float> {
  typedef MmaBF16 mma;  // of the planes
  typedef MmaF32 whole;
  static constexpr int split = kBF16x3;
  static constexpr bool f16 = false;
};
template <> struct Kind<BF16> {
  typedef MmaBF16 mma;
  typedef MmaBF16 whole;
  static constexpr int split = kBF16x1;
  static constexpr bool f16 = false;
};
template <> struct Kind<F16> {
  typedef MmaF16 mma;
  typedef MmaF16 whole;
  static constexpr int split = kF16x1;
  static constexpr bool f16 = true;
};

// What D is multiplied by before it becomes 16-bit planes: float16 reaches down
// to 2^-24, and probabilities of a large vocabulary well below; 2^14 brings
// them up, |D| <= 1 staying far from its largest value. bfloat16 has float32's
// range.
template <typename X> constexpr float dscale() { return Kind<X>::f16 ? 16384.0f : 1.0f; }

template <typename X> inline PlanePairs pairs_of() {
  if (kPlanes[Kind<X>::split] == 3) return {6, 0x120100, 0x102010};
  return {1, 0, 0};
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = 1.925963033500606e-8f;  // log2 e - kLog2e
// exp by one instruction (2^-23), its argument rounded once in base 2: 2^-24 |x| and without
// a bias. A logit's own rounding to float32 moves its exponential as far.
__device__ inline float exp_of(float x) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(x, kLog2e, x * kLog2eLow));
}
// exp to 2^-22 at any x whose result is a normal number: what the argument lost, r, is
// put back as a factor 1 + r ln 2. For float32 gradients, which keep all of its bits: 0 to
// 2 % of their time (333 x 1000 x 10007: 215 -> 219 us, 512 x 1024 x 32000: 697 -> 698); in
// the forward, whose logits' roundings weigh as much, it would be 2 % of 4096 x 4096 x 128256
// in bfloat16 (3144 -> 3211 us; exp_of's own second product 0.6 %).
__device__ inline float exp_exactly(float x) {
  const float t = x * kLog2e, e = __builtin_amdgcn_exp2f(t);
  const float r = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
  return e > 0.0f ? __builtin_fmaf(e, r * 0.6931471805599453f, e) : e;  // -inf: 0, r being NaN
}

struct MaxSum {
  float m, s;
};
// The sums of two sets of terms, each relative to its largest; an empty set has
// m = -inf, s = 0.
__device__ inline MaxSum join(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -__builtin_inff()) return {m, a.s + b.s};
  return {m, a.s * exp_of(a.m - m) + b.s * exp_of(b.m - m)};
}

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// parts[(part0 + tile * WR + wave row) * T + t], and zy[t] from the wave that
// holds row y[t]; W's rows are the vocabulary's from v0 on.
template <class M, int BR, int BC, int WR, int WC, bool ANY>
__global__ __launch_bounds__(64 * WR * WC) void entropy_kernel(
    TileOperand W, TileOperand X, int64_t kbytes, PlanePairs pairs, const int64_t* __restrict__ y,
    int64_t v0, MaxSum* __restrict__ parts, int64_t part0, float* __restrict__ zy, unsigned nr,
    unsigned nc) {
  typedef TileProduct<M, BR, BC, WR, WC> TP;
  extern __shared__ char lds[];
  int tr, tc;
  tile_of(blockIdx.x, nr, nc, tr, tc);
  const int64_t r0 = (int64_t)tr * BR, c0 = (int64_t)tc * BC;
  TP tp;
  tp.zero();
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int64_t rb = r0 + tp.wave_r(), T = X.rows;
  // rows of this lane's that are W's: 16 i + 4 q + e < left
  const int left = (int)(W.rows - rb < TP::FR * 16 ? W.rows - rb : TP::FR * 16) - 4 * q;
  // where 16 i + e of the lane's rows is the target: read before the product, whose
  // end would otherwise wait for them
  int target[TP::FC];
#pragma unroll
  for (int j = 0; j < TP::FC; ++j) {
    const int64_t t = c0 + tp.wave_c() + j * 16 + (lane & 15);
    const int64_t yt = y[t < T ? t : T - 1], at = yt - v0 - rb - 4 * q;
    target[j] = yt >= 0 && at >= 0 && at < left && t < T ? (int)at : -1;
  }
  if (ANY)
    tp.run_any(W, X, kbytes, r0, c0, lds);
  else
    tp.run(W, X, kbytes, pairs, r0, c0, 0, TP::steps(kbytes, pairs), lds);
  if (rb + TP::FR * 16 > W.rows) {  // the last tile: rows past W's add nothing
#pragma unroll
    for (int i = 0; i < TP::FR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (16 * i + e >= left) {
#pragma unroll
          for (int j = 0; j < TP::FC; ++j) tp.acc[i][j][e] = -__builtin_inff();
        }
  }
  const int64_t part = part0 + (int64_t)tr * WR + (threadIdx.x >> 6) / WC;
#pragma unroll
  for (int j = 0; j < TP::FC; ++j) {
    const int64_t t = c0 + tp.wave_c() + j * 16 + (lane & 15);
    float m = tp.acc[0][j][0];
#pragma unroll
    for (int i = 0; i < TP::FR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = fmaxf(m, tp.acc[i][j][e]);
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    // a set of -inf alone sums to 0 (and one with a NaN to NaN)
    const float base = m == -__builtin_inff() ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < TP::FR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s += exp_of(tp.acc[i][j][e] - base);
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (t < T && q == 0) parts[part * T + t] = {m, s};
    if (target[j] >= 0) {
#pragma unroll
      for (int i = 0; i < TP::FR; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * i + e == target[j]) zy[t] = tp.acc[i][j][e];
    }
  }
}

// The same for few tokens, bound by reading W once: part blockIdx.x * RT + i are
// its 16 rows of that number.
template <class M, int RT, int NT, bool ANY>
__global__ __launch_bounds__(512) void skinny_entropy_kernel(TileOperand W, TileOperand X,
                                                             int64_t kbytes,
                                                             const int64_t* __restrict__ y,
                                                             MaxSum* __restrict__ parts,
                                                             float* __restrict__ zy) {
  typedef SkinnyProduct<M, RT, NT, RT == 1 ? 4 : 2, ANY> SP;
  __shared__ __attribute__((aligned(16))) char lds[SP::kLds];
  const int64_t r0 = (int64_t)blockIdx.x * SP::kRows, r = r0 + SP::tile_r();
  const int64_t t = SP::tile_c(), T = X.rows;
  const int64_t yt = SP::has_tile() && t < T ? y[t] : -1;
  SP::run(W, X, kbytes, r0, lds, [&](f32x4 z) {
    const int left = W.rows - r < 4 ? (int)(W.rows - r) : 4;
    float m = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) m = fmaxf(m, z[e]);
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    const float base = m == -__builtin_inff() ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) s += exp_of(z[e] - base);
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (t >= T) return;
    const int64_t part = r / 16;
    if ((threadIdx.x & 63) < 16 && part * 16 < W.rows) parts[part * T + t] = {m, s};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left && yt == r + e) zy[t] = z[e];
  });
}

// TX tokens per workgroup, 256 / TX threads to each, the parts in a fixed order.
template <int TX>
__global__ __launch_bounds__(256) void entropy_join_kernel(
    int64_t T, int64_t V, int64_t nparts, const MaxSum* __restrict__ parts,
    const float* __restrict__ zy, const int64_t* __restrict__ y, float* __restrict__ loss,
    float* __restrict__ lse) {
  constexpr int TY = 256 / TX;
  __shared__ MaxSum red[256];
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int64_t t = (int64_t)blockIdx.x * TX + tx;
  MaxSum a = {-__builtin_inff(), 0.0f};
  if (t < T) {
    int64_t p = ty;
    for (; p + 3 * TY < nparts; p += 4 * TY) {  // four loads on their way at once
      MaxSum b[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) b[k] = parts[(p + k * TY) * T + t];
      a = join(a, join(join(b[0], b[1]), join(b[2], b[3])));
    }
    for (; p < nparts; p += TY) a = join(a, parts[p * T + t]);
  }
  red[threadIdx.x] = a;
  __syncthreads();
#pragma unroll
  for (int k = TY / 2; k > 0; k /= 2) {
    if (ty < k) red[threadIdx.x] = join(red[threadIdx.x], red[threadIdx.x + k * TX]);
    __syncthreads();
  }
  if (ty == 0 && t < T) {
    a = red[tx];
    const float l = a.m + logf(a.s);
    lse[t] = l;
    loss[t] = y[t] >= 0 && y[t] < V ? l - zy[t] : 0.0f;
  }
}

// The largest |x| of each token, for float16's weights below.
template <typename X>
__global__ __launch_bounds__(256) void entropy_reach_kernel(int64_t d, const X* __restrict__ x,
                                                            int64_t ldx, bool vec,
                                                            float* __restrict__ reach) {
  __shared__ unsigned red[4];
  const RowOf<X, 0> row(x + (int64_t)blockIdx.x * ldx, d, vec);
  unsigned top = 0;
  row.each(d, [&](int64_t, const Eight<X>& t) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned a = __float_as_uint(to_f32(t.v[e])) & 0x7fffffffu;
      top = a > top ? a : top;
    }
  });
  top = max_of_256(top, red);
  if (threadIdx.x == 0) reach[blockIdx.x] = __uint_as_float(top);
}

// w[t] = g[t] for a token with a target, else 0; top = max |w|; rel = w / top
// (0 where top is 0). rel X is rounded to X's type for dW. With `reach`
// (float16, whose normal numbers end at 2^-14): rel times, and top divided by, the power
// of two that brings the largest |rel X| to [2^14, 2^15), so that 11 bits are kept down to
// 2^-28 of it. One workgroup. Maxima are taken over bits, in which a NaN is larger than
// infinity.
__global__ __launch_bounds__(1024) void entropy_weights_kernel(
    int64_t T, int64_t V, const int64_t* __restrict__ y, const float* __restrict__ g,
    const float* __restrict__ reach, float* __restrict__ w, float* __restrict__ rel,
    float* __restrict__ top) {
  __shared__ unsigned red[16];
  auto largest = [&](unsigned m) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const unsigned u = __shfl_xor(m, o, 64);
      m = u > m ? u : m;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int k = 0; k < 16; ++k) m = red[k] > m ? red[k] : m;
    return m;
  };
  unsigned m = 0;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const float v = y[t] >= 0 && y[t] < V ? g[t] : 0.0f;
    w[t] = v;
    const unsigned a = __float_as_uint(v) & 0x7fffffffu;
    m = a > m ? a : m;
  }
  m = largest(m);
  const float mx = __uint_as_float(m);
  int k = 0;
  if (reach) {
    unsigned r = 0;
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
      const float v = w[t] == 0.0f ? 0.0f : w[t] / mx * reach[t];
      const unsigned a = __float_as_uint(v) & 0x7fffffffu;
      r = a > r ? a : r;
    }
    r = largest(r);
    const int e = (int)(r >> 23) - 127;
    k = r == 0 || e > 127 ? 0 : e < -112 ? 126 : 14 - e;  // 2^k and 2^-k normal
  }
  const float up = __uint_as_float((unsigned)(127 + k) << 23);
  if (threadIdx.x == 0) *top = mx * __uint_as_float((unsigned)(127 - k) << 23);
  for (int64_t t = threadIdx.x; t < T; t += 1024)
    rel[t] = w[t] == 0.0f ? 0.0f : w[t] / mx * up;
}

// D's planes of a piece, rows the tokens, written up to the planes' padding, with
// zeros there.
template <class M, int KIND, int BR, int BC, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) void entropy_diff_kernel(
    TileOperand W, TileOperand X, int64_t kbytes, PlanePairs pairs, const int64_t* __restrict__ y,
    int64_t V, int64_t v0, const float* __restrict__ lse, float scale, Planes P, unsigned nr,
    unsigned nc) {
  typedef TileProduct<M, BR, BC, WR, WC> TP;
  constexpr int NP = kPlanes[KIND];
  extern __shared__ char lds[];
  int tr, tc;
  tile_of(blockIdx.x, nr, nc, tr, tc);
  const int64_t r0 = (int64_t)tr * BR, c0 = (int64_t)tc * BC;
  TP tp;
  tp.zero();
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int64_t T = X.rows, rb = r0 + tp.wave_r() + 4 * q;
  // The token's lse, and where 16 i + e of the lane's rows is the target (-1:
  // nowhere, -2: the token has none); read before the product, whose end would
  // otherwise wait for them.
  int target[TP::FC];
  float norm[TP::FC];
#pragma unroll
  for (int j = 0; j < TP::FC; ++j) {
    const int64_t t = c0 + tp.wave_c() + j * 16 + (lane & 15), tt = t < T ? t : T - 1;
    const int64_t yt = y[tt], at = yt - v0 - rb;
    target[j] = yt < 0 || yt >= V ? -2 : at >= 0 && at < TP::FR * 16 ? (int)at : -1;
    norm[j] = lse[tt];
  }
  tp.run(W, X, kbytes, pairs, r0, c0, 0, TP::steps(kbytes, pairs), lds);
  const bool whole = r0 + tp.wave_r() + TP::FR * 16 <= W.rows;
#pragma unroll
  for (int j = 0; j < TP::FC; ++j) {
    const int64_t t = c0 + tp.wave_c() + j * 16 + (lane & 15);
    const bool has = target[j] != -2;
#pragma unroll
    for (int i = 0; i < TP::FR; ++i) {
      const int64_t r = rb + i * 16;
      unsigned short w[NP][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = tp.acc[i][j][e] - norm[j];
        float v = KIND == kBF16x3 ? exp_exactly(a) : exp_of(a);
        if (16 * i + e == target[j]) v -= 1.0f;
        v = has && (whole || r + e < W.rows) ? v * scale : 0.0f;
        unsigned short k[NP];
        split16<KIND>(v, k);
#pragma unroll
        for (int p = 0; p < NP; ++p) w[p][e] = k[p];
      }
#pragma unroll
      for (int p = 0; p < NP; ++p)
        if (t < T && r * 2 < P.ld)
          *(uint2*)(P.w + p * P.plane + t * P.ld + r * 2) = __builtin_bit_cast(uint2, w[p]);
    }
  }
}

template <class M, int BR, int BC, int WR, int WC, bool ANY>
static hipError_t start_entropy(const TileOperand& W, const TileOperand& X, int64_t kbytes,
                                const PlanePairs& pairs, const int64_t* y, int64_t v0,
                                MaxSum* parts, int64_t& part0, float* zy, hipStream_t s) {
  typedef TileProduct<M, BR, BC, WR, WC> TP;
  auto* k = entropy_kernel<M, BR, BC, WR, WC, ANY>;
  if (TP::kLds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, TP::kLds);
    if (e != hipSuccess) return e;
  }
  const int64_t nr = (W.rows + BR - 1) / BR, nc = (X.rows + BC - 1) / BC;
  hipLaunchKernelGGL(k, dim3((unsigned)(nr * nc)), dim3(TP::kThreads), TP::kLds, s, W, X, kbytes,
                     pairs, y, v0, parts, part0, zy, (unsigned)nr, (unsigned)nc);
  part0 += nr * WR;
  return hipGetLastError();
}

template <class M, bool ANY>
static hipError_t start_skinny_entropy(const TileOperand& W, const TileOperand& X, int64_t kbytes,
                                       const int64_t* y, MaxSum* parts, float* zy, hipStream_t s) {
  const int nt = (int)((X.rows + 15) / 16);
#define BK_SKINNY(RT, NT)                                                            \
  hipLaunchKernelGGL((skinny_entropy_kernel<M, RT, NT, ANY>),                        \
                     dim3((unsigned)((W.rows + 16 * RT - 1) / (16 * RT))), dim3(512), 0, s, W, X, \
                     kbytes, y, parts, zy)
  switch (nt) {
    case 1: BK_SKINNY(1, 1); break;
    case 2: BK_SKINNY(2, 2); break;
    case 3: BK_SKINNY(2, 3); break;
    default: BK_SKINNY(2, 4);
  }
#undef BK_SKINNY
  return hipGetLastError();
}

template <class M, int KIND, int BR, int BC, int WR, int WC>
static hipError_t start_entropy_diff(const TileOperand& W, const TileOperand& X, int64_t kbytes,
                                     const PlanePairs& pairs, const int64_t* y, int64_t V,
                                     int64_t v0, const float* lse, float scale, Planes P,
                                     hipStream_t s) {
  typedef TileProduct<M, BR, BC, WR, WC> TP;
  auto* k = entropy_diff_kernel<M, KIND, BR, BC, WR, WC>;
  if (TP::kLds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, TP::kLds);
    if (e != hipSuccess) return e;
  }
  const int64_t nr = (W.rows + BR - 1) / BR, nc = (X.rows + BC - 1) / BC;
  hipLaunchKernelGGL(k, dim3((unsigned)(nr * nc)), dim3(TP::kThreads), TP::kLds, s, W, X, kbytes,
                     pairs, y, V, v0, lse, scale, P, (unsigned)nr, (unsigned)nc);
  return hipGetLastError();
}

// ---- workspaces -------------------------------------------------------------
// Rows at once of what takes `per` bytes a row, `room` in all.
static int64_t rows_in(int64_t room, int64_t per, int64_t V) {
  int64_t p = per ? room / per / 256 * 256 : V;
  if (p < 256) p = 256;
  return p < V ? p : V;
}
// Rows of a float32 W whose planes are held at once: 512 MiB of them.
static int64_t plane_piece(int64_t d, int64_t V) {
  return rows_in((int64_t)512 << 20, 3 * plane_ld(d), V);
}
// Columns of D held at once: 256 MiB, what the last-level cache holds. `direct`: W is read as
// it is. A 16-bit W that is laid out shares them with D, so that misaligned operands need
// little more than aligned ones (of 4096 tokens, d 4096, 128256 words 384 MiB, not 672, and of one
// token 256, not 1002; misaligned 10.77 ms against 10.61 and 1.40 against 1.38).
static int64_t diff_piece(int es, int64_t T, int64_t d, int64_t V, bool direct) {
  const int64_t per = 2 * T * (es == 4 ? 3 : 1);
  int64_t p = rows_in((int64_t)256 << 20, per + (es == 4 || direct ? 0 : plane_ld(d)), V);
  if (p > ((int64_t)1 << 20)) p = (int64_t)1 << 20;  // rows the direct loads can step over
  if (es == 4 && p > plane_piece(d, V)) p = plane_piece(d, V);
  return p;
}

// The most tokens the forward's skinny kernel takes.
constexpr int64_t kSkinnyTokens = 64;

// Offsets into the workspaces.
struct EntropyLayout {
  size_t parts, zy, xp, wp, total;
};
// Of the forward: parts of a launch over `rows` of W, two waves of rows in each tile.
static int64_t entropy_parts(int64_t rows, int64_t tile) { return 2 * ((rows + tile - 1) / tile); }
static int entropy_tile(int es, int64_t rows, int64_t T, int64_t d) {
  const int64_t kbytes = es == 4 ? (d + 7) / 8 * 16 : d * es;
  return plan_tiles(rows, T, (kbytes + kStepBytes - 1) / kStepBytes, es == 4 ? 6 : 1, false, false)
      .tile;
}
static EntropyLayout entropy_layout(int es, int64_t T, int64_t d, int64_t V) {
  EntropyLayout L;
  L.parts = 0;
  const bool skinny = T <= kSkinnyTokens, planes = es == 4 && !skinny;
  const int64_t piece = planes ? plane_piece(d, V) : V;
  int64_t nparts = (V + 15) / 16;  // every 16 rows
  if (!skinny) {
    const int64_t whole = V / piece, rest = V % piece;
    nparts = whole * entropy_parts(piece, entropy_tile(es, piece, T, d)) +
             (rest ? entropy_parts(rest, entropy_tile(es, rest, T, d)) : 0);
    // 16-bit operands that the direct loads cannot take go through tiles of 128
    const int64_t any = entropy_parts(V, 128);
    if (!planes && any > nparts) nparts = any;
  }
  L.zy = L.parts + up256((size_t)(nparts * T) * sizeof(MaxSum));
  L.xp = L.zy + up256((size_t)T * 4);
  L.wp = L.xp + (planes ? (size_t)(3 * T * plane_ld(d)) : 0);
  L.total = L.wp + (planes ? (size_t)(3 * piece * plane_ld(d)) : 0);
  return L;
}
size_t entropy_bytes(int es, int64_t T, int64_t d, int64_t V) {
  return entropy_layout(es, T, d, V).total;
}

struct GradLayout {
  size_t w, rel, reach, top, xp, xs, wp, p, acc, parts, total;
  int64_t piece, ldacc;
};
// direct: X and W are read as they are, and no planes of them are held.
static GradLayout grad_layout(int es, int64_t T, int64_t d, int64_t V, bool direct) {
  GradLayout L;
  const int64_t np = es == 4 ? 3 : 1;
  L.piece = diff_piece(es, T, d, V, direct);
  L.ldacc = (d + 3) / 4 * 4;
  L.w = 0;
  L.rel = L.w + up256((size_t)T * 4);
  L.reach = L.rel + up256((size_t)T * 4);
  L.top = L.reach + (es == 2 ? up256((size_t)T * 4) : 0);
  L.xp = L.top + 256;
  L.xs = L.xp + (direct ? 0 : up256((size_t)(np * T * plane_ld(d))));
  L.wp = L.xs + up256((size_t)(np * T * plane_ld(d)));
  L.p = L.wp + (direct ? 0 : up256((size_t)(np * L.piece * plane_ld(d))));
  L.acc = L.p + up256((size_t)(np * T * plane_ld(L.piece)));
  L.parts = L.acc + (L.piece < V ? up256((size_t)(T * L.ldacc) * 4) : 0);
  // both products, of whole pieces and of the last one
  const int n = es == 4 ? 6 : 1;
  size_t most = 0;
  for (int64_t rows : {L.piece, L.piece ? V % L.piece : 0})
    for (size_t b : {plane_product_bytes(d, T, rows, n), plane_product_bytes(d, rows, T, n)})
      if (rows && b > most) most = b;
  L.total = L.parts + most;
  return L;
}
size_t entropy_grad_bytes(int es, int64_t T, int64_t d, int64_t V) {
  // a query knows the sizes alone: 16-bit rows may be aligned or not
  const size_t laid = grad_layout(es, T, d, V, false).total;
  const size_t direct = es == 2 && d % 8 == 0 ? grad_layout(es, T, d, V, true).total : 0;
  return direct > laid ? direct : laid;
}

// ---- calls --------------------------------------------------------------------
template <typename X>
hipError_t launch_entropy(int64_t T, int64_t d, int64_t V, const X* x, int64_t ldx, const X* w,
                          int64_t ldw, const int64_t* y, float* loss, float* lse, void* ws,
                          hipStream_t s) {
  typedef Kind<X> K;
  typedef typename K::mma M;
  if (T <= 0) return hipSuccess;
  const EntropyLayout L = entropy_layout(sizeof(X), T, d, V);
  char* b = (char*)ws;
  MaxSum* parts = (MaxSum*)(b + L.parts);
  float* zy = (float*)(b + L.zy);
  const PlanePairs pairs = pairs_of<X>();
  int64_t nparts = 0;
  hipError_t e;
  constexpr bool split = sizeof(X) == 4;
  TileOperand xo = {(const char*)x, ldx * (int64_t)sizeof(X), 0, T, 0};
  int64_t kbytes = d * (int64_t)sizeof(X), piece = V;
  if (T <= kSkinnyTokens) {
    const TileOperand wo = {(const char*)w, ldw * (int64_t)sizeof(X), 0, V, 0};
    typedef typename K::whole MW;
    e = tile_direct(wo, kbytes) && tile_direct(xo, kbytes)
            ? start_skinny_entropy<MW, false>(wo, xo, kbytes, y, parts, zy, s)
            : start_skinny_entropy<MW, true>(wo, xo, kbytes, y, parts, zy, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(entropy_join_kernel<1>, dim3((unsigned)T), dim3(256), 0, s, T, V,
                       (V + 15) / 16, parts, zy, y, loss, lse);
    return hipGetLastError();
  }
  if (split) {
    const Planes p = {b + L.xp, plane_ld(d), T * plane_ld(d)};
    if ((e = launch_planes<X, K::split>(T, d, x, ldx, nullptr, nullptr, p, s)) != hipSuccess) return e;
    xo = {p.w, p.ld, p.plane, T, 0};
    kbytes = (d + 7) / 8 * 16;
    piece = plane_piece(d, V);
  }
  for (int64_t v0 = 0; v0 < V; v0 += piece) {
    const int64_t rows = V - v0 < piece ? V - v0 : piece;
    TileOperand wo = {(const char*)(w + v0 * ldw), ldw * (int64_t)sizeof(X), 0, rows, 0};
    if (split) {
      const Planes p = {b + L.wp, plane_ld(d), rows * plane_ld(d)};
      if ((e = launch_planes<X, K::split>(rows, d, w + v0 * ldw, ldw, nullptr, nullptr, p, s)) != hipSuccess)
        return e;
      wo = {p.w, p.ld, p.plane, rows, 0};
    }
    const int tile = entropy_tile(sizeof(X), rows, T, d);
    if (!tile_direct(wo, kbytes) || !tile_direct(xo, kbytes))
      e = start_entropy<M, 128, 128, 2, 2, true>(wo, xo, kbytes, pairs, y, v0, parts, nparts, zy, s);
    else if (tile == 256)
      e = start_entropy<M, 256, 256, 2, 4, false>(wo, xo, kbytes, pairs, y, v0, parts, nparts, zy, s);
    else if (tile == 128)
      e = start_entropy<M, 128, 128, 2, 2, false>(wo, xo, kbytes, pairs, y, v0, parts, nparts, zy, s);
    else
      e = start_entropy<M, 64, 64, 2, 2, false>(wo, xo, kbytes, pairs, y, v0, parts, nparts, zy, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(entropy_join_kernel<16>, dim3((unsigned)((T + 15) / 16)), dim3(256), 0, s, T,
                     V, nparts, parts, zy, y, loss, lse);
  return hipGetLastError();
}

template <typename X>
hipError_t launch_entropy_grad(int64_t T, int64_t d, int64_t V, const X* x, int64_t ldx, const X* w,
                               int64_t ldw, const int64_t* y, const float* lse, const float* g,
                               X* dX, int64_t lddx, X* dW, int64_t lddw, void* ws, hipStream_t s) {
  typedef Kind<X> K;
  typedef typename K::mma M;
  if (T <= 0) {  // no tokens: dW is zero, an empty sum
    const Planes none = {(char*)ws, 0, 0};
    const PlaneEpilogue ep = {nullptr, nullptr, nullptr, 1.0f, nullptr, 0};
    return dW ? launch_plane_product<X, K::f16, true>(d, V, 0, none, none, pairs_of<X>(), ep, dW,
                                                      lddw, nullptr, s)
              : hipSuccess;
  }
  // Both operands as they are, where the direct loads can take them (along d for
  // the logits, W also k-major for dX); else as planes.
  constexpr int64_t es = sizeof(X);
  const int64_t kbytes = (d + 7) / 8 * 16;
  TileOperand xo = {(const char*)x, ldx * es, 0, T, 0};
  const bool direct = es == 2 && d % 8 == 0 && tile_direct(xo, kbytes) &&
                      tile_direct({(const char*)w, ldw * es, 0, V, 0}, kbytes);
  const GradLayout L = grad_layout(es, T, d, V, direct);
  char* b = (char*)ws;
  float *wt = (float*)(b + L.w), *rel = (float*)(b + L.rel), *top = (float*)(b + L.top);
  float *acc = (float*)(b + L.acc), *parts = (float*)(b + L.parts);
  const PlanePairs pairs = pairs_of<X>();
  hipError_t e;
  float* reach = nullptr;
  if (K::f16 && dW) {
    reach = (float*)(b + L.reach);
    hipLaunchKernelGGL(entropy_reach_kernel<X>, dim3((unsigned)T), dim3(256), 0, s, d, x, ldx,
                       load8_ok(x, ldx), reach);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL(entropy_weights_kernel, dim3(1), dim3(1024), 0, s, T, V, y, g, reach, wt, rel,
                     top);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (!direct) {
    const Planes p = {b + L.xp, plane_ld(d), T * plane_ld(d)};
    if ((e = launch_planes<X, K::split>(T, d, x, ldx, nullptr, nullptr, p, s)) != hipSuccess)
      return e;
    xo = {p.w, p.ld, p.plane, T, 0};
  }
  const Planes xs = {b + L.xs, plane_ld(d), T * plane_ld(d)};
  if (dW && (e = launch_planes<X, K::split>(T, d, x, ldx, rel, nullptr, xs, s)) != hipSuccess)
    return e;
  for (int64_t v0 = 0; v0 < V; v0 += L.piece) {
    const int64_t rows = V - v0 < L.piece ? V - v0 : L.piece;
    const X* wv = w + v0 * ldw;
    Planes wp = {(char*)const_cast<X*>(wv), ldw * es, 0};
    if (!direct) {
      wp = {b + L.wp, plane_ld(d), rows * plane_ld(d)};
      if ((e = launch_planes<X, K::split>(rows, d, wv, ldw, nullptr, nullptr, wp, s)) != hipSuccess)
        return e;
    }
    const TileOperand wo = {wp.w, wp.ld, wp.plane, rows, 0};
    const Planes P = {b + L.p, plane_ld(rows), T * plane_ld(rows)};
    const int tile = entropy_tile(sizeof(X), rows, T, d);
    if (tile == 256)
      e = start_entropy_diff<M, K::split, 256, 256, 2, 4>(wo, xo, kbytes, pairs, y, V, v0, lse,
                                                          dscale<X>(), P, s);
    else if (tile == 128)
      e = start_entropy_diff<M, K::split, 128, 128, 2, 2>(wo, xo, kbytes, pairs, y, V, v0, lse,
                                                          dscale<X>(), P, s);
    else
      e = start_entropy_diff<M, K::split, 64, 64, 2, 2>(wo, xo, kbytes, pairs, y, V, v0, lse,
                                                        dscale<X>(), P, s);
    if (e != hipSuccess) return e;
    if (dX) {
      const bool last = v0 + rows == V;
      const float* prev = v0 > 0 ? acc : nullptr;
      if (last) {
        const PlaneEpilogue ep = {nullptr, wt, nullptr, 1.0f / dscale<X>(), prev, L.ldacc};
        e = launch_plane_product<X, K::f16, false>(d, T, rows, wp, P, pairs, ep, dX, lddx, parts, s);
      } else {
        const PlaneEpilogue ep = {nullptr, nullptr, nullptr, 1.0f, prev, L.ldacc};
        e = launch_plane_product<float, K::f16, false>(d, T, rows, wp, P, pairs, ep, acc, L.ldacc,
                                                       parts, s);
      }
      if (e != hipSuccess) return e;
    }
    if (dW) {
      const PlaneEpilogue ep = {nullptr, nullptr, top, 1.0f / dscale<X>(), nullptr, 0};
      e = launch_plane_product<X, K::f16, true>(d, rows, T, xs, P, pairs, ep, dW + v0 * lddw, lddw,
                                                parts, s);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

#define BK_INST(X)                                                                             \
  template hipError_t launch_entropy<X>(int64_t, int64_t, int64_t, const X*, int64_t,          \
                                        const X*, int64_t, const int64_t*, float*, float*,     \
                                        void*, hipStream_t);                                   \
  template hipError_t launch_entropy_grad<X>(int64_t, int64_t, int64_t, const X*, int64_t,     \
                                             const X*, int64_t, const int64_t*, const float*,  \
                                             const float*, X*, int64_t, X*, int64_t, void*,    \
                                             hipStream_t);
BK_INST(float)
BK_INST(BF16)
BK_INST(F16)
#undef BK_INST

}  // namespace bk
