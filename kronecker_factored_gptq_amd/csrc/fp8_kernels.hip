// 8-bit floating point on gfx950: matrices quantised to e4m3 codes with a float32
// scale for each block of 1 x 128 or 128 x 128, the product of such tokens with such
// weights, for one layer or for groups of tokens with weights of their own, and its input
// gradient.
#include "block_tile.hpp"
#include "fp8_product.hpp"
#include "launch.hpp"

namespace bk {

// ---------------------------------------------------------------------------
// Blocks to e4m3: s = max |x| / 448 (448 = the largest code), at least 2^-126, 1 for an
// all-zero block; code = x / s rounded to nearest even, the division correctly
// rounded. The maximum is taken over the bits of |x|, in which a NaN is larger than
// infinity: a block with either gets it as its scale.
//
// Bound by memory once a division is not the ten instructions of a general one: with r =
// 1 / s correctly rounded, q = x r is within two units of x / s in the last place, q + r (x - q s)
// within one, and the same once more is x / s correctly rounded (Markstein: a faithful quotient
// and a correctly rounded reciprocal give it), the remainders being exact. They are while s >=
// 2^-92: quotients below 2^-11 give the code 0 whatever their last bits, and above it q s
// has no bit below 2^-57 s >= 2^-149. Other scales, those that are not finite among them, divide.
// ---------------------------------------------------------------------------
struct BlockScale {
  float s, r;
  bool fast;
  __device__ inline BlockScale(float top) {
    s = top / 448.0f;
    s = top == 0.0f ? 1.0f : s < 0x1p-126f ? 0x1p-126f : s;
    fast = s >= 0x1p-92f && s <= 0x1p126f;
    r = 1.0f / s;
  }
  __device__ inline float over(float x) const {
    const float q = x * r, u = __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
    return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-u, s, x), r, u), x);  // -0 stays -0
  }
  // four codes
  __device__ inline int codes(const float* x) const {
    float v[4];
    if (fast) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = over(x[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = x[e] / s;
    }
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
  }
};
// The largest |x| of eight elements, as float32 bits (16-bit ones two at a time).
template <typename X> __device__ inline unsigned top8(const Eight<X>& t) {
  unsigned top = 0;
  if constexpr (sizeof(X) == 4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned a = __float_as_uint(to_f32(t.v[e])) & 0x7fffffffu;
      top = a > top ? a : top;
    }
  } else {
    typedef unsigned short v2us __attribute__((ext_vector_type(2)));
    unsigned w[4];
    __builtin_memcpy(w, t.v, 16);
    v2us m = __builtin_bit_cast(v2us, w[0] & 0x7fff7fffu);
#pragma unroll
    for (int i = 1; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(v2us, w[i] & 0x7fff7fffu));
    const unsigned short h = m[0] > m[1] ? m[0] : m[1];
    X x;
    __builtin_memcpy(&x, &h, 2);
    top = __float_as_uint(to_f32(x));
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
// The 128 columns of a block from c on, eight to each of 16 lanes: side by side where rows are
// aligned to them (VEC), else 16 apart, so that a load of all lanes is still one piece of the row
// (eight loads side by side a lane: 4003 x 11009 float32 90 us).
template <typename X, bool VEC>
__device__ inline Eight<X> load_block(const X* row, int64_t c, int64_t n, int l) {
  if (VEC) return load8(row, c + 8 * l, n, true);
  Eight<X> t;
  __builtin_memset(&t, 0, sizeof t);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + 16 * e + l < n) t.v[e] = row[c + 16 * e + l];
  return t;
}
// Their codes; without VEC they change lanes through LDS (`swap`: the 16 lanes' 128 bytes, in
// one wave: no barrier), so that stores are of eight neighbouring codes all the same.
template <typename X, bool VEC>
__device__ inline void store_block(char* row, int64_t c, int64_t n, const Eight<X>& t, int l,
                                   const BlockScale& f, bool vec, char* swap) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = to_f32(t.v[e]);
  int w[2] = {f.codes(v), f.codes(v + 4)};
  if (!VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) swap[16 * e + l] = (char)(w[e / 4] >> 8 * (e % 4));
    __builtin_amdgcn_wave_barrier();
    const int2 x = *(const int2*)(swap + 8 * l);
    __builtin_amdgcn_wave_barrier();
    w[0] = x.x;
    w[1] = x.y;
  }
  c += 8 * l;
  if (vec && c + 8 <= n) {
    *(int2*)(row + c) = int2{w[0], w[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = (char)(w[e / 4] >> 8 * (e % 4));
  }
}

// Blocks of 1 x 128: 16 lanes to kRun neighbouring blocks of a row, a workgroup to 16 rows, so that
// their scales are stored side by side where the scales' rows are, and neighbouring workgroups
// along the rows (8192 x 14336 bfloat16 71.6 us, 4.9 TB/s; rows first 80, a workgroup along one row 76).
constexpr int kRun = 4;
template <typename X, bool VEC>
__global__ __launch_bounds__(256) void quantize_rows_kernel(
    int64_t rows, int64_t n, int64_t runs, const X* __restrict__ x, int64_t ldx, int64_t sX,
    char* __restrict__ q, int64_t ldq, int64_t sQ, float* __restrict__ s, int64_t srow,
    int64_t sblock, int64_t sS, bool vecq) {
  __shared__ __attribute__((aligned(16))) char swap[VEC ? 16 : 16 * kBlock];
  const int64_t band = blockIdx.x / runs, run = blockIdx.x - band * runs;
  const int64_t r = band * 16 + (threadIdx.x >> 4);
  if (r >= rows) return;  // whole groups of 16 lanes
  const int l = threadIdx.x & 15;
  x += blockIdx.y * sX + r * ldx;
  q += blockIdx.y * sQ + r * ldq;
  s += blockIdx.y * sS + r * srow;
  Eight<X> t[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) t[i] = load_block<X, VEC>(x, (run * kRun + i) * kBlock, n, l);
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int64_t b = run * kRun + i;
    if (b * kBlock >= n) break;
    const BlockScale f(__uint_as_float(max_of_16(top8(t[i]))));
    if (l == 0) s[b * sblock] = f.s;
    store_block<X, VEC>(q, b * kBlock, n, t[i], l, f, vecq, swap + (VEC ? 0 : (threadIdx.x >> 4) * kBlock));
  }
}

// Blocks of 128 x 128, a workgroup each, held in registers between the maximum and the codes
// (8192 x 14336 bfloat16 75 us; 4003 x 11009 float32, unaligned rows, 55 from memory, 46 where the
// last-level cache holds some of them).
template <typename X, bool VEC>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(
    int64_t rows, int64_t n, unsigned across, const X* __restrict__ x, int64_t ldx, int64_t sX,
    char* __restrict__ q, int64_t ldq, int64_t sQ, float* __restrict__ s, int64_t srow,
    int64_t sblock, int64_t sS, bool vecq) {
  __shared__ unsigned red[4];
  __shared__ __attribute__((aligned(16))) char swap[VEC ? 16 : 16 * kBlock];
  const int64_t a = blockIdx.x / across, b = blockIdx.x - a * across;
  const int l = threadIdx.x & 15;
  x += blockIdx.y * sX;
  q += blockIdx.y * sQ;
  Eight<X> t[8];
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = a * kBlock + 16 * i + (threadIdx.x >> 4);
    t[i] = load_block<X, VEC>(x + (r < rows ? r : rows - 1) * ldx, b * kBlock, n, l);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned u = top8(t[i]);  // rows past the last count as it, columns past n as zero
    top = u > top ? u : top;
  }
  const BlockScale f(__uint_as_float(max_of_256(top, red)));
  if (threadIdx.x == 0) s[blockIdx.y * sS + a * srow + b * sblock] = f.s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = a * kBlock + 16 * i + (threadIdx.x >> 4);
    if (r < rows)
      store_block<X, VEC>(q + r * ldq, b * kBlock, n, t[i], l, f, vecq,
                          swap + (VEC ? 0 : (threadIdx.x >> 4) * kBlock));
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
#define BK_QUANTIZE(KERNEL, GROUPS, COUNT)                                                        \
  if (vec)                                                                                        \
    hipLaunchKernelGGL((KERNEL<X, true>), dim3((unsigned)(GROUPS), (unsigned)batch), dim3(256), 0, \
                       st, rows, n, COUNT, x, ldx, sX, (char*)q, ldq, sQ, s, srow, sblock, sS,    \
                       vecq);                                                                     \
  else                                                                                            \
    hipLaunchKernelGGL((KERNEL<X, false>), dim3((unsigned)(GROUPS), (unsigned)batch), dim3(256),  \
                       0, st, rows, n, COUNT, x, ldx, sX, (char*)q, ldq, sQ, s, srow, sblock, sS, \
                       vecq)
  if (block_rows == 1) {
    const int64_t runs = (nb + kRun - 1) / kRun;
    BK_QUANTIZE(quantize_rows_kernel, (rows + 15) / 16 * runs, runs);
  } else {
    BK_QUANTIZE(quantize_blocks_kernel, (rows + kBlock - 1) / kBlock * nb, (unsigned)nb);
  }
#undef BK_QUANTIZE
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Y[r][i] = sum over blocks b of k of sx[t][b] sw[i / 128][b] sum_{j in b} Xq[t][j] Wq[i][j],
// t the token of row r, W its group's: tiles of channels x rows. With `splits` ranges of the
// steps (one layer only) their sums go to parts[range]. ANY: operands that the direct loads
// cannot take (8192 x 14336 x 4096 to bfloat16 1457 us with one operand off 16 bytes, 1922 with both).
// 8192 x 14336 x 4096 to bfloat16 456 to 487 us from card to card, 2.0 to 2.1e15
// flop/s (a library's product without block scales reaches 2.6 here); to float32, on the
// float16 instructions, 940 to 990. 4096 tokens to 8 of 64 experts of 2048 x 4096 375 to 433 us, 1.3 to
// 1.5e15 of the products asked for: groups end inside tiles.
// ---------------------------------------------------------------------------
template <class Mul, typename O, int B, int WR, int WC, bool ANY>
__global__ __launch_bounds__(64 * WR * WC) void matmul_fp8_kernel(
    Groups groups, Fp8Tokens X, Fp8Weights W, int64_t n, O* __restrict__ Y, int64_t ldy, bool vec,
    int splits, float* __restrict__ parts, int64_t ldp) {
  typedef BlockTile<Mul, B, WR, WC> TP;
  extern __shared__ char lds[];
  const unsigned nr = (unsigned)((W.m + B - 1) / B);
  const unsigned nc = groups.offsets ? (unsigned)groups.tiles<B>() : (unsigned)((groups.R + B - 1) / B);
  const int range = splits > 1 ? blockIdx.x / (nr * nc) : 0;
  if (blockIdx.x - range * nr * nc >= nr * nc) return;
  int tr, tc;
  tile_of(blockIdx.x - range * nr * nc, nr, nc, tr, tc);
  int64_t group = 0, c0 = (int64_t)tc * B, cols = groups.R - c0;
  if (groups.offsets && !groups.tile<B>(tc, group, c0, cols)) return;
  cols = cols < B ? cols : B;
  const int64_t r0 = (int64_t)tr * B, rows = W.m - r0 < B ? W.m - r0 : B;
  const int lane = threadIdx.x & 63, wave = TP::wave();
  const int total = (int)((n + kStepBytes - 1) / kStepBytes);
  TP tp;
  tp.zero();
  // Rows without a token are 0 whatever the weights hold (0 times a NaN code or a scale that is not
  // finite is NaN): before the sums of any range of k leave.
  auto clear = [&]() {
    if (!X.order) return;
#pragma unroll
    for (int j = 0; j < TP::FC; ++j) {
      const int col = tp.wave_c() + j * 16 + (lane & 15);
      if (X.token(c0 + (col < (int)cols ? col : (int)cols - 1)) >= 0) continue;
#pragma unroll
      for (int i = 0; i < TP::FR; ++i) tp.acc[i][j] = f32x4{0, 0, 0, 0};
    }
  };
  if constexpr (ANY) {
    const char* w = W.p + group * W.stride + r0 * W.ld;
    const float* sw = W.s + group * W.strides + (r0 + tp.wave_r() < W.m ? r0 + tp.wave_r() : W.m - 1) / kBlock * W.lds;
    auto token = [&](int col) { return X.token(c0 + (col < (int)cols ? col : (int)cols - 1)); };
    tp.run_any(
        total, lds,
        [&](int s, int row) {
          return typename TP::Bytes{w + (row < (int)rows ? row : (int)rows - 1) * W.ld, (int64_t)s * kBlock, n};
        },
        [&](int s, int col) {
          const int64_t t = token(col);
          return typename TP::Bytes{t < 0 ? nullptr : X.p + t * X.ld, (int64_t)s * kBlock, n};
        },
        [&](int s, int j) {
          const int64_t t = token(tp.wave_c() + j * 16 + (lane & 15));
          return t < 0 ? 0.0f : X.s[t * X.st + s * X.sb] * sw[s];
        });
    clear();
    store_tile(tp, r0, c0, W.m, c0 + cols, Y, ldy, vec, [](float a, int, int, int) { return a; });
    return;
  }
  typename TP::Side R, C;
  const int s0 = (int)((int64_t)total * range / splits), s1 = (int)((int64_t)total * (range + 1) / splits);
  const int64_t words = (n + 3) / 4 * 4;  // of the last row no word is read that holds none of it
  R.init(W.p + group * W.stride + r0 * W.ld, (int)((rows - 1) * W.ld + words), n, 0, s0,
         [&](int row) { return (row < (int)rows ? row : (int)rows - 1) * (int)W.ld; });
  // the token of a tile's column: its offset in rows from `first`, -1 if none
  const int64_t first = X.order ? 0 : c0;
  auto token = [&](int col) {
    col = col < (int)cols ? col : (int)cols - 1;
    return X.order ? (int)X.token(c0 + col) : col;
  };
  const int64_t last_row = X.order ? (X.T > 0 ? X.T - 1 : 0) : cols - 1;
  C.init(X.p + first * X.ld, (int)(last_row * X.ld + words), n, 0, s0, [&](int col) {
    const int t = token(col);
    return t < 0 ? TP::kNone : t * (int)X.ld;
  });
  const char* scale;
  int per;
  if (wave < B / 64) {
    const int t = token(wave * 64 + lane);
    scale = (const char*)(X.s + first * X.st);
    per = t < 0 ? TP::kNone : t * (int)X.st * 4;
  } else {
    const int last = (int)((rows - 1) / kBlock);
    scale = (const char*)(W.s + group * W.strides + r0 / kBlock * W.lds);
    per = (lane < last ? lane : last) * (int)W.lds * 4;
  }
  tp.run(R, C, scale, per, (wave < B / 64 ? X.sb : 1) * 4, s0, s1, lds,
         n % 16 && s1 == total ? (int)(n % kStepBytes) : 0);
  clear();
  if (splits > 1) {
    store_sums(tp, r0, c0, groups.R, parts + range * groups.R * ldp, ldp);
    return;
  }
  store_tile(tp, r0, c0, W.m, c0 + cols, Y, ldy, vec, [](float a, int, int, int) { return a; });
}

// The ranges' sums; four channels of one row a thread (join_ranges).
template <typename O, int S>
__global__ __launch_bounds__(256) void join_fp8_kernel(int64_t m, int64_t R, int splits,
                                                       const float* __restrict__ parts, int64_t ldp,
                                                       O* __restrict__ Y, int64_t ldy, bool vec) {
  __shared__ f32x4 red[S > 1 ? 256 : 1];
  const int64_t per = ldp / 4, at = JoinAt<S>::at();
  const int64_t t = at / per, r = (at - t * per) * 4;
  f32x4 a;
  if (!join_ranges<S>(parts + t * ldp + r, R * ldp, splits, at < R * per, a, red)) return;
  O y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = from_f32<O>(a[e]);
  if (vec && r + 4 <= m) {
    *(typename Vec4<O>::type*)(Y + t * ldy + r) = __builtin_bit_cast(typename Vec4<O>::type, y);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r + e < m) Y[t * ldy + r + e] = y[e];
  }
}

template <typename O>
static hipError_t join_fp8(int64_t m, int64_t R, int splits, const float* parts, int64_t ldp, O* Y,
                           int64_t ldy, bool vec, hipStream_t s) {
  const int64_t four = R * (ldp / 4);
#define BK_JOIN(S)                                                                             \
  hipLaunchKernelGGL((join_fp8_kernel<O, S>),                                                  \
                     dim3((unsigned)((four + 256 / S - 1) / (256 / S))), dim3(256), 0, s, m, R, \
                     splits, parts, ldp, Y, ldy, vec)
  if (join_slices(splits) == 1) BK_JOIN(1);
  else BK_JOIN(8);
#undef BK_JOIN
  return hipGetLastError();
}

// Rows that do not start on 16 bytes, of a length that is no multiple of 16, are copied to
// zero-padded lines first, 16 bytes a thread: the tokens', and behind them every expert's.
__global__ __launch_bounds__(256) void pack_fp8_kernel(Fp8Tokens X, Fp8Weights W, int64_t experts,
                                                       int64_t n, char* __restrict__ px,
                                                       char* __restrict__ pw, int64_t ldp) {
  const int64_t per = ldp / 16, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t r = at / per;
  const int64_t k = (at - r * per) * 16;
  const char* row;
  char* to;
  if (r < X.T) {
    row = X.p + r * X.ld;
    to = px + r * ldp;
  } else {
    r -= X.T;
    if (r >= experts * W.m) return;
    const int64_t e = r / W.m;
    row = W.p + e * W.stride + (r - e * W.m) * W.ld;
    to = pw + r * ldp;
  }
  *(v4i*)(to + k) = load_any<1>(row, k, n);
}

// ---------------------------------------------------------------------------
// Few rows: bound by reading the weights once. A workgroup of 8 waves takes 16 RT channels of
// one layer and all of its rows, 16 NT at a time; its waves divide k between them, U blocks
// a turn, straight from memory to registers with the next turn on its way, and their
// sums meet in LDS (skinny_product.hpp, with the blocks' scales). Every result type takes the
// float16 instructions, exact products and float32 sums: the 8-bit ones' coarser sums (MulFP8) would buy
// 0 to 4 % here (14336 x 4096, one row: 14.1 and 14.7 us a call; 256 rows of 64 experts of 2048 x 4096
// 104.0 and 106.2). Grid: channels x (tiles of rows, or experts). One row: 4096 x 4096 5.8 us on the GPU,
// 14336 x 4096 14.7 us a call among others (4.0 TB/s); 256 rows of 64 experts of 2048 x 4096 102 to 110
// us from card to card (4.9 to 5.3 TB/s).
// ---------------------------------------------------------------------------
template <typename O, int RT, int NT, int U, bool ANY>
__global__ __launch_bounds__(512) void skinny_fp8_kernel(Groups groups, Fp8Tokens X, Fp8Weights W,
                                                         int64_t n, O* __restrict__ Y, int64_t ldy,
                                                         bool vec) {
  constexpr int kWaves = 8, kTiles = RT * NT, kCols = 16 * NT;
  static_assert(kTiles <= kWaves, "a wave to each tile");
  __shared__ f32x4 lds[kWaves * kTiles * 64];
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t group = 0, c0 = (int64_t)blockIdx.y * kCols, end = groups.R;
  if (groups.offsets) {
    group = blockIdx.y;
    int before = 0, a, rows;
    for (int64_t e0 = 0;; e0 += 64) {
      groups.ranges(e0, before, a, rows);
      if (group < e0 + 64) break;
    }
    const int l = (int)(group & 63);
    c0 = Groups::lane_of(a, l);
    end = c0 + Groups::lane_of(rows, l);
  } else {
    end = c0 + kCols < end ? c0 + kCols : end;
  }
  const int64_t r0 = (int64_t)blockIdx.x * (16 * RT);
  const char* pr[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t r = r0 + 16 * i + r16;
    pr[i] = W.p + group * W.stride + (r < W.m ? r : W.m - 1) * W.ld;
  }
  const float* sw = W.s + group * W.strides + r0 / kBlock * W.lds;  // one block of rows: 16 RT divides 128
  const int nb = (int)((n + kBlock - 1) / kBlock);
  auto load = [&](const char* row, int64_t k) {
    if (ANY) return load_any<1>(row, k, n);
    return k < n ? *(const v4i*)(row + k) : v4i{0, 0, 0, 0};
  };
  for (; c0 < end; c0 += kCols) {
    const char* pc[NT];
    const float* ps[NT];
    bool has[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t c = c0 + 16 * j + r16, t = X.token(c < end ? c : end - 1);
      has[j] = t >= 0;
      pc[j] = X.p + (has[j] ? t : 0) * X.ld;
      ps[j] = X.s + (has[j] ? t : 0) * X.st;
    }
    f32x4 acc[RT][NT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    struct Turn {
      v4i a[U][RT][2], b[U][NT][2];
      float f[U][NT], w[U];
    };
    auto read = [&](Turn& t, int b0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t k = (int64_t)(b0 + u) * kBlock + 16 * q;
        const int b = b0 + u < nb ? b0 + u : nb - 1;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          t.a[u][i][0] = load(pr[i], k);
          t.a[u][i][1] = load(pr[i], k + 64);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          t.b[u][j][0] = load(pc[j], k);
          t.b[u][j][1] = load(pc[j], k + 64);
          t.f[u][j] = ps[j][b * X.sb];
        }
        t.w[u] = sw[b];
      }
    };
    auto multiply = [&](const Turn& t, int b0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (b0 + u >= nb) break;  // nothing, but for a scale that is not finite
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float f = has[j] ? t.f[u][j] * t.w[u] : 0.0f;
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const f32x4 p = MulFP8Exact::block(t.a[u][i][0], t.a[u][i][1], t.b[u][j][0], t.b[u][j][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i][j][e] = __builtin_fmaf(has[j] ? p[e] : 0.0f, f, acc[i][j][e]);
          }
        }
      }
    };
    int b = wave * U;
    if (b < nb) {
      Turn x, y;
      read(x, b);
      while (b + kWaves * U < nb) {
        read(y, b + kWaves * U);
        multiply(x, b);
        b += kWaves * U;
        if (b + kWaves * U >= nb) {
          x = y;
          break;
        }
        read(x, b + kWaves * U);
        multiply(y, b);
        b += kWaves * U;
      }
      multiply(x, b);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) lds[(wave * kTiles + i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    if (wave < kTiles) {
      f32x4 sum = lds[wave * 64 + lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += lds[(w * kTiles + wave) * 64 + lane];
      const int64_t c = c0 + wave % NT * 16 + r16, r = r0 + wave / NT * 16 + 4 * q;
      if (c < end && r < W.m) {
        O y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = from_f32<O>(sum[e]);
        if (vec && r + 4 <= W.m) {
          *(typename Vec4<O>::type*)(Y + c * ldy + r) = __builtin_bit_cast(typename Vec4<O>::type, y);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (r + e < W.m) Y[c * ldy + r + e] = y[e];
        }
      }
    }
    __syncthreads();  // the sums were read: the next rows' may be written
  }
}

// Whether the kernel above takes a call. Of one layer as many rows as the int8 product's takes
// (4096 x 4096, 64 rows: 12.9 us against 15.4 of tiles; 14336 x 4096, 16 and 32 rows: 14.8 and 22.9 against
// 18.2 and 20.8). Of experts, whose number of rows each is
// not known here, up to 8 on average where k is long enough for eight waves: 2048 x 4096 of 64
// experts, f16, 1 / 4 / 8 / 16 rows each on average 80 / 106 / 119 / 167 us against 96 / 143 / 129 / 132 of
// tiles; 4096 x 1024 of 16, 2 / 8 / 32 rows: 20 / 22 / 45 against 14.9 / 15.8 / 20.3. One expert with far
// more than the average is gone through 16 rows at a time by its own workgroups alone: all of 512 rows
// to one of the 64 take 320 us, even ones 118.
static bool fp8_skinny(int64_t R, int64_t experts, int64_t m, int64_t n) {
  if (experts == 1) return R <= (m * n <= (1 << 24) ? 64 : m * n <= (1 << 26) ? 16 : 8);
  return R <= 8 * experts && n >= 2048;
}
template <typename O, bool ANY>
static hipError_t start_skinny_fp8(const Groups& groups, const Fp8Tokens& X, const Fp8Weights& W,
                                   int64_t n, O* Y, int64_t ldy, hipStream_t s) {
  const bool vec = vec4_ok(Y, ldy);
  // rows at a time; channels a workgroup, more where that leaves nearly every CU one: the rows
  // are then read less often (measured on the 8-bit instructions: 14336 x 4096, one row: 13.9 us with 64
  // channels, 15.1 with 16; 4096 x 14336 30.8 and 12.8; 64 experts of 2048 x 4096, 256 rows: 104 with
  // 64, 116 with 32, 122 with 16)
  const int64_t each = (groups.R + groups.count - 1) / groups.count;
  const int nt = each > 32 ? 4 : each > 16 ? 2 : 1;
  const int64_t work = W.m * (groups.offsets ? groups.count : (groups.R + 16 * nt - 1) / (16 * nt));
  const int rt = work >= 64 * 192 ? 4 : work >= 32 * 192 ? 2 : 1;
#define BK_SKINNY(RT, NT, U)                                                                   \
  hipLaunchKernelGGL(                                                                          \
      (skinny_fp8_kernel<O, RT, NT, U, ANY>),                                             \
      dim3((unsigned)((W.m + 16 * RT - 1) / (16 * RT)),                                        \
           (unsigned)(groups.offsets ? groups.count : (groups.R + 16 * NT - 1) / (16 * NT))),  \
      dim3(512), 0, s, groups, X, W, n, Y, ldy, vec)
  if (nt == 1) {
    if (rt == 4) BK_SKINNY(4, 1, 1);
    else if (rt == 2) BK_SKINNY(2, 1, 2);
    else BK_SKINNY(1, 1, 2);
  } else if (nt == 2) {
    if (rt >= 2) BK_SKINNY(2, 2, 1);
    else BK_SKINNY(1, 2, 2);
  } else {
    BK_SKINNY(1, 4, 1);
  }
#undef BK_SKINNY
  return hipGetLastError();
}

static inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
static int64_t packed_ld(int64_t n) { return (n + kStepBytes - 1) / kStepBytes * kStepBytes; }
static TilePlan fp8_plan(int es, int64_t R, int64_t m, int64_t n) {
  TilePlan p = plan_tiles(m, R, (n + kStepBytes - 1) / kStepBytes, 1, false, true,
                          es == 4 ? &kCostsExact : &kCostsBlocks);
  if (es == 4 && p.tile == 256) p.tile = 128;
  return p;
}
// Of groups, whose sizes are not known here, `a` rows of the tiles' other operand and `steps`: tiles of
// 64 below `few` rows each on average (64 experts of 2048 x 4096, us with 64 and 128: 8 rows each 129
// and 136, 32 161 and 142, 128 233 and 179; 32 of 1024 x 2048: 64 rows 22 and 25, 128 33 and 28;
// gradient of 32 of 4096 x 2048: 64 rows 108 and 112, 128 163 and 145), then 128 or 256 by the rounds of
// tiles, half a round of them empty, if every group leaves half a tile empty; a round of 256 is
// `ratio` as long as one of 128 and fills its ring for four steps more (64 experts, 128 and 256:
// 192 rows 223 and 230, 256 271 and 239, 1024 824 and 748; 8 of 4096 x 1024, 1024 rows 83 and 90; gradient
// 128 rows 145 and 227, 512 355 and 372).
static TilePlan group_plan(int64_t R, int64_t experts, int64_t a, int64_t steps, int64_t few, double ratio) {
  if (R < few * experts) return {64, 1};
  auto time = [&](int64_t B, double at_once, double fill) {
    const int64_t half = R / B + experts / 2;
    const double tiles = (double)((a + B - 1) / B * (half > experts ? half : experts));
    return (tiles / at_once + 0.5) * ((double)steps + fill);
  };
  return {time(256, 256, 6) * ratio < time(128, 512, 2) ? 256 : 128, 1};
}
static TilePlan fp8_plan(int es, int64_t R, int64_t experts, int64_t m, int64_t n, bool grouped) {
  return grouped ? group_plan(R, experts, m, (n + 127) / 128, 32, es == 4 ? 1e9 : 1.39) : fp8_plan(es, R, m, n);
}
struct Fp8Offsets {
  size_t x, w, parts, total;
};
static Fp8Offsets fp8_offsets(int es, int64_t T, int64_t R, int64_t experts, int64_t m, int64_t n, bool aligned) {
  const bool skinny = fp8_skinny(R, experts, m, n), packs = n % 16 != 0 && !aligned && !skinny;
  Fp8Offsets o;
  o.x = 0;
  o.w = o.x + up256(packs ? (size_t)(T * packed_ld(n)) : 0);
  o.parts = o.w + up256(packs ? (size_t)(experts * m * packed_ld(n)) : 0);
  // with one expert the call may or may not be by groups
  o.total = o.parts + (experts == 1 && !skinny ? (size_t)split_words(m, R, fp8_plan(es, R, m, n).splits) * 4 : 0);
  return o;
}
size_t matmul_fp8_bytes(int es, int64_t T, int64_t R, int64_t experts, int64_t m, int64_t n, bool aligned) {
  return fp8_offsets(es, T, R, experts, m, n, aligned).total;
}

template <class Mul, typename O, int B, int WR, int WC, bool ANY = false>
static hipError_t start_fp8_tile(const Groups& groups, const Fp8Tokens& X, const Fp8Weights& W,
                                 int64_t n, O* Y, int64_t ldy, int splits, float* parts,
                                 hipStream_t s) {
  typedef BlockTile<Mul, B, WR, WC> TP;
  auto* k = matmul_fp8_kernel<Mul, O, B, WR, WC, ANY>;
  constexpr int lds = ANY ? TP::kAnyLds : TP::kLds;
  if (lds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t tiles = (W.m + B - 1) / B * groups.most(B), ldp = (W.m + 3) / 4 * 4;
  const bool vec = vec4_ok(Y, ldy);
  hipLaunchKernelGGL(k, dim3((unsigned)(tiles * splits)), dim3(TP::kThreads), lds, s, groups, X,
                     W, n, Y, ldy, vec, splits, parts, ldp);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  return join_fp8(W.m, groups.R, splits, parts, ldp, Y, ldy, vec, s);
}

// Whether the direct loads can take the operands: rows on 16 bytes, and 32-bit offsets, which an order
// needs to all tokens (8192 rows of 500000 tokens of 4096 bytes 143 us, of 530000, beyond 2 GiB, 719).
static bool on_16(const Fp8Tokens& X, const Fp8Weights& W) {
  return fp8_rows_on_16(X.p, X.ld, 0) && fp8_rows_on_16(W.p, W.ld, W.stride);  // 0 where there is one row or expert
}
static bool fp8_direct(const Fp8Tokens& X, const Fp8Weights& W, int64_t n) {
  const int64_t kMost = (int64_t)1 << 31;
  const int64_t reach = X.order ? X.T : 256;
  return on_16(X, W) && W.ld <= kTileMaxLd && reach * X.ld + n + 16 < kMost &&
         reach * X.st * 4 < kMost && W.lds * 8 < kMost;
}

template <typename O>
hipError_t launch_matmul_fp8(int64_t T, int64_t R, int64_t experts, int64_t m, int64_t n,
                             const uint8_t* Xq, int64_t ldx, const float* sx, int64_t sx_token,
                             int64_t sx_block, const uint8_t* Wq, int64_t ldw, int64_t stride_w,
                             const float* sw, int64_t ldsw, int64_t stride_sw,
                             const int32_t* offsets, const int32_t* order, int64_t per_token, O* Y,
                             int64_t ldy, void* ws, hipStream_t s) {
  if (R <= 0 || m <= 0) return hipSuccess;
  typedef typename std::conditional<sizeof(O) == 4, MulFP8Exact, MulFP8>::type Mul;
  const Groups groups = {offsets, experts, R};
  Fp8Tokens X = {(const char*)Xq, T > 1 ? ldx : 0, T, sx, sx_token, sx_block, order, per_token};
  Fp8Weights W = {(const char*)Wq, m > 1 ? ldw : 0, experts > 1 ? stride_w : 0, m, sw, ldsw, stride_sw};
  if (T == 0) {  // rows without a token read one all the same: readable memory of that size
    X.p = W.p;
    X.ld = W.ld;
    X.s = W.s;
    X.st = 0;
    X.sb = 1;
  }
  if (fp8_skinny(R, experts, m, n))
    return n % 16 == 0 && fp8_direct(X, W, n) ? start_skinny_fp8<O, false>(groups, X, W, n, Y, ldy, s)
                                              : start_skinny_fp8<O, true>(groups, X, W, n, Y, ldy, s);
  const bool aligned = on_16(X, W);
  const Fp8Offsets o = fp8_offsets(sizeof(O), T, R, experts, m, n, aligned);
  if (n % 16 && !aligned) {
    const int64_t ld = packed_ld(n);
    char *px = (char*)ws + o.x, *pw = (char*)ws + o.w;
    hipLaunchKernelGGL(pack_fp8_kernel,
                       dim3((unsigned)(((T + experts * m) * (ld / 16) + 255) / 256)), dim3(256), 0,
                       s, X, W, experts, n, px, pw, ld);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    X.p = px;
    W.p = pw;
    X.ld = W.ld = ld;
    W.stride = m * ld;
    n = (n + 15) / 16 * 16;
  }
  float* parts = (float*)((char*)ws + o.parts);
  if (!fp8_direct(X, W, n))
    return start_fp8_tile<Mul, O, 64, 2, 2, true>(groups, X, W, n, Y, ldy, 1, parts, s);
  const TilePlan plan = fp8_plan(sizeof(O), R, experts, m, n, offsets != nullptr);
  if constexpr (sizeof(O) != 4) {
    if (plan.tile == 256)
      return start_fp8_tile<Mul, O, 256, 2, 4>(groups, X, W, n, Y, ldy, 1, parts, s);
  }
  if (plan.tile == 128)
    return start_fp8_tile<Mul, O, 128, 2, 2>(groups, X, W, n, Y, ldy, plan.splits, parts, s);
  return start_fp8_tile<Mul, O, 64, 2, 2>(groups, X, W, n, Y, ldy, plan.splits, parts, s);
}

// ---------------------------------------------------------------------------
// dX[r][j] = sum_i G[r][i] sw[i / 128][j / 128] Wq[i][j]: tiles of columns j x rows r, the codes
// k-major and made 16-bit in registers (BlockTile, kTransposed). A bfloat16 or float16 G is
// multiplied as it is, a float32 one as its three bfloat16 planes, one after the other
// over all of k. With `splits` ranges of the steps (one layer only) their sums go to
// parts[range]. 8192 x 4096 x 14336 bfloat16 860 to 935 us from card to card (1.0 to 1.1 PFLOP/s; a
// library's 16-bit product of two matrices reaches 1.6); 4096 tokens to 4 of 32 experts of 4096 x 2048 330 to
// 350 us (0.82). ANY: G or codes off 16 bytes (2740 us and more for the former).
// ---------------------------------------------------------------------------
struct Fp8Gradient {
  const char* p;
  int64_t ld, plane;  // bytes
};
template <class Mul, typename O, int B, int WR, int WC, bool ANY, int DEEP>
__global__ __launch_bounds__(64 * WR * WC) void matmul_fp8_grad_kernel(
    Groups groups, Fp8Gradient G, Fp8Weights W, int64_t n, O* __restrict__ dX, int64_t ldx,
    bool vec, int splits, float* __restrict__ parts, int64_t ldp) {
  typedef BlockTile<Mul, B, WR, WC, DEEP> TP;
  extern __shared__ char lds[];
  const unsigned nr = (unsigned)((n + B - 1) / B);
  const unsigned nc = groups.offsets ? (unsigned)groups.tiles<B>() : (unsigned)((groups.R + B - 1) / B);
  const int range = splits > 1 ? blockIdx.x / (nr * nc) : 0;
  if (blockIdx.x - range * nr * nc >= nr * nc) return;
  int tr, tc;
  tile_of(blockIdx.x - range * nr * nc, nr, nc, tr, tc);
  int64_t group = 0, c0 = (int64_t)tc * B, cols = groups.R - c0;
  if (groups.offsets && !groups.tile<B>(tc, group, c0, cols)) return;
  cols = cols < B ? cols : B;
  const int64_t r0 = (int64_t)tr * B, rows = n - r0 < B ? n - r0 : B;
  const int lane = threadIdx.x & 63;
  const int64_t kbytes = (W.m + 7) / 8 * 16;  // whole chunks: G's rows are zero up to them
  const int64_t total = (kbytes + kStepBytes - 1) / kStepBytes * Mul::kPlanes;
  const int s0 = (int)(total * range / splits), s1 = (int)(total * (range + 1) / splits);
  const int last = (int)((rows - 1) / kBlock);
  TP tp;
  tp.zero();
  if constexpr (ANY) {
    const char* w = W.p + group * W.stride + r0;
    const int block = tp.wave_r() / kBlock;
    const float* sw = W.s + group * W.strides + r0 / kBlock + (block < last ? block : last);
    const int64_t each = total / Mul::kPlanes;
    tp.run_any(
        (int)total, lds,
        [&](int s, int k) {
          const int64_t i = s % each * 64 + k;
          return typename TP::Bytes{i < W.m ? w + i * W.ld : nullptr, 0, rows};
        },
        [&](int s, int col) {
          const int64_t c = c0 + (col < (int)cols ? col : (int)cols - 1);
          return typename TP::Bytes{G.p + s / each * G.plane + c * G.ld, s % each * kStepBytes, W.m * 2};
        },
        [&](int s, int) { return sw[s % each / 2 * W.lds]; });
    store_tile(tp, r0, c0, n, c0 + cols, dX, ldx, vec, [](float a, int, int, int) { return a; });
    return;
  }
  typename TP::SideR R;
  typename TP::Side C;
  R.init(W.p + group * W.stride + r0, W.ld, W.m, (int)rows, s0);
  C.init(G.p + c0 * G.ld, (int)((cols - 1) * G.ld + kbytes), kbytes, G.plane, s0,
         [&](int col) { return (col < (int)cols ? col : (int)cols - 1) * (int)G.ld; });
  tp.run(R, C, (const char*)(W.s + group * W.strides + r0 / kBlock), (lane < last ? lane : last) * 4,
         W.lds * 4, s0, s1, lds);
  if (splits > 1) {
    store_sums(tp, r0, c0, groups.R, parts + range * groups.R * ldp, ldp);
    return;
  }
  store_tile(tp, r0, c0, n, c0 + cols, dX, ldx, vec, [](float a, int, int, int) { return a; });
}

// The operands that the tiles cannot read as they are, laid out by one launch: a float32 G as
// three bfloat16 planes, a 16-bit one whose rows are no multiple of 8 long in zero-padded lines; behind
// it codes whose rows are no multiple of 16 long and do not start on 16 bytes, in zero-padded lines
// (two launches: 333 x 1000 x 1531 float32 26.7 us, one 24.9).
struct Fp8Layout {
  char* g;  // null: as it is
  int64_t ldg, plane, blocks;
  char* w;
  int64_t ldw, rows;
};
template <typename G>
__global__ __launch_bounds__(256) void grad_layout_kernel(int64_t R, int64_t m, int64_t n,
                                                          const G* __restrict__ g, int64_t ldg,
                                                          Fp8Weights W, Fp8Layout to, bool vec) {
  if ((int64_t)blockIdx.x < to.blocks) {
    const int64_t per = to.ldg / 16, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t r = at / per, c = (at - r * per) * 8;
    if (r >= R) return;
    const Eight<G> t = load8(g + r * ldg, c, m, vec);
    char* p = to.g + r * to.ldg + c * 2;
    if constexpr (sizeof(G) == 4) {
      unsigned short w[3][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        unsigned short x[3];
        split16<kBF16x3>(to_f32(t.v[e]), x);
#pragma unroll
        for (int i = 0; i < 3; ++i) w[i][e] = x[i];
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) *(v4i*)(p + i * to.plane) = __builtin_bit_cast(v4i, w[i]);
    } else {
      *(v4i*)p = __builtin_bit_cast(v4i, t);
    }
    return;
  }
  const int64_t per = to.ldw / 16, at = (int64_t)(blockIdx.x - to.blocks) * 256 + threadIdx.x;
  const int64_t r = at / per, k = (at - r * per) * 16;
  if (r >= to.rows) return;
  const int64_t z = r / W.m;
  *(v4i*)(to.w + r * to.ldw + k) = load_any<1>(W.p + z * W.stride + (r - z * W.m) * W.ld, k, n);
}

static TilePlan fp8_grad_plan(int es, int64_t R, int64_t experts, int64_t m, int64_t n, bool grouped) {
  return grouped ? group_plan(R, experts, n, (m + 63) / 64, 65, 1.61)
                 : plan_tiles(n, R, (m + 63) / 64, es == 4 ? 3 : 1, false, true, &kCostsBlocks);
}
struct Fp8GradOffsets {
  size_t w, g, parts, total;
};
static Fp8GradOffsets fp8_grad_offsets(int es, int64_t R, int64_t experts, int64_t m, int64_t n, bool aligned) {
  Fp8GradOffsets o;
  o.w = 0;
  o.g = o.w + up256(n % 16 && !aligned ? (size_t)(experts * m * packed_ld(n)) : 0);
  o.parts = o.g + up256(es == 4 ? (size_t)(3 * R * plane_ld(m)) : m % 8 ? (size_t)(R * plane_ld(m)) : 0);
  o.total = o.parts + (experts == 1 ? (size_t)split_words(n, R, fp8_grad_plan(es, R, 1, m, n, false).splits) * 4 : 0);
  return o;
}
size_t matmul_fp8_grad_bytes(int es, int64_t R, int64_t experts, int64_t m, int64_t n, bool aligned) {
  return fp8_grad_offsets(es, R, experts, m, n, aligned).total;
}

template <class Mul, typename O, int B, int WR, int WC, bool ANY = false, int DEEP = 3>
static hipError_t start_fp8_grad(const Groups& groups, const Fp8Gradient& G, const Fp8Weights& W,
                                 int64_t n, O* dX, int64_t ldx, int splits, float* parts,
                                 hipStream_t s) {
  typedef BlockTile<Mul, B, WR, WC, DEEP> TP;
  auto* k = matmul_fp8_grad_kernel<Mul, O, B, WR, WC, ANY, DEEP>;
  constexpr int lds = ANY ? TP::kAnyLds : TP::kLds;
  if (lds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t tiles = (n + B - 1) / B * groups.most(B), ldp = (n + 3) / 4 * 4;
  const bool vec = vec4_ok(dX, ldx);
  hipLaunchKernelGGL(k, dim3((unsigned)(tiles * splits)), dim3(TP::kThreads), lds, s, groups, G,
                     W, n, dX, ldx, vec, splits, parts, ldp);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  return join_fp8(n, groups.R, splits, parts, ldp, dX, ldx, vec, s);
}

template <typename G>
hipError_t launch_matmul_fp8_grad(int64_t R, int64_t experts, int64_t m, int64_t n, const G* g,
                                  int64_t ldg, const uint8_t* Wq, int64_t ldw, int64_t stride_w,
                                  const float* sw, int64_t ldsw, int64_t stride_sw,
                                  const int32_t* offsets, G* dX, int64_t ldx, void* ws,
                                  hipStream_t s) {
  if (R <= 0 || n <= 0) return hipSuccess;
  constexpr bool wide = sizeof(G) == 4;
  typedef MulWide<typename std::conditional<std::is_same<G, F16>::value, MmaF16, MmaBF16>::type, wide ? 3 : 1> Mul;
  const Groups groups = {offsets, experts, R};
  Fp8Weights W = {(const char*)Wq, m > 1 ? ldw : 0, experts > 1 ? stride_w : 0, m, sw, ldsw, stride_sw};
  const bool aligned = fp8_rows_on_16(W.p, W.ld, W.stride);
  const Fp8GradOffsets o = fp8_grad_offsets(sizeof(G), R, experts, m, n, aligned);
  char* b = (char*)ws;
  Fp8Gradient x = {(const char*)g, ldg * (int64_t)sizeof(G), 0};
  const bool lay_g = (wide || m % 8) && m > 0;
  const bool lay_w = n % 16 && !aligned && m > 0;
  if (lay_g || lay_w) {
    Fp8Layout to = {nullptr, plane_ld(m), R * plane_ld(m), 0, b + o.w, packed_ld(n), lay_w ? experts * m : 0};
    if (lay_g) {
      to.g = b + o.g;
      to.blocks = (R * (to.ldg / 16) + 255) / 256;
      x = {to.g, to.ldg, wide ? to.plane : 0};
    }
    const int64_t blocks = to.blocks + (to.rows * (to.ldw / 16) + 255) / 256;
    hipLaunchKernelGGL(grad_layout_kernel<G>, dim3((unsigned)blocks), dim3(256), 0, s, R, m, n, g, ldg,
                       W, to, load8_ok(g, ldg));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (lay_w) {
      W.p = to.w;
      W.ld = to.ldw;
      W.stride = m * W.ld;
    }
  }
  float* parts = (float*)(b + o.parts);
  // 16-byte rows and 32-bit offsets
  if (((uintptr_t)W.p | W.ld | W.stride | (uintptr_t)x.p | x.ld | x.plane) % 16 != 0 ||
      W.ld > kTileMaxLd || x.ld > kTileMaxLd)
    return start_fp8_grad<Mul, G, 64, 2, 2, true>(groups, x, W, n, dX, ldx, 1, parts, s);
  const TilePlan plan = fp8_grad_plan(sizeof(G), R, experts, m, n, offsets != nullptr);
  if (plan.tile == 256)
    return start_fp8_grad<Mul, G, 256, 2, 4>(groups, x, W, n, dX, ldx, 1, parts, s);
  if (plan.tile == 128) {
    // more tiles than two a CU: three, with two steps in the ring (4096 tokens to 4 of 32 experts, 4096
    // x 2048 bfloat16: 356 -> 338 us; with one tile a CU the shorter ring is slower: 777 x 4096 x 4096
    // 44.5 and 50.3)
    const int64_t tiles = (n + 127) / 128 * ((R + 127) / 128 + (offsets ? experts / 2 : 0)) * plan.splits;
    if (tiles > 512)
      return start_fp8_grad<Mul, G, 128, 2, 2, false, 2>(groups, x, W, n, dX, ldx, plan.splits, parts, s);
    return start_fp8_grad<Mul, G, 128, 2, 2>(groups, x, W, n, dX, ldx, plan.splits, parts, s);
  }
  return start_fp8_grad<Mul, G, 64, 2, 2>(groups, x, W, n, dX, ldx, plan.splits, parts, s);
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
