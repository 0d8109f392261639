// The 8-bit product on gfx950: tokens quantised to int8 with a scale each, the
// product of the int8 tokens with a layer's int8 codes (the solve's V), scaled
// per token and output channel, and its input gradient.
#include "launch.hpp"
#include "skinny_product.hpp"
#include "tile_product.hpp"

namespace bk {

// ---------------------------------------------------------------------------
// Tokens to int8: x = X[t][j] * c[j] in float32, s = max_j |x| / 127 (1 for an
// all-zero token), q = clamp(rint(x / s), -127, 127), the division correctly
// rounded as in the solve's quantizer. The maximum is taken over the bits of
// |x|, in which a NaN is larger than infinity: a token with an infinity or a
// NaN gets that as its scale, and codes whose products it makes NaN.
//
// Bound by memory. A workgroup keeps its row in registers between the maximum and
// the codes, so that the row is read once (8192 x 14336 float32: 146 us, 4.0 TB/s,
// a large copy reaching 5.0; reading it twice took 253). Eight elements to a
// thread's group make 8-byte stores of codes; groups of four (4-byte stores) took
// 171 us, groups of sixteen (half the workgroups on a CU) 176, and a multiplication
// by 1 / s with a division near ties only 161. One token of 4096: 3.4 us.
// ---------------------------------------------------------------------------
template <typename X, int NV>
__global__ __launch_bounds__(256) void quantize_tokens_kernel(
    int64_t n, const X* __restrict__ x, int64_t ldx, const float* __restrict__ c,
    signed char* __restrict__ q, int64_t ldq, float* __restrict__ s, bool vec, bool vecc,
    bool vecq) {
  __shared__ unsigned red[4];
  const RowOf<X, NV> row(x + (int64_t)blockIdx.x * ldx, n, vec);
  signed char* out = q + (int64_t)blockIdx.x * ldq;
  auto values = [&](int64_t j, const Eight<X>& t, float* v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(t.v[e]);
    if (c) {
      float f[8];
      factors8(c, j, n, vecc, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= f[e];
    }
  };
  unsigned top = 0;
  row.each(n, [&](int64_t j, const Eight<X>& t) {
    float v[8];
    values(j, t, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // what lies past n was read as zero
      const unsigned a = __float_as_uint(v[e]) & 0x7fffffffu;
      top = a > top ? a : top;
    }
  });
  top = max_of_256(top, red);
  const float scale = top == 0 ? 1.0f : __uint_as_float(top) / 127.0f;
  if (threadIdx.x == 0) s[blockIdx.x] = scale;
  row.each(n, [&](int64_t j, const Eight<X>& t) {
    float v[8];
    values(j, t, v);
    signed char w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = __builtin_rintf(v[e] / scale);
      // a NaN compares false everywhere: code 0
      w[e] = (signed char)(u >= 127.0f ? 127 : u <= -127.0f ? -127 : u == u ? (int)u : 0);
    }
    if (vecq && j + 8 <= n) {
      *(uint2*)(out + j) = __builtin_bit_cast(uint2, w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < n) out[j + e] = w[e];
    }
  });
}

template <typename X>
hipError_t launch_quantize_tokens(int64_t T, int64_t n, const X* x, int64_t ldx, const float* c,
                                  int8_t* q, int64_t ldq, float* s, hipStream_t st) {
  if (T <= 0) return hipSuccess;
  const bool vec = load8_ok(x, ldx), vecc = load8_ok(c, 0), vecq = load8_ok(q, ldq);
#define BK_ROWS(NV)                                                                            \
  hipLaunchKernelGGL((quantize_tokens_kernel<X, NV>), dim3((unsigned)T), dim3(256), 0, st, n, x, \
                     ldx, c, (signed char*)q, ldq, s, vec, vecc, vecq)
  switch (row_groups(n)) {
    case 1: BK_ROWS(1); break;
    case 2: BK_ROWS(2); break;
    case 4: BK_ROWS(4); break;
    case 8: BK_ROWS(8); break;
    default: BK_ROWS(0);
  }
#undef BK_ROWS
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Y[t][i] = sx[t] * sv[i] * sum_j Xq[t][j] Vq[i][j]. The int32 sums are exact
// (n <= 131071); one float32 rounding each for the sum and the two scales, one
// to the output's type. The tile's rows are channels and its columns tokens,
// so a lane's four accumulators are four consecutive outputs of one token.
// 8192 x 14336 x 4096 to bfloat16, 256 x 256 tiles: 381 to 404 us from card to card,
// 2.4 to 2.5e15 op/s (a library's largest int8 product reaches 2.4e15 here).
// ---------------------------------------------------------------------------
template <typename O, int BR, int BC, int WR, int WC, bool ANY, int SLOTS = 5>
__global__ __launch_bounds__(64 * WR * WC) void matmul_int8_kernel(
    TileOperand V, TileOperand Xq, int64_t n, const float* __restrict__ sx,
    const float* __restrict__ sv, O* __restrict__ Y, int64_t ldy, bool vec, unsigned nr,
    unsigned nc, int splits, int* __restrict__ parts, int64_t ldp) {
  typedef TileProduct<MmaI8, BR, BC, WR, WC, false, false, SLOTS> TP;
  extern __shared__ char lds[];
  const unsigned tiles = nr * nc;
  const int range = blockIdx.x / tiles;
  int tr, tc;
  tile_of(blockIdx.x - range * tiles, nr, nc, tr, tc);
  const int64_t r0 = (int64_t)tr * BR, c0 = (int64_t)tc * BC;
  TP tp;
  tp.zero();
  if (ANY) {
    tp.run_any(V, Xq, n, r0, c0, lds);
  } else {
    const PlanePairs one = {1, 0, 0};
    const int64_t total = TP::steps(n, one);
    tp.run(V, Xq, n, one, r0, c0, (int)(total * range / splits),
           (int)(total * (range + 1) / splits), lds);
    if (splits > 1) {
      store_sums(tp, r0, c0, Xq.rows, parts + range * Xq.rows * ldp, ldp);
      return;
    }
  }
  const int lane = threadIdx.x & 63;
  float st[TP::FC], sr[TP::FR][4];
#pragma unroll
  for (int j = 0; j < TP::FC; ++j) {
    const int64_t t = c0 + tp.wave_c() + j * 16 + (lane & 15);
    st[j] = sx[t < Xq.rows ? t : Xq.rows - 1];
  }
#pragma unroll
  for (int i = 0; i < TP::FR; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sr[i][e] = 1.0f;
  if (sv) {
#pragma unroll
    for (int i = 0; i < TP::FR; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t r = r0 + tp.wave_r() + i * 16 + 4 * (lane >> 4) + e;
        sr[i][e] = sv[r < V.rows ? r : V.rows - 1];
      }
  }
  store_tile(tp, r0, c0, V.rows, Xq.rows, Y, ldy, vec,
             [&](int a, int i, int j, int e) { return (float)a * st[j] * sr[i][e]; });
}

// The ranges' sums and the scales; four channels of one token a thread (join_ranges).
template <typename O, int S>
__global__ __launch_bounds__(256) void join_int8_kernel(int64_t m, int64_t T, int splits,
                                                        const int* __restrict__ parts, int64_t ldp,
                                                        const float* __restrict__ sx,
                                                        const float* __restrict__ sv,
                                                        O* __restrict__ Y, int64_t ldy, bool vec) {
  __shared__ v4i red[S > 1 ? 256 : 1];
  const int64_t per = ldp / 4, at = JoinAt<S>::at();
  const int64_t t = at / per, r = (at - t * per) * 4;
  v4i a;
  if (!join_ranges<S>(parts + t * ldp + r, T * ldp, splits, at < T * per, a, red)) return;
  const float st = sx[t];
  O y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    y[e] = from_f32<O>((float)a[e] * st * (sv ? sv[r + e < m ? r + e : m - 1] : 1.0f));
  if (vec && r + 4 <= m) {
    *(typename Vec4<O>::type*)(Y + t * ldy + r) = __builtin_bit_cast(typename Vec4<O>::type, y);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r + e < m) Y[t * ldy + r + e] = y[e];
  }
}

// Rows whose length is no multiple of 16 are copied to zero-padded lines first
// (both operands, 16 bytes a thread): read as they are by the tiles they would
// come through registers, byte by byte at their ends, once per tile (777 x 1003
// x 1531: 33 us against 21).
__global__ __launch_bounds__(256) void pack_int8_kernel(TileOperand a, TileOperand b, int64_t n,
                                                        char* __restrict__ pa,
                                                        char* __restrict__ pb, int64_t ldp) {
  const int64_t per = ldp / 16;
  int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool second = at >= a.rows * per;
  if (second) at -= a.rows * per;
  if (second && at >= b.rows * per) return;
  const int64_t r = at / per, k = (at - r * per) * 16;
  *(v4i*)((second ? pb : pa) + r * ldp + k) =
      load_any<1>((second ? b.p + r * b.ld : a.p + r * a.ld), k, n);
}

template <typename O, int BR, int BC, int WR, int WC, bool ANY, int SLOTS = 5>
static hipError_t start_matmul_int8(const TileOperand& V, const TileOperand& X, int64_t n,
                                    const float* sx, const float* sv, O* Y, int64_t ldy,
                                    int splits, int* parts, hipStream_t s) {
  typedef TileProduct<MmaI8, BR, BC, WR, WC, false, false, SLOTS> TP;
  auto* k = matmul_int8_kernel<O, BR, BC, WR, WC, ANY, SLOTS>;
  constexpr int lds = TP::kLds;
  if (lds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t nr = (V.rows + BR - 1) / BR, nc = (X.rows + BC - 1) / BC;
  const int64_t ldp = (V.rows + 3) / 4 * 4;
  const bool vec = vec4_ok(Y, ldy);
  hipLaunchKernelGGL(k, dim3((unsigned)(nr * nc * splits)), dim3(TP::kThreads), lds, s, V, X, n, sx,
                     sv, Y, ldy, vec, (unsigned)nr, (unsigned)nc, splits, parts, ldp);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int64_t groups = X.rows * (ldp / 4);
#define BK_JOIN(S)                                                                               \
  hipLaunchKernelGGL((join_int8_kernel<O, S>),                                                   \
                     dim3((unsigned)((groups + 256 / S - 1) / (256 / S))), dim3(256), 0, s,      \
                     V.rows, X.rows, splits, parts, ldp, sx, sv, Y, ldy, vec)
  if (join_slices(splits) == 1) BK_JOIN(1);
  else BK_JOIN(8);
#undef BK_JOIN
  return hipGetLastError();
}

// Few tokens: the codes are read once, by workgroups of 16 RT channels. One token:
// 4096 x 4096 5.6 us, 14336 x 4096 13.5 us (4.3 TB/s).
template <typename O, int RT, int NT, bool ANY>
__global__ __launch_bounds__(512) void skinny_int8_kernel(TileOperand V, TileOperand Xq, int64_t n,
                                                          const float* __restrict__ sx,
                                                          const float* __restrict__ sv,
                                                          O* __restrict__ Y, int64_t ldy, bool vec) {
  typedef SkinnyProduct<MmaI8, RT, NT, RT == 1 ? 4 : 2, ANY> SP;
  __shared__ __attribute__((aligned(16))) char lds[SP::kLds];
  const int64_t c0 = (int64_t)blockIdx.y * SP::kCols;
  const TileOperand X = {Xq.p + c0 * Xq.ld, Xq.ld, 0, Xq.rows - c0, 0};
  const int64_t r0 = (int64_t)blockIdx.x * SP::kRows;
  // the scales are on their way while the product is formed
  const int64_t t = c0 + SP::tile_c(), r = r0 + SP::tile_r();
  const bool mine = SP::has_tile() && t < Xq.rows && r < V.rows;
  float st = 0.0f, sr[4] = {1.0f, 1.0f, 1.0f, 1.0f};
  if (mine) {
    st = sx[t];
    if (sv) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sr[e] = sv[r + e < V.rows ? r + e : r];
    }
  }
  SP::run(V, X, n, r0, lds, [&](v4i sum) {
    if (!mine) return;
    O y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = from_f32<O>((float)sum[e] * st * sr[e]);
    if (vec && r + 4 <= V.rows) {
      *(typename Vec4<O>::type*)(Y + t * ldy + r) =
          __builtin_bit_cast(typename Vec4<O>::type, y);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r + e < V.rows) Y[t * ldy + r + e] = y[e];
    }
  });
}

template <typename O, bool ANY>
static hipError_t start_skinny_int8(const TileOperand& V, const TileOperand& X, int64_t n,
                                    const float* sx, const float* sv, O* Y, int64_t ldy,
                                    hipStream_t s) {
  const bool vec = vec4_ok(Y, ldy);
  // several tiles of tokens: 32 channels a workgroup where that still gives every
  // CU one, since the tokens are then read half as often (14336 x 4096, 32 tokens:
  // 23 us against 28; 16 tokens: 18 against 19; one: 15 against 13.5)
  const int nt = X.rows > 48 ? 4 : (int)((X.rows + 15) / 16);
  const bool wide = V.rows >= 32 * 256 && X.rows > 8;
#define BK_SKINNY(RT, NT)                                                                     \
  hipLaunchKernelGGL((skinny_int8_kernel<O, RT, NT, ANY>),                                    \
                     dim3((unsigned)((V.rows + 16 * RT - 1) / (16 * RT)),                     \
                          (unsigned)((X.rows + 16 * NT - 1) / (16 * NT))),                    \
                     dim3(512), 0, s, V, X, n, sx, sv, Y, ldy, vec)
  if (wide) switch (nt) {
      case 1: BK_SKINNY(2, 1); break;
      case 2: BK_SKINNY(2, 2); break;
      case 3: BK_SKINNY(2, 3); break;
      default: BK_SKINNY(2, 4);
    }
  else switch (nt) {
      case 1: BK_SKINNY(1, 1); break;
      case 2: BK_SKINNY(1, 2); break;
      case 3: BK_SKINNY(1, 3); break;
      default: BK_SKINNY(1, 4);
    }
#undef BK_SKINNY
  return hipGetLastError();
}

// The most tokens the skinny kernel takes. It reads the tokens once for every 16
// or 32 channels, so the more codes there are the sooner tiles of 128 channels are
// faster (4096 x 4096, 64 tokens: 12.3 us against 12.6; 8192 x 8192, 48: 25 against
// 21, 16: 17 against 18; 28672 x 4096, 16: 34 against 28, 4: 25).
static int64_t skinny_tokens(int64_t m, int64_t n) {
  return m * n <= (1 << 24) ? 64 : m * n <= (1 << 26) ? 16 : 8;
}

static TilePlan int8_plan(int64_t T, int64_t m, int64_t n) {
  return plan_tiles(m, T, (n + kStepBytes - 1) / kStepBytes, 1, false, true);
}
static bool int8_packs(int64_t T, int64_t m, int64_t n) {
  return n % 16 != 0 && T > skinny_tokens(m, n);
}
static int64_t packed_ld(int64_t n) { return (n + kStepBytes - 1) / kStepBytes * kStepBytes; }
size_t matmul_int8_bytes(int64_t T, int64_t m, int64_t n) {
  if (T <= skinny_tokens(m, n)) return 0;
  return (size_t)split_words(m, T, int8_plan(T, m, n).splits) * 4 +
         (int8_packs(T, m, n) ? (size_t)((T + m) * packed_ld(n)) : 0);
}

template <typename O>
hipError_t launch_matmul_int8(int64_t T, int64_t m, int64_t n, const int8_t* Xq, int64_t ldx,
                              const float* sx, const int8_t* Vq, int64_t ldv, const float* sv, O* Y,
                              int64_t ldy, void* ws, hipStream_t s) {
  if (T <= 0 || m <= 0) return hipSuccess;
  TileOperand V = {(const char*)Vq, ldv, 0, m, 0}, X = {(const char*)Xq, ldx, 0, T, 0};
  if (int8_packs(T, m, n)) {
    const int64_t ld = packed_ld(n);
    char *pv = (char*)ws, *px = pv + m * ld;
    hipLaunchKernelGGL(pack_int8_kernel, dim3((unsigned)(((T + m) * (ld / 16) + 255) / 256)),
                       dim3(256), 0, s, V, X, n, pv, px, ld);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    V = {pv, ld, 0, m, 0};
    X = {px, ld, 0, T, 0};
    n = (n + 15) / 16 * 16;
    ws = px + T * ld;
  }
  const bool direct = tile_direct(V, n) && tile_direct(X, n);
  if (T <= skinny_tokens(m, n))
    return direct ? start_skinny_int8<O, false>(V, X, n, sx, sv, Y, ldy, s)
                  : start_skinny_int8<O, true>(V, X, n, sx, sv, Y, ldy, s);
  if (!direct)
    return start_matmul_int8<O, 128, 128, 2, 2, true>(V, X, n, sx, sv, Y, ldy, 1, nullptr, s);
  const TilePlan plan = int8_plan(T, m, n);
  if (plan.tile == 256)
    return start_matmul_int8<O, 256, 256, 2, 4, false>(V, X, n, sx, sv, Y, ldy, 1, nullptr, s);
  // One workgroup of 128 x 128 a CU, or two of 64 x 64, leave room for a ring of
  // nine slots, four steps ahead: 14336 x 4096 and 20 tokens 12.4 us against 16.6
  // (five slots), 100 tokens 18.8 against 21, 4096 x 14336 and 777 60 against 63.
  // 4096 x 4096 and 256 tokens 12.0 against 11.7; with 4 to 16 steps of n they
  // are within 4% of each other, as they are for the bfloat16 and float32 products.
  const bool deep = plan.splits * tiles_of(m, T, plan.tile) <= (plan.tile == 128 ? 256 : 512);
#define BK_TILE(B, SLOTS) \
  start_matmul_int8<O, B, B, 2, 2, false, SLOTS>(V, X, n, sx, sv, Y, ldy, plan.splits, (int*)ws, s)
  if (plan.tile == 128) return deep ? BK_TILE(128, 9) : BK_TILE(128, 5);
  return deep ? BK_TILE(64, 9) : BK_TILE(64, 5);
#undef BK_TILE
}

#define BK_INST_Q(X)                                                                        \
  template hipError_t launch_quantize_tokens<X>(int64_t, int64_t, const X*, int64_t,        \
                                                const float*, int8_t*, int64_t, float*, \
                                                hipStream_t);
BK_INST_Q(float)
BK_INST_Q(BF16)
BK_INST_Q(F16)
#undef BK_INST_Q
#define BK_INST_O(O)                                                                          \
  template hipError_t launch_matmul_int8<O>(int64_t, int64_t, int64_t, const int8_t*,         \
                                            int64_t, const float*, const int8_t*, int64_t,    \
                                            const float*, O*, int64_t, void*, hipStream_t);
BK_INST_O(float)
BK_INST_O(BF16)
BK_INST_O(F16)
#undef BK_INST_O

}  // namespace bk
