// The 8-bit product on gfx950: tokens quantised to int8 with a scale each, the
// product of the int8 tokens with a layer's int8 codes (the solve's V), scaled
// per token and output channel, and its input gradient.
#include "launch.hpp"
#include "tile_product.hpp"

namespace bk {

// ---------------------------------------------------------------------------
// Tokens to int8: x = X[t][j] * c[j] in float32, s = max_j |x| / 127 (1 for an
// all-zero token), q = clamp(rint(x / s), -127, 127), the division correctly
// rounded as in the solve's quantizer. The maximum is taken over the bits of
// |x|, in which a NaN is larger than infinity: a token with an infinity or a
// NaN gets that as its scale, and codes whose products it makes NaN.
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
// ---------------------------------------------------------------------------
template <typename O, int BR, int BC, int WR, int WC, bool ANY>
__global__ __launch_bounds__(64 * WR * WC) void matmul_int8_kernel(
    TileOperand V, TileOperand Xq, int64_t n, const float* __restrict__ sx,
    const float* __restrict__ sv, O* __restrict__ Y, int64_t ldy, bool vec, unsigned nr,
    unsigned nc) {
  typedef TileProduct<MmaI8, BR, BC, WR, WC> TP;
  extern __shared__ char lds[];
  int tr, tc;
  tile_of(blockIdx.x, nr, nc, tr, tc);
  const int64_t r0 = (int64_t)tr * BR, c0 = (int64_t)tc * BC;
  TP tp;
  tp.zero();
  if (ANY) {
    tp.run_any(V, Xq, n, r0, c0, lds);
  } else {
    const PlanePairs one = {1, 0, 0};
    tp.run(V, Xq, n, one, r0, c0, 0, TP::steps(n, one), lds);
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

template <typename O, int BR, int BC, int WR, int WC, bool ANY>
static hipError_t start_matmul_int8(const TileOperand& V, const TileOperand& X, int64_t n,
                                    const float* sx, const float* sv, O* Y, int64_t ldy,
                                    hipStream_t s) {
  typedef TileProduct<MmaI8, BR, BC, WR, WC> TP;
  auto* k = matmul_int8_kernel<O, BR, BC, WR, WC, ANY>;
  constexpr int lds = TP::kLds;
  if (lds > 65536) {
    const hipError_t e =
        hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const int64_t nr = (V.rows + BR - 1) / BR, nc = (X.rows + BC - 1) / BC;
  hipLaunchKernelGGL(k, dim3((unsigned)(nr * nc)), dim3(TP::kThreads), lds, s, V, X, n, sx, sv, Y,
                     ldy, vec4_ok(Y, ldy), (unsigned)nr, (unsigned)nc);
  return hipGetLastError();
}

template <typename O>
hipError_t launch_matmul_int8(int64_t T, int64_t m, int64_t n, const int8_t* Xq, int64_t ldx,
                              const float* sx, const int8_t* Vq, int64_t ldv, const float* sv, O* Y,
                              int64_t ldy, hipStream_t s) {
  if (T <= 0 || m <= 0) return hipSuccess;
  const TileOperand V = {(const char*)Vq, ldv, 0, m, 0}, X = {(const char*)Xq, ldx, 0, T, 0};
  const bool direct = tile_direct(V, n) && tile_direct(X, n);
  if (!direct) return start_matmul_int8<O, 128, 128, 2, 2, true>(V, X, n, sx, sv, Y, ldy, s);
  const int64_t big = ((m + 255) / 256) * ((T + 255) / 256);
  if (big >= 192)
    return start_matmul_int8<O, 256, 256, 2, 4, false>(V, X, n, sx, sv, Y, ldy, s);
  return start_matmul_int8<O, 128, 128, 2, 2, false>(V, X, n, sx, sv, Y, ldy, s);
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
                                            const float*, O*, int64_t, hipStream_t);
BK_INST_O(float)
BK_INST_O(BF16)
BK_INST_O(F16)
#undef BK_INST_O

}  // namespace bk
