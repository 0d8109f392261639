// Tokens in the order of their experts, and back: the stable sort of the routes
// (token, choice) by expert, rows gathered in that order, the weighted sum of
// their results at each token, and its gradient. All bound by memory or, for
// few tokens, by latency.
#include "launch.hpp"
#include "tile_product.hpp"

namespace bk {

// ---------------------------------------------------------------------------
// Counting sort of N = T k routes p = t k + j by expert, stable: order[s] = p and
// slots[p] = s for s in p's expert's range [offsets[e], offsets[e + 1]). A route
// whose expert is outside [0, E) is dropped: the last range, marked -1.
//
// A workgroup takes a chunk of the routes, its 16 waves equal parts of it, and
// every (wave, expert) gets its first place: the expert's first, the routes of
// the chunks before (count_routes_kernel), those of the waves before. Then each
// wave goes through its part 64 routes at a time; a route's place among the 64
// comes from the mask of lanes with the same expert, a ballot for each bit of
// the expert's number. Counts are whole numbers, so the order in which LDS
// atomics add them does not matter. Up to 2048 routes are one launch, 4.7 us;
// 65536 to 128 experts two, 4.8 and 8.8 us.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int64_t kSortChunk = 2048;  // routes of a workgroup while there are at most kSortChunks
constexpr int64_t kSortChunks = 256;

struct Routes {
  const int64_t* ids;  // T rows of k, ld apart
  int64_t ld, k, N;
  int E;
  // p's expert, E where it is dropped
  __device__ inline int expert(int64_t p) const {
    const int64_t e = ld == k ? ids[p] : ids[p / k * ld + p % k];
    return e >= 0 && e < E ? (int)e : E;
  }
};

__global__ __launch_bounds__(kSortThreads) void count_routes_kernel(Routes r, int64_t chunk,
                                                                    int* __restrict__ counts) {
  extern __shared__ int hist[];
  for (int e = threadIdx.x; e <= r.E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * chunk, end = first + chunk < r.N ? first + chunk : r.N;
  for (int64_t p = first + threadIdx.x; p < end; p += kSortThreads) atomicAdd(&hist[r.expert(p)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= r.E; e += kSortThreads) counts[blockIdx.x * (int64_t)(r.E + 1) + e] = hist[e];
}

__global__ __launch_bounds__(kSortThreads) void place_routes_kernel(
    Routes r, int64_t chunk, const int* __restrict__ counts, int* __restrict__ order,
    int* __restrict__ slots, int* __restrict__ offsets) {
  extern __shared__ int lds[];
  const int B = r.E + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int *at = lds, *total = lds + kSortWaves * B, *scan = total + B;  // scan: 16 words
  for (int i = tid; i < kSortWaves * B; i += kSortThreads) at[i] = 0;
  __syncthreads();
  const int64_t part = chunk / kSortWaves;
  const int64_t first = blockIdx.x * chunk + wave * part;
  const int64_t end = first + part < r.N ? first + part : r.N;
  for (int64_t p = first + lane; p < end; p += 64) atomicAdd(&at[wave * B + r.expert(p)], 1);
  __syncthreads();
  // at: the routes of the chunks and waves before, by expert; total: all of them
  for (int e = tid; e < B; e += kSortThreads) {
    int before = 0, all = 0;
    if (gridDim.x > 1)
      for (unsigned c0 = 0; c0 < gridDim.x; c0 += 16) {  // 16 loads on their way at once
        int n[16];
#pragma unroll
        for (unsigned i = 0; i < 16; ++i)
          n[i] = c0 + i < gridDim.x ? counts[(c0 + i) * (int64_t)B + e] : 0;
#pragma unroll
        for (unsigned i = 0; i < 16; ++i) {
          all += n[i];
          before += c0 + i < blockIdx.x ? n[i] : 0;
        }
      }
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = at[w * B + e];
      at[w * B + e] = before;
      before += n;
    }
    total[e] = gridDim.x > 1 ? all : before;
  }
  __syncthreads();
  // exclusive prefix sums of the totals, 1024 at a time
  int base = 0;
  for (int e0 = 0; e0 < B; e0 += kSortThreads) {
    const int e = e0 + tid, n = e < B ? total[e] : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(sum, o, 64);
      sum += lane >= o ? u : 0;
    }
    if (lane == 63) scan[wave] = sum;
    __syncthreads();
    int before = base, all = base;
    for (int w = 0; w < kSortWaves; ++w) {
      before += w < wave ? scan[w] : 0;
      all += scan[w];
    }
    if (e < B) {
      total[e] = before + sum - n;
      if (blockIdx.x == 0) offsets[e] = total[e];
    }
    base = all;
    __syncthreads();
  }
  for (int i = tid; i < kSortWaves * B; i += kSortThreads) at[i] += total[i % B];
  __syncthreads();
  const int bits = 32 - __builtin_clz(r.E);  // of 0 .. E
  int* mine = at + wave * B;
  for (int64_t p0 = first; p0 < end; p0 += 64) {  // the wave's own places from here on
    const int64_t p = p0 + lane;
    const bool has = p < end;
    const int e = has ? r.expert(p) : 0;
    uint64_t same = __ballot(has);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(e >> b & 1);
      same &= (e >> b & 1) ? set : ~set;
    }
    const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
    int s = 0;
    if (has) s = mine[e] + rank;
    __builtin_amdgcn_wave_barrier();  // all lanes read before the last of each expert adds
    if (has && same >> lane == 1) mine[e] = s + 1;
    __builtin_amdgcn_wave_barrier();
    if (has) {
      order[s] = e < r.E ? (int)p : -1;
      slots[p] = e < r.E ? s : -1;
    }
  }
}

static int64_t sort_chunk(int64_t N) {
  const int64_t c = (N + kSortChunks - 1) / kSortChunks;
  return c <= kSortChunk ? kSortChunk : (c + kSortThreads - 1) / kSortThreads * kSortThreads;
}
size_t sort_tokens_bytes(int64_t N, int64_t E) {
  const int64_t chunks = (N + sort_chunk(N) - 1) / sort_chunk(N);
  return chunks > 1 ? (size_t)(chunks * (E + 1)) * 4 : 0;
}
hipError_t launch_sort_tokens(int64_t T, int64_t k, int64_t E, const int64_t* ids, int64_t ld,
                              int32_t* order, int32_t* slots, int32_t* offsets, void* ws,
                              hipStream_t s) {
  const Routes r = {ids, ld, k, T * k, (int)E};
  const int64_t chunk = sort_chunk(r.N);
  const unsigned chunks = r.N ? (unsigned)((r.N + chunk - 1) / chunk) : 1;
  const int lds = (int)((kSortWaves + 1) * (E + 1) + kSortWaves) * 4;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void*)place_routes_kernel,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  if (chunks > 1) {
    hipLaunchKernelGGL(count_routes_kernel, dim3(chunks), dim3(kSortThreads), (size_t)(E + 1) * 4,
                       s, r, chunk, (int*)ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(place_routes_kernel, dim3(chunks), dim3(kSortThreads), lds, s, r, chunk,
                     (const int*)ws, order, slots, offsets);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Xs[s] = X[order[s] / k], zeros where order[s] names no token. A wave to a row, 16
// bytes a lane where rows are aligned to them (`vec`), else element by element.
// Bound by writing: 65536 rows of 2048 bfloat16 72 us (3.7 TB/s written; four or eight loads
// at once and stores past the caches: the same).
// ---------------------------------------------------------------------------
template <typename X>
__global__ __launch_bounds__(256) void gather_kernel(int64_t T, int64_t n, const X* __restrict__ x,
                                                     int64_t ldx, int64_t k, int64_t R,
                                                     const int* __restrict__ order,
                                                     X* __restrict__ xs, int64_t lds, bool vec) {
  const int64_t r = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (r >= R) return;
  const int p = order[r];
  const int64_t t = p / k;
  const bool has = p >= 0 && t < T;
  const X* from = x + (has ? t : 0) * ldx;
  X* to = xs + r * lds;
  constexpr int E = 16 / sizeof(X);
  int64_t c = 0;  // what is left for the loops below begins here
  if (vec) {
    for (c = lane * E; c + E <= n; c += 64 * E)
      *(v4i*)(to + c) = has ? *(const v4i*)(from + c) : v4i{0, 0, 0, 0};
    c = n / E * E;
  }
  X zero;
  __builtin_memset(&zero, 0, sizeof zero);
  for (c += lane; c + 7 * 64 < n; c += 8 * 64) {  // eight on their way at once
    X v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = has ? from[c + 64 * i] : zero;
#pragma unroll
    for (int i = 0; i < 8; ++i) to[c + 64 * i] = v[i];
  }
  for (; c < n; c += 64) to[c] = has ? from[c] : zero;
}
template <typename X>
hipError_t launch_gather_tokens(int64_t T, int64_t n, const X* x, int64_t ldx, int64_t k, int64_t R,
                                const int32_t* order, X* xs, int64_t lds, hipStream_t s) {
  if (R <= 0 || n <= 0) return hipSuccess;
  const bool vec = ((uintptr_t)x | (uintptr_t)xs | (uintptr_t)(ldx * sizeof(X)) |
                    (uintptr_t)(lds * sizeof(X))) % 16 == 0;
  hipLaunchKernelGGL(gather_kernel<X>, dim3((unsigned)((R + 3) / 4)), dim3(256), 0, s, T, n, x, ldx,
                     k, R, order, xs, lds, vec);
  return hipGetLastError();
}

// Eight elements of a row for thread t of 256: from column 8 (256 k + t) on where every row is
// aligned to them (VEC), else 256 columns apart, so that a wave's load is one piece of
// the row all the same (combine_grad of 777 x 6 rows of 1531 float32: 43 us with eight
// loads side by side).
template <bool VEC> __device__ inline int64_t column(int64_t k, int e) {
  return VEC ? 8 * (256 * k + threadIdx.x) + e : 256 * (8 * k + e) + threadIdx.x;
}
template <typename X, bool VEC>
__device__ inline Eight<X> load_row(const X* row, int64_t k, int64_t n) {
  if (VEC) return load8(row, column<true>(k, 0), n, true);
  Eight<X> t;
  __builtin_memset(&t, 0, sizeof t);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (column<false>(k, e) < n) t.v[e] = row[column<false>(k, e)];
  return t;
}
template <typename X, bool VEC>
__device__ inline void store_row(X* row, int64_t k, int64_t n, const float* v) {
  X t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = from_f32<X>(v[e]);
  const int64_t c = column<VEC>(k, 0);
  if (VEC && c + 8 <= n) {
    constexpr int kPer = kLoadBytes<X> / sizeof(X);
#pragma unroll
    for (int i = 0; i < 8; i += kPer)
      __builtin_memcpy(__builtin_assume_aligned(row + c + i, kLoadBytes<X>), t + i, kLoadBytes<X>);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (column<VEC>(k, e) < n) row[column<VEC>(k, e)] = t[e];
  }
}

// ---------------------------------------------------------------------------
// Y[t] = sum_j w[t][j] Ys[slots[t][j]], j in order, in float32, rounded once; slots
// outside [0, R) take no part. A workgroup to 2048 columns of a token, the rows
// of four choices on their way at once (8192 tokens of 8 rows of 2048 bfloat16, a tenth
// dropped: 57 us, 4.8 TB/s).
// ---------------------------------------------------------------------------
template <typename X, bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(int64_t k, int64_t n, int64_t R,
                                                      const X* __restrict__ ys, int64_t ldys,
                                                      const int* __restrict__ slots,
                                                      const float* __restrict__ w,
                                                      X* __restrict__ y, int64_t ldy,
                                                      unsigned parts) {
  const int64_t t = blockIdx.x / parts, part = blockIdx.x - t * parts;
  if (column<VEC>(part, 0) >= n) return;
  float sum[8] = {};
  for (int64_t j0 = 0; j0 < k; j0 += 4) {
    Eight<X> v[4];
    float f[4];
    bool has[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t j = j0 + i;
      const int64_t s = j < k ? slots[t * k + j] : -1;
      has[i] = s >= 0 && s < R;
      f[i] = w && has[i] ? w[t * k + j] : 1.0f;
      if (has[i]) v[i] = load_row<X, VEC>(ys + s * ldys, part, n);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (has[i]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = __builtin_fmaf(f[i], to_f32(v[i].v[e]), sum[e]);
      }
  }
  store_row<X, VEC>(y + t * ldy, part, n, sum);
}
template <typename X>
hipError_t launch_combine_tokens(int64_t T, int64_t k, int64_t n, int64_t R, const X* ys,
                                 int64_t ldys, const int32_t* slots, const float* w, X* y,
                                 int64_t ldy, hipStream_t s) {
  if (T <= 0 || n <= 0) return hipSuccess;
  const unsigned parts = (unsigned)((n + 2047) / 2048);
  const bool vec = load8_ok(ys, ldys) && load8_ok(y, ldy);
  auto* kernel = vec ? combine_kernel<X, true> : combine_kernel<X, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(T * parts)), dim3(256), 0, s, k, n, R, ys, ldys, slots,
                     w, y, ldy, parts);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Its gradient: dYs[slots[t][j]] = w[t][j] G[t], dw[t][j] = G[t] . Ys[slots[t][j]]
// (0 where the slot is outside [0, R)). A workgroup to a token and kGradChoices of its
// choices, all of whose rows are on their way at once; the products' sums meet across the
// workgroup in a fixed order (8192 x 8 rows of 2048 bfloat16 136 us, 4.2 TB/s; 777 x 6 rows of 1531
// float32 12).
// ---------------------------------------------------------------------------
constexpr int kGradChoices = 4;
template <typename X, bool VEC>
__global__ __launch_bounds__(256) void combine_grad_kernel(
    int64_t k, int64_t n, int64_t R, const X* __restrict__ g, int64_t ldg,
    const X* __restrict__ ys, int64_t ldys, const int* __restrict__ slots,
    const float* __restrict__ w, X* __restrict__ dys, int64_t lddys, float* __restrict__ dw,
    unsigned parts) {
  __shared__ float red[4][kGradChoices];
  const int64_t t = blockIdx.x / parts;
  const int64_t j0 = (int64_t)(blockIdx.x - t * parts) * kGradChoices;
  g += t * ldg;
  int64_t slot[kGradChoices];
  bool has[kGradChoices];
  float f[kGradChoices], dot[kGradChoices] = {};
#pragma unroll
  for (int i = 0; i < kGradChoices; ++i) {
    const int64_t j = j0 + i;
    slot[i] = j < k ? slots[t * k + j] : -1;
    has[i] = slot[i] >= 0 && slot[i] < R;
    f[i] = w && has[i] ? w[t * k + j] : 1.0f;
  }
  for (int64_t c = 0; column<VEC>(c, 0) < n; ++c) {
    const Eight<X> g8 = load_row<X, VEC>(g, c, n);
    Eight<X> y8[kGradChoices];
    if (dw) {
#pragma unroll
      for (int i = 0; i < kGradChoices; ++i)
        if (has[i]) y8[i] = load_row<X, VEC>(ys + slot[i] * ldys, c, n);
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(g8.v[e]);
#pragma unroll
    for (int i = 0; i < kGradChoices; ++i) {
      if (!has[i]) continue;
      if (dw) {
#pragma unroll
        for (int e = 0; e < 8; ++e) dot[i] = __builtin_fmaf(v[e], to_f32(y8[i].v[e]), dot[i]);
      }
      if (dys) {
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = v[e] * f[i];
        store_row<X, VEC>(dys + slot[i] * lddys, c, n, d);
      }
    }
  }
  if (!dw) return;
#pragma unroll
  for (int i = 0; i < kGradChoices; ++i) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot[i] += __shfl_xor(dot[i], o, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][i] = dot[i];
  }
  __syncthreads();
  const int64_t j = j0 + threadIdx.x;
  if (threadIdx.x < kGradChoices && j < k)
    dw[t * k + j] = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
}
template <typename X>
hipError_t launch_combine_tokens_grad(int64_t T, int64_t k, int64_t n, int64_t R, const X* g,
                                      int64_t ldg, const X* ys, int64_t ldys, const int32_t* slots,
                                      const float* w, X* dys, int64_t lddys, float* dw,
                                      hipStream_t s) {
  if (T <= 0 || k <= 0) return hipSuccess;
  const unsigned parts = (unsigned)((k + kGradChoices - 1) / kGradChoices);
  const bool vec = load8_ok(g, ldg) && load8_ok(ys, ldys) && load8_ok(dys, lddys);
  auto* kernel = vec ? combine_grad_kernel<X, true> : combine_grad_kernel<X, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(T * parts)), dim3(256), 0, s, k, n, R, g, ldg, ys, ldys,
                     slots, w, dys, lddys, dw, parts);
  return hipGetLastError();
}

#define BK_INST(X)                                                                               \
  template hipError_t launch_gather_tokens<X>(int64_t, int64_t, const X*, int64_t, int64_t,      \
                                              int64_t, const int32_t*, X*, int64_t, hipStream_t); \
  template hipError_t launch_combine_tokens<X>(int64_t, int64_t, int64_t, int64_t, const X*,     \
                                               int64_t, const int32_t*, const float*, X*,        \
                                               int64_t, hipStream_t);                            \
  template hipError_t launch_combine_tokens_grad<X>(                                             \
      int64_t, int64_t, int64_t, int64_t, const X*, int64_t, const X*, int64_t, const int32_t*,  \
      const float*, X*, int64_t, float*, hipStream_t);
BK_INST(float)
BK_INST(BF16)
BK_INST(F16)
#undef BK_INST

}  // namespace bk
