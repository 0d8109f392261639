// The tiled product with a scale for each block of k:
//   D[r][c] = sum over steps s of f_s(r, c) sum_{k in step s} R[r][k] C[c][k],
// a step being 128 bytes of k, f_s = sw[r / 128][b] sx[c][b] for the step's block b. The
// blocks' sums leave the matrix instructions after every step and are added to the
// accumulators times their scale, four multiply-adds a lane to each instruction or
// pair of instructions of 32 cycles.
//
// Layout of the operands in LDS, their loads and the order of steps are those of
// tile_product.hpp, with three differences. A step is not read in halves: a wave holds its
// columns' fragments and up to four rows' at a time, rows coming in while the rows before
// are multiplied, and the next step's columns while the last rows are (column by column,
// as each is used for the last time). The ring's unit is half of one operand's step: nine
// of them (of 256 x 128 bytes: 144 KB; two whole steps and half an operand more), which leaves
// room for the steps' scales. And those come the same way, 4 bytes a lane: the first waves
// load the columns' scales, the others the rows'.
#pragma once

#include "fp8_product.hpp"

namespace bk {

template <class Mul, int B, int WR, int WC>
struct BlockTile {
  typedef f32x4 acc_t;
  static constexpr int kWaves = WR * WC, kThreads = 64 * kWaves;
  static constexpr int FR = B / WR / 16, FC = B / WC / 16;
  static constexpr int kUnit = B * kStepBytes / 2, kUnits = 9;
  static constexpr int LU = kUnit / 1024 / kWaves;  // a wave's loads to a unit
  static constexpr int kScaleSlot = kWaves * 256, kScaleSlots = 3;
  static constexpr int kLds = kUnits * kUnit + kScaleSlots * kScaleSlot;
  static constexpr int NB = FR < 4 ? FR : 4;                  // rows' fragments held
  static constexpr int P = FR == 8 ? 3 : FR == 4 ? 2 : 1;     // rows multiplied after the barrier
  static constexpr int kLoads = 4 * LU + 1;                   // a wave's loads to a step
  static constexpr int kEarly = kLoads / 3;                   // of them, those that go out first
  static_assert(LU * 1024 * kWaves == kUnit && kWaves % 2 == 0, "a unit's bytes divide over the waves");
  static_assert(FR % NB == 0 && P < FR && P <= NB, "rows' fragments go round");
  static_assert(B / WR >= 32 && B / WR <= 128 && B / WC <= B / 2, "a wave's rows and columns lie in one unit");
  static_assert(B / 64 < kWaves, "a wave for the rows' scales");

  f32x4 acc[FR][FC];

  __device__ static inline int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
  __device__ inline int wave_r() const { return (threadIdx.x >> 6) / WC * (FR * 16); }
  __device__ inline int wave_c() const { return (threadIdx.x >> 6) % WC * (FC * 16); }
  __device__ inline void zero() {
#pragma unroll
    for (int i = 0; i < FR; ++i)
#pragma unroll
      for (int j = 0; j < FC; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  }
  __device__ static inline int chunk_at(int row, int pos) { return pos ^ ((row >> 1) & 7); }

  // as TileProduct::load_lds; BYTES a lane
  template <int BYTES>
  __device__ static inline void load_lds(v4i rsrc, int voff, int soff, unsigned lds) {
    if (BYTES == 16)
      asm volatile(
          "s_nop 4\n\t"
          "buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff),
          "s"(rsrc), "s"(soff), "{m0}"(lds)
          : "memory");
    else
      asm volatile(
          "s_nop 4\n\t"
          "buffer_load_dword %0, %1, %2 offen lds" ::"v"(voff),
          "s"(rsrc), "s"(soff), "{m0}"(lds)
          : "memory");
  }
  __device__ static inline v4i buffer(const void* p, int bytes) {
    const uint64_t a = (uint64_t)p;
    return v4i{__builtin_amdgcn_readfirstlane((int)(unsigned)a),
               __builtin_amdgcn_readfirstlane((int)(unsigned)(a >> 32) & 0xffff),
               __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
  }
  static constexpr int kNone = (int)0x80000000;  // an offset past every buffer: reads zero

  // An operand's loads: a lane's byte offset from `p` for each of a step's wave loads, row
  // `row` of the tile at at(row) (kNone: zeros). Chunks past the end of k read as zero.
  struct Side {
    v4i rsrc;
    int off[2 * LU];
    bool past;
    int k, last;

    template <typename F>
    __device__ inline void init(const void* p, int bytes, int64_t kbytes, int s0, F at) {
      const int lane = threadIdx.x & 63, w = wave(), row8 = lane >> 3;
      const int chunk = chunk_at((w & 1) * 8 + row8, lane & 7);
      rsrc = buffer(p, bytes);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < LU; ++j) {
          const int o = at(h * (B / 2) + (j * kWaves + w) * 8 + row8);
          off[h * LU + j] = o == kNone ? kNone : o + chunk * 16;
        }
      last = (int)((kbytes + kStepBytes - 1) / kStepBytes) - 1;
      past = chunk * 16 + last * kStepBytes >= (int)kbytes;
      k = __builtin_amdgcn_readfirstlane(s0);
    }
    __device__ inline void load(int h, int j, unsigned lds) const {
      load_lds<16>(rsrc, k == last && past ? kNone : off[h * LU + j], k * kStepBytes,
                   lds + j * kWaves * 1024);
    }
  };

  template <int N> __device__ static inline void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
  }

  // D's tile, its steps [s0, s1). `scale`: this wave's scales, per[lane] bytes from the step's
  // pointer, which moves `stride` bytes a block, `each` steps to a block.
  __device__ inline void run(Side& R, Side& C, const char* scale, int per, int64_t stride, int each,
                             int s0, int s1, char* lds) {
    s0 = __builtin_amdgcn_readfirstlane(s0);
    const int total = __builtin_amdgcn_readfirstlane(s1) - s0;
    if (total <= 0) return;
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4, w = wave();
    const unsigned base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    const unsigned mine = base + w * 1024, smine = base + kUnits * kUnit + w * 256;
    unsigned u = 0, us = 0;  // the next unit and scale slot to load
    int block = s0 / each, in = s0 - block * each;
    scale += block * stride;

    auto next_unit = [&]() { u = u == kUnits - 1 ? 0 : u + 1; };
    auto load_unit = [&](const Side& side, int h) {
#pragma unroll
      for (int j = 0; j < LU; ++j) side.load(h, j, mine + u * kUnit);
      next_unit();
    };
    auto load_scale = [&]() {
      load_lds<4>(buffer(scale, 0x7fffffff), per, 0, smine + us * kScaleSlot);
      us = us == kScaleSlots - 1 ? 0 : us + 1;
      if (++in == each) {
        in = 0;
        scale += stride;
      }
    };
    // the n-th load after a step's barrier: R's second half, C and the scales of the step
    // after the next, and R's first half of the one behind it
    auto load_n = [&](int n) {
      if (n < LU) {
        R.load(1, n, mine + u * kUnit);
        if (n == LU - 1) {
          ++R.k;
          next_unit();
        }
      } else if (n < 3 * LU) {
        const int h = n < 2 * LU ? 0 : 1, j = n - (h + 1) * LU;
        C.load(h, j, mine + u * kUnit);
        if (j == LU - 1) {
          C.k += h;
          next_unit();
        }
      } else if (n == 3 * LU) {
        load_scale();
      } else {
        R.load(0, n - 3 * LU - 1, mine + u * kUnit);
        if (n == 4 * LU) next_unit();
      }
    };
    auto load_step = [&](bool first) {
      if (first) load_unit(R, 0);
      load_unit(R, 1);
      ++R.k;
      load_unit(C, 0);
      load_unit(C, 1);
      ++C.k;
      load_scale();
    };
    load_step(true);
    if (total > 1) load_step(true);
    if (total > 2) {
      load_unit(R, 0);
      wait_barrier<kLoads + LU>();
    } else {
      wait_barrier<0>();
    }

    const int hr = w / WC * FR * 16 >= B / 2, hc = w % WC * FC * 16 >= B / 2;
    const int lr = (w / WC * FR * 16 - hr * (B / 2)) * kStepBytes;
    const int lc = (w % WC * FC * 16 - hc * (B / 2)) * kStepBytes;
    int at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) at[h] = r16 * kStepBytes + chunk_at(r16, h * 4 + q) * 16;
    unsigned step = 0, sslot = 0;  // unit and scale slot of the step that is read
    const char *pr, *pc, *ps;
    auto point = [&]() {
      const unsigned a = step + hr >= kUnits ? step + hr - kUnits : step + hr;
      const unsigned b = step + 2 + hc >= kUnits ? step + 2 + hc - kUnits : step + 2 + hc;
      pr = lds + a * kUnit + lr;
      pc = lds + b * kUnit + lc;
      ps = lds + kUnits * kUnit + sslot * kScaleSlot;
    };
    v4i r[NB][2], c[FC][2];
    float sx[FC], sw, f[FC];
    auto read_r = [&](int i, int h) { r[i % NB][h] = *(const v4i*)(pr + i * 16 * kStepBytes + at[h]); };
    auto read_c = [&](int j, int h) { c[j][h] = *(const v4i*)(pc + j * 16 * kStepBytes + at[h]); };
    auto read_s = [&](int j) {
      if (j < FC)
        sx[j] = *(const float*)(ps + (w % WC * FC * 16 + j * 16 + r16) * 4);
      else
        sw = *(const float*)(ps + B * 4 + (w / WC * FR * 16 >> 7) * 4);
    };
    // Instruction n of a step is of row_of(n) and column_of(n): the first rows row by row, the
    // others column by column. Its sums are added when two more have been started.
    constexpr int kFirst = (FR - P) * FC, kAll = FR * FC;
    auto row_of = [](int n) { return n < kFirst ? n / FC : FR - P + (n - kFirst) % P; };
    auto column_of = [](int n) { return n < kFirst ? n % FC : (n - kFirst) / P; };
    f32x4 part[3];
    auto add = [&](int n) {
      const int i = row_of(n), j = column_of(n);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[n % 3][e], f[j], acc[i][j][e]);
    };
    auto multiply = [&](int n) {
      const int i = row_of(n), j = column_of(n);
      part[n % 3] = Mul::block(r[i % NB][0], r[i % NB][1], c[j][0], c[j][1]);
      if (n >= 2) add(n - 2);
      __builtin_amdgcn_sched_barrier(0);
    };
    // the rows before the barrier; rows up to i + NB - 1 are read by the end of row i
    auto first_rows = [&](auto loads) {
      constexpr bool LOADS = decltype(loads)::value;
      constexpr int kRest = kLoads - kEarly, kEvery = kFirst / kRest > 0 ? kFirst / kRest : 1;
#pragma unroll
      for (int j = 0; j < FC; ++j) f[j] = sx[j] * sw;
#pragma unroll
      for (int n = 0; n < kFirst; ++n) {
        const int i = n / FC, j = n % FC;
        const int have = i == 0 ? 1 : i + NB - 1, want = i + NB < FR ? i + NB : FR;
#pragma unroll
        for (int x = j; x < 2 * (want - have); x += FC) read_r(have + x / 2, x & 1);
        if (LOADS && n % kEvery == 0 && n / kEvery < kRest) load_n(kEarly + n / kEvery);
        multiply(n);
      }
      if (LOADS) {
#pragma unroll
        for (int x = (kFirst + kEvery - 1) / kEvery; x < kRest; ++x) load_n(kEarly + x);
      }
    };
    // the rest, and the next step's first row, scales and columns, each column once it was used
    // for the last time
    auto last_rows = [&](auto loads, auto next) {
      constexpr bool LOADS = decltype(loads)::value, NEXT = decltype(next)::value;
      if (NEXT) {
        read_r(0, 0);
        read_r(0, 1);
#pragma unroll
        for (int j = 0; j <= FC; ++j) read_s(j);
      }
#pragma unroll
      for (int n = kFirst; n < kAll; ++n) {
        if (LOADS && n - kFirst < kEarly) load_n(n - kFirst);
        multiply(n);
        if (NEXT && (n - kFirst) % P == P - 1) {
          read_c(column_of(n), 0);
          read_c(column_of(n), 1);
        }
      }
      if (LOADS) {
#pragma unroll
        for (int x = kAll - kFirst; x < kEarly; ++x) load_n(x);
      }
      add(kAll - 2);
      add(kAll - 1);
      __builtin_amdgcn_sched_barrier(0);
    };
    const std::true_type yes;
    const std::false_type no;
    point();
    read_r(0, 0);
    read_r(0, 1);
#pragma unroll
    for (int j = 0; j < FC; ++j) {
      read_c(j, 0);
      read_c(j, 1);
    }
#pragma unroll
    for (int j = 0; j <= FC; ++j) read_s(j);
    auto advance = [&]() {
      step = step + 4 >= kUnits ? step + 4 - kUnits : step + 4;
      sslot = sslot == kScaleSlots - 1 ? 0 : sslot + 1;
      point();
    };
    first_rows(no);
    int s = 0;
    for (; s + 3 < total; ++s) {
      wait_barrier<LU>();
      advance();
      last_rows(yes, yes);
      first_rows(yes);
    }
    for (; s + 1 < total; ++s) {
      if (s + 2 < total)
        wait_barrier<LU>();
      else
        wait_barrier<0>();
      advance();
      if (s + 2 < total) load_step(false);
      last_rows(no, yes);
      first_rows(no);
    }
    last_rows(no, no);
  }
};

}  // namespace bk
