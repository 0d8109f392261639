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
//
// With Mul::kTransposed R is e4m3 codes k-major (k its rows, D's rows side by side, as a
// layer's weights are for its input gradient) and C 16-bit along k: a step is 64 k, one unit of R and
// two of C, so the ring holds three whole steps (or two, DEEP, which lets three workgroups of 128 x
// 128 share a CU: a wave's additions do not run beside its own matrix instructions). R is read
// from LDS by the transposing 8-byte reads, 8 k of a column to a lane, and made 16-bit in
// registers, once for each row of instructions: no 16-bit copy of the weights is written or
// read. Only R has scales.
//
// What bounds a large product (8192 x 14336 x 4096 e4m3, 256 x 256, 470 us): the matrix instructions
// alone would keep their units busy for 0.48 of its cycles. Without the multiply-adds it took 420
// us, without loads as well 352, without barriers as well 336: a wave's additions do not
// run beside its own matrix instructions, the chip slows its clock down under them (1.7 GHz of
// 2.4 on average), and no single wait is what is missing. Tried: the two waves of a SIMD
// taking turns, one multiplying while the other reads (508 us: its additions then run beside
// nothing); sums added two or three products later: the same.
#pragma once

#include "fp8_product.hpp"

namespace bk {

template <class Mul, int B, int WR, int WC, int DEEP = Mul::kTransposed ? 3 : 2>
struct BlockTile {
  typedef f32x4 acc_t;
  static constexpr int kWaves = WR * WC, kThreads = 64 * kWaves;
  static constexpr int FR = B / WR / 16, FC = B / WC / 16;
  static constexpr bool T = Mul::kTransposed;
  static constexpr int kUnit = B * kStepBytes / 2;
  static constexpr int kStepUnits = T ? 3 : 4;
  static constexpr int kDeep = DEEP;  // whole steps in the ring
  static constexpr int kUnits = T ? 3 * kDeep : 9;
  static constexpr int LU = kUnit / 1024 / kWaves;  // a wave's loads to a unit
  static constexpr int kScaleSlot = kWaves * 256, kScaleSlots = 3;
  static constexpr int kLds = kUnits * kUnit + kScaleSlots * kScaleSlot;
  static constexpr int NB = FR < 4 ? FR : 4;                  // rows' fragments held
  static constexpr int P = FR == 8 ? (T ? 2 : 3) : FR == 4 ? 2 : 1;  // rows multiplied after the barrier
  static constexpr int kLoads = kStepUnits * LU + 1;          // a wave's loads to a step
  static constexpr int kAhead = T ? (kDeep - 2) * kLoads : LU;  // in flight at a step's barrier
  static constexpr int kEarly = kLoads / 3;                   // of them, those that go out first
  static constexpr int kLate = T ? 3 : 2;                     // products between a product and its sums' addition
  static_assert(T ? kDeep == 2 || kDeep == 3 : kDeep == 2, "as the waits count");
  static_assert(LU * 1024 * kWaves == kUnit && kWaves % 2 == 0, "a unit's bytes divide over the waves");
  static_assert(FR % NB == 0 && P < FR && P <= NB, "rows' fragments go round");
  static_assert(B / WR >= 32 && B / WR <= 128 && B / WC <= B / 2, "a wave's rows and columns lie in one unit");
  static_assert(T || B / 64 < kWaves, "a wave for the rows' scales");

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
  // `row` of the tile at at(row) (kNone: zeros). Chunks past the end of k read as zero. With
  // several planes, `plane` bytes apart, the steps of one follow those of the one before.
  struct Side {
    const char* p;
    int64_t plane;
    v4i rsrc;
    int off[2 * LU];
    bool past;
    int k, last, bytes;

    template <typename F>
    __device__ inline void init(const void* p_, int bytes_, int64_t kbytes, int64_t plane_, int s0, F at) {
      const int lane = threadIdx.x & 63, w = wave(), row8 = lane >> 3;
      const int chunk = chunk_at((w & 1) * 8 + row8, lane & 7);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < LU; ++j) {
          const int o = at(h * (B / 2) + (j * kWaves + w) * 8 + row8);
          off[h * LU + j] = o == kNone ? kNone : o + chunk * 16;
        }
      last = (int)((kbytes + kStepBytes - 1) / kStepBytes) - 1;
      past = chunk * 16 + last * kStepBytes >= (int)kbytes;
      const int pl = last < 0 ? 0 : __builtin_amdgcn_readfirstlane(s0) / (last + 1);
      k = __builtin_amdgcn_readfirstlane(s0) - pl * (last + 1);
      plane = plane_;
      bytes = bytes_;
      p = (const char*)p_ + pl * plane;
      rsrc = buffer(p, bytes);
    }
    __device__ inline void load(int h, int j, unsigned lds) const {
      load_lds<16>(rsrc, k == last && past ? kNone : off[h * LU + j], k * kStepBytes,
                   lds + j * kWaves * 1024);
    }
    __device__ inline void next() {
      if (Mul::kPlanes > 1) {  // without a branch, which would split the order of instructions
        const bool wrap = k == last;
        k = wrap ? 0 : k + 1;
        p += wrap ? plane : 0;
        rsrc = buffer(p, bytes);
      } else {
        ++k;
      }
    }
  };
  // R of kTransposed: `krows` rows of k, `ld` bytes apart, each holding that k of the tile's
  // `cols` columns from `p` on; what follows them in their last chunk makes columns that are not
  // for storing, and of the last row no word is read that holds none of them. A step's 64 k lie
  // in LDS one after the other, the 16 bytes b of k at b ^ swap_at(k): the 16 k that two groups
  // of 16 lanes read at one b then fall on different banks.
  __device__ static inline int swap_at(int k) { return B == 256 ? k & 15 : B == 128 ? (k >> 1) & 7 : (k >> 2) & 3; }
  struct SideT {
    const char *p, *first;
    int64_t stride;
    v4i rsrc;
    int off[LU];
    int krow, k, last, bytes, bytes_last;
    __device__ inline void init(const char* p_, int64_t ld, int64_t krows, int cols, int s0) {
      const int lane = threadIdx.x & 63;
      constexpr int per = B / 16, lanes_k = 64 / per;  // chunks of a k; k of a wave load
#pragma unroll
      for (int j = 0; j < LU; ++j) {
        const int kr = (j * kWaves + wave()) * lanes_k + lane / per, chunk = lane % per ^ swap_at(kr);
        off[j] = chunk * 16 < cols ? kr * (int)ld + chunk * 16 : kNone;
      }
      last = (int)((krows + 63) / 64) - 1;
      krow = wave() * lanes_k + lane / per + last * 64 - (int)krows;  // >= 0 in the last step: past the last k
      stride = 64 * ld;
      bytes = 63 * (int)ld + (cols + 15) / 16 * 16;
      bytes_last = ((int)(krows - 1) - last * 64) * (int)ld + (cols + 3) / 4 * 4;
      first = p_;
      k = last < 0 ? 0 : __builtin_amdgcn_readfirstlane(s0) % (last + 1);
      p = p_ + k * stride;
      bytes = __builtin_amdgcn_readfirstlane(bytes);  // in next(): 8192 x 4096 x 14336 857 us, not 850
      bytes_last = __builtin_amdgcn_readfirstlane(bytes_last);
      last = __builtin_amdgcn_readfirstlane(last);
      rsrc = buffer(p, k == last ? bytes_last : bytes);
    }
    __device__ inline void load(int, int j, unsigned lds) const {
      constexpr int lanes_k = 64 / (B / 16);
      load_lds<16>(rsrc, k == last && krow + j * kWaves * lanes_k >= 0 ? kNone : off[j], 0,
                   lds + j * kWaves * 1024);
    }
    __device__ inline void next() {
      const bool wrap = Mul::kPlanes > 1 && k == last;
      k = wrap ? 0 : k + 1;
      p = wrap ? first : p + stride;
      rsrc = buffer(p, k == last ? bytes_last : bytes);
    }
  };
  typedef typename std::conditional<T, SideT, Side>::type SideR;

  template <int N> __device__ static inline void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
  }

  // Rows of a length that is no multiple of 16: what follows them in their last chunk came along and
  // may be anything, a NaN for instance. It is made zero in LDS, in the units of one step from
  // `first` on, byte `tail` of a row on. (Copied to zero-padded lines first, 1000 x 2000 x 4095
  // bfloat16 takes 32 us in place of 21.)
  __device__ static inline void zero_tail(char* lds, unsigned first, int tail) {
    for (int row = threadIdx.x; row < 2 * B; row += kThreads) {
      unsigned u = first + row / (B / 2);
      u = u >= kUnits ? u - kUnits : u;
      const int r = row % (B / 2);
      v4i* at = (v4i*)(lds + u * kUnit + r * kStepBytes + chunk_at(r, tail / 16) * 16);
      v4i x = *at;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int keep = tail % 16 - 4 * d;  // bytes of this word
        x[d] &= keep >= 4 ? -1 : keep <= 0 ? 0 : (1 << 8 * keep) - 1;
      }
      *at = x;
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  }

  // D's tile, its steps [s0, s1). `scale`: this wave's scales, `per` bytes from the block's
  // pointer, which moves `stride` bytes a block of k. `tail`: where rows end in the last of these
  // steps, 0 at a multiple of 16 (zero_tail).
  __device__ inline void run(SideR& R, Side& C, const char* scale, int per, int64_t stride, int s0,
                             int s1, char* lds, int tail = 0) {
    s0 = __builtin_amdgcn_readfirstlane(s0);
    const int total = __builtin_amdgcn_readfirstlane(s1) - s0;
    if (total <= 0) return;
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4, w = wave();
    const unsigned base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    const unsigned mine = base + w * 1024, smine = base + kUnits * kUnit + w * 256;
    unsigned u = 0, us = 0;  // the next unit and scale slot to load
    constexpr int kEach = T ? 2 : 1;  // steps to a block
    const char* const scale0 = scale;
    int ks = C.k;  // the step of k whose scales are loaded next
    scale += ks / kEach * stride;

    auto next_unit = [&]() { u = u == kUnits - 1 ? 0 : u + 1; };
    auto load_unit = [&](const auto& side, int h) {
#pragma unroll
      for (int j = 0; j < LU; ++j) side.load(h, j, mine + u * kUnit);
      next_unit();
    };
    auto load_scale = [&]() {
      load_lds<4>(buffer(scale, 0x7fffffff), per, 0, smine + us * kScaleSlot);
      us = us == kScaleSlots - 1 ? 0 : us + 1;
      const bool wrap = Mul::kPlanes > 1 && ks == C.last;
      ks = wrap ? 0 : ks + 1;
      scale = wrap ? scale0 : scale + (ks % kEach == 0 ? stride : 0);
    };
    // The n-th load after a step's barrier. R's second half, C and the scales of the step
    // after the next, and R's first half of the one behind it; kTransposed: all of the third
    // step from there.
    auto load_n = [&](int n) {
      constexpr int kR = LU;
      if (n < kR) {
        R.load(1, n, mine + u * kUnit);
        if (n == kR - 1) {
          R.next();
          next_unit();
        }
      } else if (n < kR + 2 * LU) {
        const int h = n < kR + LU ? 0 : 1, j = n - kR - h * LU;
        C.load(h, j, mine + u * kUnit);
        if (j == LU - 1) {
          if (h) C.next();
          next_unit();
        }
      } else if (n == kR + 2 * LU) {
        load_scale();
      } else {
        R.load(0, n - kR - 2 * LU - 1, mine + u * kUnit);
        if (n == 4 * LU) next_unit();
      }
    };
    auto load_step = [&](bool first) {
      if (!T && first) load_unit(R, 0);
      load_unit(R, 1);
      R.next();
      load_unit(C, 0);
      load_unit(C, 1);
      C.next();
      load_scale();
    };
    load_step(true);
    if (total > 1) load_step(true);
    if (total > 2) {
      if (T && kDeep > 2) load_step(true);
      if (!T) load_unit(R, 0);
      wait_barrier<kLoads + kAhead>();
    } else {
      wait_barrier<0>();
      if (!T && tail && total == 1) zero_tail(lds, 0, tail);
    }

    const int hr = w / WC * FR * 16 >= B / 2, hc = w % WC * FC * 16 >= B / 2;
    const int lr = T ? 0 : (w / WC * FR * 16 - hr * (B / 2)) * kStepBytes;
    const int lc = (w % WC * FC * 16 - hc * (B / 2)) * kStepBytes;
    int at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) at[h] = r16 * kStepBytes + chunk_at(r16, h * 4 + q) * 16;
    // kTransposed: two lanes give the 16 bytes of one k, 16 lanes those of eight
    const int kt = 8 * q + r16 / 2;
    const int atT = kt * B + (w / WC * FR ^ swap_at(kt)) * 16 + r16 % 2 * 8;
    unsigned step = 0, sslot = 0;  // unit and scale slot of the step that is read
    const char *pr, *pc, *ps;
    auto point = [&]() {
      const unsigned ur = T ? step : step + hr, uc = step + kStepUnits - 2 + hc;
      const unsigned a = ur >= kUnits ? ur - kUnits : ur, b = uc >= kUnits ? uc - kUnits : uc;
      pr = lds + a * kUnit + lr;
      pc = lds + b * kUnit + lc;
      ps = lds + kUnits * kUnit + sslot * kScaleSlot;
    };
    v4i r[NB][T ? 1 : 2], c[FC][2], wide[4][2];
    float sx[FC], sw, f[FC], old[kLate];
    auto read_r = [&](int i, int h) {
      if constexpr (T) {
        // 32 k further on swap_at is the same, and so it is in the rows of one wave, whose first
        // block is a multiple of their number
        typedef int v2i __attribute__((ext_vector_type(2)));
        typedef __attribute__((address_space(3))) v2i lds_v2i;
        const v2i x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(pr + (atT ^ i * 16) + h * 32 * B));
        r[i % NB][0][2 * h] = x[0];
        r[i % NB][0][2 * h + 1] = x[1];
      } else {
        r[i % NB][h] = *(const v4i*)(pr + i * 16 * kStepBytes + at[h]);
      }
    };
    // Row i made 16-bit: rows before the barrier in two places in turn, those after it in two others.
    auto place = [](int i) { return i < FR - P ? i % 2 : 2 + i - (FR - P); };
    auto widen = [&](int i) {
      if constexpr (T) Mul::widen(r[i % NB][0], wide[place(i)][0], wide[place(i)][1]);
    };
    auto read_c = [&](int j, int h) { c[j][h] = *(const v4i*)(pc + j * 16 * kStepBytes + at[h]); };
    auto read_s = [&](int j) {
      if (j == FC)
        sw = *(const float*)(ps + (T ? w * 256 : B * 4) + (w / WC * FR * 16 >> 7) * 4);
      else if (!T)
        sx[j] = *(const float*)(ps + (w % WC * FC * 16 + j * 16 + r16) * 4);
    };
    // Product n of a step is of row_of(n) and column_of(n): the first rows row by row, the
    // others column by column. kTransposed ones are two instructions, the second of them issued after the
    // next product's first, since it waits for its own first. Sums are added kLate products
    // later, those of a step's last ones in the next step, with the scales that were theirs.
    constexpr int kFirst = (FR - P) * FC, kAll = FR * FC;
    auto row_of = [](int n) { return n < kFirst ? n / FC : FR - P + (n - kFirst) % P; };
    auto column_of = [](int n) { return n < kFirst ? n % FC : (n - kFirst) / P; };
    f32x4 part[4];
    static_assert(kAll % 4 == 0 && kLate <= 3, "sums that wait are not overwritten");
    auto add = [&](int n, float by) {
      const int i = row_of(n), j = column_of(n);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[i][j][e] = __builtin_fmaf(part[n % 4][e], by, acc[i][j][e]);
    };
    auto finish = [&](int n) {
      const int x = place(row_of(n)), j = column_of(n);
      if constexpr (T) part[n % 4] = Mul::second(wide[x][1], c[j][1], part[n % 4]);
    };
    auto multiply = [&](int n) {
      const int i = row_of(n), j = column_of(n);
      if constexpr (T)
        part[n % 4] = Mul::first(wide[place(i)][0], c[j][0]);
      else
        part[n % 4] = Mul::block(r[i % NB][0], r[i % NB][1], c[j][0], c[j][1]);
      if (n >= 1) finish(n - 1);
      if (n >= kLate) add(n - kLate, T ? f[0] : f[column_of(n - kLate)]);
    };
    // the rows before the barrier; rows up to i + NB - 1 are read by the end of row i, and widened in
    // the row before their own
    auto first_rows = [&](auto loads, auto later) {
      constexpr bool LOADS = decltype(loads)::value, LATER = decltype(later)::value;
      constexpr int kRest = kLoads - kEarly, kEvery = kFirst / kRest > 0 ? kFirst / kRest : 1;
#pragma unroll
      for (int j = 0; j < FC; ++j) f[j] = T ? sw : sx[j] * sw;
#pragma unroll
      for (int n = 0; n < kFirst; ++n) {
        const int i = n / FC, j = n % FC;
        const int have = i == 0 ? 1 : i + NB - 1, want = i + NB < FR ? i + NB : FR;
#pragma unroll
        for (int x = j; x < 2 * (want - have); x += FC) read_r(have + x / 2, x & 1);
        if (LOADS && n % kEvery == 0 && n / kEvery < kRest) load_n(kEarly + n / kEvery);
        multiply(n);
        if (LATER && n < kLate) add(kAll - kLate + n, old[n]);
        if (T && j == FC / 2 && i + 1 <= FR - P) widen(i + 1);
        if (T && j == FC - 1 && i == FR - P - 1 && P == 2) widen(FR - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (LATER) {
#pragma unroll
        for (int n = kFirst; n < kLate; ++n) add(kAll - kLate + n, old[n]);
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
        // a column's last product: its first half may be read anew, its second one product later
        // if that is still to be multiplied
        if (NEXT && (n - kFirst) % P == P - 1) {
          read_c(column_of(n), 0);
          if (!T) read_c(column_of(n), 1);
        }
        if (T && NEXT && n > kFirst && (n - 1 - kFirst) % P == P - 1) read_c(column_of(n - 1), 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (LOADS) {
#pragma unroll
        for (int x = kAll - kFirst; x < kEarly; ++x) load_n(x);
      }
      finish(kAll - 1);
      if (NEXT) {
        if (T) read_c(FC - 1, 1);
        widen(0);
#pragma unroll
        for (int x = 0; x < kLate; ++x) old[x] = T ? f[0] : f[column_of(kAll - kLate + x)];
      } else {
#pragma unroll
        for (int n = kAll - kLate; n < kAll; ++n) add(n, T ? f[0] : f[column_of(n)]);
      }
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
    widen(0);
    auto advance = [&]() {
      step = step + kStepUnits >= kUnits ? step + kStepUnits - kUnits : step + kStepUnits;
      sslot = sslot == kScaleSlots - 1 ? 0 : sslot + 1;
      point();
    };
    first_rows(no, no);
    int s = 0;
    for (; s + (T ? kDeep : 3) < total; ++s) {
      wait_barrier<kAhead>();
      advance();
      last_rows(yes, yes);
      first_rows(yes, yes);
    }
    for (; s + 1 < total; ++s) {
      if (s + 2 < total)
        wait_barrier<kAhead>();
      else
        wait_barrier<0>();
      advance();
      if (!T && tail && s + 2 == total) zero_tail(lds, step, tail);
      if (!T && s + 2 < total) load_step(false);
      last_rows(no, yes);
      first_rows(no, yes);
    }
    last_rows(no, no);
  }

  // The same for operands of any alignment and stride, through registers, a step being read while
  // the one before is computed. rows(s, r): the bytes of R's row r (kTransposed: of its k r) of
  // step s, `cols` those of C, as {address, first byte, end}, zeros past the end and where the
  // address is null; scale(s, j): f of this lane's column in fragment j.
  struct Bytes {
    const char* p;
    int64_t at, end;
  };
  static constexpr int kAnyLds = 4 * B * kStepBytes;
  template <typename RF, typename CF, typename SF>
  __device__ inline void run_any(int steps, char* lds, RF rows, CF cols, SF scale) {
    constexpr int kR = T ? 64 * B / 16 : B * 8, kC = B * 8;  // chunks of a step
    constexpr int NR = kR / kThreads, NC = kC / kThreads, kER = 1, kEC = T ? 2 : 1;
    static_assert(NR * kThreads == kR && NC * kThreads == kC, "chunks divide over the threads");
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q = lane >> 4, w = wave();
    v4i vr[NR], vc[NC];
    auto load = [&](int s) {
      auto take = [&](const Bytes& x, int chunk, auto es) {
        return x.p ? load_any<decltype(es)::value>(x.p, x.at + chunk * 16, x.end) : v4i{0, 0, 0, 0};
      };
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int e = i * kThreads + tid, per = T ? B / 16 : 8;
        vr[i] = take(rows(s, e / per), e % per, std::integral_constant<int, kER>());
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e = i * kThreads + tid;
        vc[i] = take(cols(s, e >> 3), e & 7, std::integral_constant<int, kEC>());
      }
    };
    auto store = [&](char* to) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int e = i * kThreads + tid;
        if (T)
          *(v4i*)(to + e / (B / 16) * B + (e % (B / 16) ^ swap_at(e / (B / 16))) * 16) = vr[i];
        else
          *(v4i*)(to + (e >> 3) * kStepBytes + chunk_at(e >> 3, e & 7) * 16) = vr[i];
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e = i * kThreads + tid;
        *(v4i*)(to + (B + (e >> 3)) * kStepBytes + chunk_at(e >> 3, e & 7) * 16) = vc[i];
      }
    };
    if (steps > 0) {
      load(0);
      store(lds);
    }
    __syncthreads();
    const int wr = w / WC * FR * 16, wc = w % WC * FC * 16;
    for (int s = 0; s < steps; ++s) {
      if (s + 1 < steps) load(s + 1);
      const char *lr = lds + (s & 1) * 2 * B * kStepBytes, *lc = lr + B * kStepBytes;
      v4i c[FC][2];
      float f[FC];
#pragma unroll
      for (int j = 0; j < FC; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          c[j][h] = *(const v4i*)(lc + (wc + j * 16 + r16) * kStepBytes + chunk_at(r16, h * 4 + q) * 16);
        f[j] = scale(s, j);
      }
#pragma unroll
      for (int i = 0; i < FR; ++i) {
        v4i x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (T) {
            v4i codes = {0, 0, 0, 0};
            const int kt = 32 * h + 8 * q;
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // byte by byte: plain, and few calls come here
              const int k = kt + e, at = (wr / 16 + i) ^ swap_at(k);
              codes[e / 4] |= (int)*(const unsigned char*)(lr + k * B + at * 16 + r16) << (8 * (e % 4));
            }
            v4i none;
            Mul::widen(codes, x[h], none);  // the first 8 k of the two
          } else {
            x[h] = *(const v4i*)(lr + (wr + i * 16 + r16) * kStepBytes + chunk_at(r16, h * 4 + q) * 16);
          }
        }
#pragma unroll
        for (int j = 0; j < FC; ++j) {
          const f32x4 p = Mul::block(x[0], x[1], c[j][0], c[j][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], f[j], acc[i][j][e]);
        }
      }
      if (s + 1 < steps) store(lds + ((s + 1) & 1) * 2 * B * kStepBytes);
      __syncthreads();
    }
  }
};

}  // namespace bk
