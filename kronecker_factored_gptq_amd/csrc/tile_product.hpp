// The tiled matrix product behind the int8 product, its input gradient and the
// cross entropy:
//   D[r][c] = sum over pairs p of sum_k R_p[r][k] C_p[c][k]
// of two operands whose rows run along k (both k-contiguous), on 16x16 MFMA.
//
// Everything about the layout is counted in bytes, so one template serves
// int8 (64 k per instruction), bfloat16 and float16 (32 k): each takes 64
// bytes of k per operand row and instruction, lane l holding 16 bytes of row
// l % 16, and both operands are given the same k per lane, so the order of k
// inside an instruction does not matter. The result's lane l, register i holds
// D[4 * (l / 16) + i][l % 16].
//
// What bounds a large product: with 256 x 256 tiles a step (128 bytes of k) is 64
// matrix instructions of 16 cycles on each of two waves a SIMD, 24 LDS reads a wave
// and 64 KB from the L2. The instructions alone run at 4.3e15 op/s (int8 codes)
// and 2.2e15 flop/s (bfloat16) here; the loads alone would take 0.85 of the int8
// product's time and 0.55 of a bfloat16 one's, so they have to flow all the time: the
// ring of five slots (against two whole steps: 393 -> 380 us for 8192 x 14336 x
// 4096 int8), the loads spread over the step (cross entropy's gradient 11.8 -> 11.3
// ms), the LDS reads among the multiplications (412 -> 393). Four waves of 128 x
// 128 read less LDS but leave one wave to a SIMD and cost register copies: 432 us.
//
// Pairs of planes: a float32 operand is held as bfloat16 planes x = x1 + x2 +
// x3 (exact, 8 bits each, split_bf16), and a product is the sum over the pairs
// of planes whose terms reach the result's precision, all added into the same
// float32 accumulators (PlanePairs). A bfloat16, float16 or int8 product is
// the single pair (0, 0).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace bk {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

struct MmaI8 {
  typedef v4i acc_t;
  static constexpr int kElem = 1;
  __device__ static inline acc_t mma(v4i a, v4i b, acc_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};
struct MmaBF16 {
  typedef f32x4 acc_t;
  static constexpr int kElem = 2;
  __device__ static inline acc_t mma(v4i a, v4i b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};
struct MmaF16 {
  typedef f32x4 acc_t;
  static constexpr int kElem = 2;
  __device__ static inline acc_t mma(v4i a, v4i b, acc_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  }
};
// float32 itself, four k at a time (at a sixteenth of bfloat16's rate): for
// products bound by reading their operands.
struct MmaF32 {
  typedef f32x4 acc_t;
  static constexpr int kElem = 4;
  __device__ static inline acc_t mma(v4i a, v4i b, acc_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(a[e]), __int_as_float(b[e]), c, 0, 0,
                                               0);
    return c;
  }
};

// One operand, in planes `plane` bytes apart: `rows` rows of a product's kbytes
// bytes, `ld` bytes apart; or k-major: `krows` rows of k, `ld` bytes apart, each
// holding that k of all `rows`, readable up to a multiple of 16 bytes.
struct TileOperand {
  const char* p;
  int64_t ld, plane, rows, krows;
};

// The largest row stride (and row length, in bytes) the direct loads take: the
// 32-bit offsets inside a tile of 256 rows stay below 2^31.
constexpr int64_t kTileMaxLd = (int64_t)1 << 22;
constexpr int kStepBytes = 128;  // bytes of k per row and pipeline step

// Whether the direct loads (TileProduct::run) can take an operand.
inline bool tile_direct(const TileOperand& o, int64_t kbytes) {
  return (uintptr_t)o.p % 16 == 0 && o.ld % 16 == 0 && o.plane % 16 == 0 && kbytes % 16 == 0 &&
         o.ld <= kTileMaxLd && kbytes <= kTileMaxLd;
}

// The block of tiles that workgroup b of `nr` x `nc` works on. Workgroups go
// to the 8 XCDs in turn, so each XCD is given a contiguous run of the tile
// order, and the order walks groups of 8 c-tiles r-tile by r-tile: the tiles
// that run together on an XCD share operand rows in its L2.
__device__ inline void tile_of(unsigned b, unsigned nr, unsigned nc, int& tr, int& tc) {
  const unsigned total = nr * nc, q = total / 8, rem = total % 8;
  const unsigned x = b % 8, i = b / 8;
  const unsigned t = x * q + (x < rem ? x : rem) + i;
  const unsigned group = t / (8 * nr), first = group * 8;
  const unsigned width = nc - first < 8 ? nc - first : 8;
  const unsigned in = t - first * nr;
  tr = (int)(in / width);
  tc = (int)(first + in % width);
}

// 16 bytes of a row from byte k on, of any alignment; past kbytes they are zero
// (elements of E bytes, each wholly inside or outside).
template <int E>
__device__ inline v4i load_any(const char* row, int64_t k, int64_t kbytes) {
  v4i v = {0, 0, 0, 0};
  if (k + 16 <= kbytes) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
    unsigned w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; e += E)
      if (k + e < kbytes) {
        unsigned x;
        if (E == 1)
          x = *(const unsigned char*)(row + k + e);
        else if (E == 2)
          x = *(const unsigned short*)(row + k + e);
        else
          x = *(const unsigned*)(row + k + e);
        w[e / 4] |= x << (8 * (e % 4));
      }
    v = v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
  }
  return v;
}

// How an operand lies in memory and in LDS: its rows along k (kbytes of k in
// each), or k-major (k its rows, `ld` apart, its tile's rows side by side).
template <class M, int BR, int BC, int WR, int WC, bool RK = false, bool CK = false,
          int SLOTS = 5>
struct TileProduct {
  typedef typename M::acc_t acc_t;
  static constexpr int kWaves = WR * WC;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int FR = BR / WR / 16, FC = BC / WC / 16;
  // LDS is a ring of SLOTS = 2 D + 1 slots, each one step of one operand: step s of
  // R in slot 2 s mod SLOTS, of C in the next. With whole steps only, every load
  // of a step would have to land before the next go out; the odd slot keeps R of
  // one more step in flight meanwhile, and the memory path busy.
  static constexpr int kSlot = BR * kStepBytes;
  static constexpr int kLds = SLOTS * kSlot;
  static constexpr int D = SLOTS / 2;
  static_assert(SLOTS % 2 == 1 && D >= 2, "whole steps and one more");
  static_assert(BR == BC, "one slot size");
  static constexpr int LR = BR * kStepBytes / 1024 / kWaves;  // wave loads per step
  static constexpr int LC = BC * kStepBytes / 1024 / kWaves;
  static_assert(LR * kWaves * 1024 == BR * kStepBytes && LC * kWaves * 1024 == BC * kStepBytes,
                "a step's bytes divide over the waves");
  static_assert(kWaves % 2 == 0, "the chunk order of a wave's loads does not depend on the load");
  static_assert(!(RK || CK) || M::kElem == 2, "the transposing reads are of 16-bit elements");

  acc_t acc[FR][FC];
  // both operands for one instruction's k (64 bytes of it)
  struct Frags {
    v4i r[FR], c[FC];
  };

  __device__ inline int wave_r() const { return (threadIdx.x >> 6) / WC * (FR * 16); }
  __device__ inline int wave_c() const { return (threadIdx.x >> 6) % WC * (FC * 16); }

  // LDS holds a k-contiguous operand's rows 128 bytes apart; 16-byte chunk q of
  // row r lies at position q ^ ((r / 2) % 8), so that the 16 rows a fragment
  // reads at one q fall on different banks.
  __device__ static inline int chunk_at(int row, int pos) { return pos ^ ((row >> 1) & 7); }

  // A k-major operand lies k by k, 2 B bytes each. Of a transposing read, four
  // lanes take 32 bytes of one k, 16 lanes four k, and the next 16 lanes k that
  // are 8 further; the 32-byte block b of k lies at b ^ swap_at(k), so that 32
  // lanes cover 256 bytes of banks once (with B = 64, k and k + 1 share them).
  template <int B> __device__ static inline int swap_at(int k) {
    return B >= 128 ? (k & 3) | ((k >> 1) & 4) : ((k >> 1) & 1) | ((k >> 2) & 2);
  }

  // Fragment i of the operand whose wave's rows start at row0.
  template <bool K, int B>
  __device__ static inline v4i read_one(const char* lds, int row0, int kk, int i) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
    if (!K)
      return *(const v4i*)(lds + (row0 + i * 16 + r16) * kStepBytes +
                           chunk_at(r16, kk * 4 + q) * 16);
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const int k = 8 * q + (r16 >> 2);  // and 4 further, of 32 kk on
    // block row0 / 16 + i, the first a multiple of the wave's fragments
    const int at = k * (2 * B) + ((row0 / 16) ^ swap_at<B>(k)) * 32 + (r16 & 3) * 8;
    const char* a = lds + (at ^ (i * 32)) + kk * 64 * B;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)a);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(a + 8 * B));
    const int2 x = __builtin_bit_cast(int2, lo), y = __builtin_bit_cast(int2, hi);
    return v4i{x.x, x.y, y.x, y.y};
  }
  __device__ inline void read(Frags& f, const char* lr, const char* lc, int kk, int g) const {
    if (g < FC)
      f.c[g] = read_one<CK, BC>(lc, wave_c(), kk, g);
    else
      f.r[g - FC] = read_one<RK, BR>(lr, wave_r(), kk, g - FC);
  }
  __device__ inline void read(Frags& f, const char* lr, const char* lc, int kk) const {
#pragma unroll
    for (int g = 0; g < FR + FC; ++g) read(f, lr, lc, kk, g);
  }
  __device__ inline void multiply(const Frags& f, int g) {
    const int i = g / FC, j = g % FC;
    acc[i][j] = M::mma(f.r[i], f.c[j], acc[i][j]);
  }
  __device__ inline void multiply(const Frags& f) {
#pragma unroll
    for (int g = 0; g < FR * FC; ++g) {
      multiply(f, g);
      if (g % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // in order: registers
    }
  }
  // Multiplies `f` while `next` is read, and LOADS wave loads (load(u)) go out.
  // The order is fixed here: one LDS read to two multiplications, and the loads
  // evenly among all of them. The address units take 16 cycles for a wave load
  // and all waves issue theirs in the same half step; closer together they
  // would hold up the multiplications behind them.
  template <int LOADS, typename F>
  __device__ inline void half_step(const Frags& f, Frags& next, const char* lr, const char* lc,
                                   int kk, F load) {
    constexpr int kMma = FR * FC, kReads = FR + FC;
    constexpr int kPer = kMma >= 2 * kReads ? 2 : 1;
    constexpr int kEvery = LOADS ? kMma / (LOADS ? LOADS : 1) : kMma + 1;
    static_assert(kEvery >= 1, "a multiplication to each load");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < kMma; ++g) {
      if (g % kPer == 0 && g / kPer < kReads) read(next, lr, lc, kk, g / kPer);
      if (g % kEvery == 0 && g / kEvery < LOADS) load(g / kEvery);
      multiply(f, g);
      if ((g + 1) % kPer == 0) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < kReads; ++u)
      if (u * kPer >= kMma) read(next, lr, lc, kk, u);
    __builtin_amdgcn_sched_barrier(0);
  }

  __device__ inline void zero() {
#pragma unroll
    for (int i = 0; i < FR; ++i)
#pragma unroll
      for (int j = 0; j < FC; ++j) acc[i][j] = acc_t{0, 0, 0, 0};
  }

  // 64 lanes x 16 bytes from global memory straight into LDS at `lds` + 16 *
  // lane. No register is loaded, so the instruction can stand by itself: as a
  // builtin it makes the compiler wait for every such load in flight before a
  // transposing LDS read, which is what run()'s own waits are there to avoid.
  // m0 holds the LDS address; as an operand the compiler sets it and knows that it did.
  // (s_nop: the wait states from a register write to its use as an address.)
  __device__ static inline void load_lds(v4i rsrc, int voff, int soff, unsigned lds) {
    asm volatile(
        "s_nop 4\n\t"
        "buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff),
        "s"(rsrc), "s"(soff), "{m0}"(lds)
        : "memory");
  }

  // One operand's loads: a lane's byte offsets for each of a step's NL wave
  // loads. LDS is written in lane order, so each lane fetches the chunk that
  // belongs at its place. Rows past the operand's last are read as its last
  // (their results are not for storing); chunks past the end of k get an
  // offset past the buffer's end and read as zero, and so do a k-major operand's
  // chunks past its rows.
  template <bool K, int B, int NL>
  struct Loader {
    const char* p;  // k-major: of the next step
    const char* first;
    int64_t plane, kstride;
    int bytes;
    int off[NL];
    int krow;       // k-major: this lane's k of the first load
    bool past;      // this lane's chunk is past the end in the last k step
    int ksteps, k, pair, npairs;  // the next step to load
    unsigned lds, slot;           // this wave's place in slot 0; the next slot
    unsigned planes;
    v4i rsrc;

    __device__ inline void init(const TileOperand& o, int64_t row0, int64_t kbytes, int npairs_,
                                unsigned planes_, int step0, unsigned lds_,
                                unsigned slot_) {
      const int lane = threadIdx.x & 63;
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      const int rows = o.rows - row0 < B ? (int)(o.rows - row0) : B, ld = (int)o.ld;
      plane = o.plane;
      ksteps = (int)((kbytes + kStepBytes - 1) / kStepBytes);
      npairs = npairs_;
      planes = planes_;
      lds = lds_ + wave * 1024;
      slot = slot_;
      if (!K) {
        first = o.p + row0 * o.ld;
        bytes = (rows - 1) * ld + (int)kbytes;
        const int row8 = lane >> 3, chunk = chunk_at((wave & 1) * 8 + row8, lane & 7);
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const int r = (j * kWaves + wave) * 8 + row8;
          off[j] = (r < rows ? r : rows - 1) * ld + chunk * 16;
        }
        past = chunk * 16 + (ksteps - 1) * kStepBytes >= (int)kbytes;
      } else {
        first = o.p + row0 * 2;
        kstride = 64 * o.ld;  // past 32 bits over all steps, so the buffer moves along
        bytes = 63 * ld + (rows + 7) / 8 * 16;  // whole chunks: the rows are padded to them
        constexpr int per = B / 8;  // chunks of a k; kLanesK k in a wave load
        constexpr int lanes_k = 64 / per;
        krow = lane / per;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const int kr = (j * kWaves + wave) * lanes_k + krow, pos = lane % per;
          const int chunk = ((pos >> 1) ^ swap_at<B>(kr)) * 2 + (pos & 1);
          off[j] = chunk * 8 < rows ? kr * ld + chunk * 16 : (int)0x80000000;
        }
        krow += wave * lanes_k + (ksteps - 1) * 64 - (int)o.krows;  // >= 0: past the last k
      }
      pair = __builtin_amdgcn_readfirstlane(step0 / ksteps);
      k = step0 - pair * ksteps;
      select(planes >> 4 * pair & 15);
    }
    __device__ inline void select(int pl) {
      p = first + pl * plane;
      if (K) p += k * kstride;
      point();
    }
    __device__ inline void point() {
      const uint64_t a = (uint64_t)p;
      rsrc[0] = __builtin_amdgcn_readfirstlane((int)(unsigned)a);
      rsrc[1] = __builtin_amdgcn_readfirstlane((int)(unsigned)(a >> 32) & 0xffff);
      rsrc[2] = __builtin_amdgcn_readfirstlane(bytes);
      rsrc[3] = 0x00020000;
    }
    __device__ inline void load(int j) const {
      const bool last = k == ksteps - 1;
      bool cut = last && past;
      if (K) cut = last && krow + j * kWaves * (64 / (B / 8)) >= 0;
      load_lds(rsrc, cut ? (int)0x80000000 : off[j], K ? 0 : k * kStepBytes,
               lds + slot * kSlot + j * kWaves * 1024);
    }
    __device__ inline void advance() {
      slot = slot + 2 >= SLOTS ? slot + 2 - SLOTS : slot + 2;
      if (++k == ksteps && pair + 1 < npairs) {
        k = 0;
        ++pair;
        select(planes >> 4 * pair & 15);
      } else if (K) {
        p += kstride;
        point();
      }
    }
  };

  template <int N> __device__ static inline void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
  }

  // The number of steps of a product.
  __device__ static inline int steps(int64_t kbytes, const PlanePairs& pairs) {
    return (int)((kbytes + kStepBytes - 1) / kStepBytes) * pairs.n;
  }

  // D's tile at (r0, c0), summed over the product's steps [s0, s1); operands as
  // tile_direct wants them, kbytes of k.
  __device__ inline void run(const TileOperand& R, const TileOperand& C, int64_t kbytes,
                             const PlanePairs& pairs, int64_t r0, int64_t c0, int s0, int s1,
                             char* lds) {
    s0 = __builtin_amdgcn_readfirstlane(s0);
    const int total = __builtin_amdgcn_readfirstlane(s1) - s0;
    if (total <= 0) return;
    const unsigned base = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    Loader<RK, BR, LR> lr;
    Loader<CK, BC, LC> lc;
    lr.init(R, r0, kbytes, pairs.n, pairs.r, s0, base, 0);
    lc.init(C, c0, kbytes, pairs.n, pairs.c, s0, base, 1);
    auto load_r = [&]() {
#pragma unroll
      for (int u = 0; u < LR; ++u) lr.load(u);
      lr.advance();
    };
    auto load_c = [&]() {
#pragma unroll
      for (int u = 0; u < LC; ++u) lc.load(u);
      lc.advance();
    };
    auto none = [](int) {};

#pragma unroll
    for (int u = 0; u <= D; ++u) {  // steps 0 to D - 1, and R of step D
      if (u < total) load_r();
      if (u < D && u < total) load_c();
    }
    if (total > D)
      wait_barrier<D * LR + (D - 1) * LC>();
    else
      wait_barrier<0>();
    // A step's second half is multiplied while the next step's first half is
    // read from LDS, and its first half while its second half is read. In
    // between all waves have read the step, and its slots are loaded anew: with C
    // of step s + D in this half, R of step s + D + 1 in the next.
    unsigned slot = 0;  // of this step's R
    const char *pr = lds, *pc = lds + kSlot;
    auto next_slots = [&]() {
      slot = slot + 2 >= SLOTS ? slot + 2 - SLOTS : slot + 2;
      pr = lds + slot * kSlot;
      pc = slot == SLOTS - 1 ? lds : pr + kSlot;
    };
    Frags a, b;
    read(a, pr, pc, 0);
    auto next_r = [&](int u) { lr.load(u); };
    auto next_c = [&](int u) { lc.load(u); };
    int s = 0;
    half_step<0>(a, b, pr, pc, 1, none);
    // the next step has landed; what was issued after its C may be in flight
    constexpr int kAhead = (D - 1) * LR + (D - 2) * LC;
    for (; s < total - D - 1; ++s) {
      wait_barrier<kAhead>();
      next_slots();
      half_step<LC>(b, a, pr, pc, 0, next_c);
      lc.advance();
      half_step<LR>(a, b, pr, pc, 1, next_r);
      lr.advance();
    }
    for (; s < total - 1; ++s) {
      if (s == total - D - 1)
        wait_barrier<kAhead>();
      else
        wait_barrier<0>();
      next_slots();
      if (s == total - D - 1) load_c();  // the last step's
      half_step<0>(b, a, pr, pc, 0, none);
      half_step<0>(a, b, pr, pc, 1, none);
    }
    multiply(b);
  }

  // The same for operands of any alignment, stride and k (M::kElem-sized
  // elements): a step is read to registers while the one before is computed, and
  // then written to LDS.
  __device__ inline void run_any(const TileOperand& R, const TileOperand& C, int64_t kbytes,
                                 int64_t r0, int64_t c0, char* lds) {
    const int tid = threadIdx.x;
    const int64_t rows = R.rows - r0 < BR ? R.rows - r0 : BR;
    const int64_t cols = C.rows - c0 < BC ? C.rows - c0 : BC;
    constexpr int NR = BR * 8 / kThreads, NC = BC * 8 / kThreads;
    v4i vr[NR], vc[NC];
    auto gload = [&](int64_t k) {
#pragma unroll
      for (int u = 0; u < NR; ++u) {
        const int e = u * kThreads + tid, r = e >> 3;
        vr[u] = load_any<M::kElem>(R.p + (r0 + (r < rows ? r : rows - 1)) * R.ld, k + (e & 7) * 16, kbytes);
      }
#pragma unroll
      for (int u = 0; u < NC; ++u) {
        const int e = u * kThreads + tid, r = e >> 3;
        vc[u] = load_any<M::kElem>(C.p + (c0 + (r < cols ? r : cols - 1)) * C.ld, k + (e & 7) * 16, kbytes);
      }
    };
    auto sstore = [&](char* b) {
#pragma unroll
      for (int u = 0; u < NR; ++u) {
        const int e = u * kThreads + tid, r = e >> 3;
        *(v4i*)(b + r * kStepBytes + chunk_at(r, e & 7) * 16) = vr[u];
      }
#pragma unroll
      for (int u = 0; u < NC; ++u) {
        const int e = u * kThreads + tid, r = e >> 3;
        *(v4i*)(b + (BR + r) * kStepBytes + chunk_at(r, e & 7) * 16) = vc[u];
      }
    };
    const int ksteps = (int)((kbytes + kStepBytes - 1) / kStepBytes);
    if (ksteps > 0) {
      gload(0);
      sstore(lds);
    }
    __syncthreads();
    for (int s = 0; s < ksteps; ++s) {
      if (s + 1 < ksteps) gload((int64_t)(s + 1) * kStepBytes);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        Frags f;
        read(f, lds + (s & 1) * 2 * kSlot, lds + ((s & 1) * 2 + 1) * kSlot, kk);
        multiply(f);
      }
      if (s + 1 < ksteps) sstore(lds + ((s + 1) & 1) * 2 * kSlot);
      __syncthreads();
    }
  }
};

// ---- element types ----------------------------------------------------------
struct BF16 {
  unsigned short v;
};
struct F16 {
  _Float16 v;
};
__device__ inline float to_f32(float x) { return x; }
__device__ inline float to_f32(BF16 x) { return __uint_as_float((unsigned)x.v << 16); }
__device__ inline float to_f32(F16 x) { return (float)x.v; }

// Round to nearest even; a NaN stays a NaN.
template <typename T> __device__ inline T from_f32(float x);
template <> __device__ inline float from_f32<float>(float x) { return x; }
template <> __device__ inline BF16 from_f32<BF16>(float x) {
  const __bf16 b = (__bf16)x;
  return BF16{__builtin_bit_cast(unsigned short, b)};
}
template <> __device__ inline F16 from_f32<F16>(float x) { return F16{(_Float16)x}; }

// Four consecutive outputs as one store.
template <typename O> struct Vec4;
template <> struct Vec4<float> {
  typedef float type __attribute__((ext_vector_type(4)));
};
template <> struct Vec4<BF16> {
  typedef unsigned short type __attribute__((ext_vector_type(4)));
};
template <> struct Vec4<F16> {
  typedef unsigned short type __attribute__((ext_vector_type(4)));
};
// whether every group of four columns of Y starts at a multiple of its size
template <typename O>
inline bool vec4_ok(const O* y, int64_t ld) {
  return (uintptr_t)y % (4 * sizeof(O)) == 0 && ld % 4 == 0;
}

// A tile's results to Y[c][r .. r + 3] (row stride ldy): f(value, i, j, e) of
// each accumulator element, rounded to O. `vec`: vec4_ok.
template <class TP, typename O, typename F>
__device__ inline void store_tile(const TP& tp, int64_t r0, int64_t c0, int64_t rows, int64_t cols,
                                  O* __restrict__ Y, int64_t ldy, bool vec, F f) {
  const int lane = threadIdx.x & 63;
  const int64_t rb = r0 + tp.wave_r() + 4 * (lane >> 4), cb = c0 + tp.wave_c() + (lane & 15);
  if (vec && r0 + tp.wave_r() + TP::FR * 16 <= rows) {
#pragma unroll
    for (int j = 0; j < TP::FC; ++j) {
      if (cb + j * 16 >= cols) continue;
      O* p = Y + (cb + j * 16) * ldy + rb;
#pragma unroll
      for (int i = 0; i < TP::FR; ++i) {
        O t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = from_f32<O>(f(tp.acc[i][j][e], i, j, e));
        *(typename Vec4<O>::type*)(p + i * 16) = __builtin_bit_cast(typename Vec4<O>::type, t);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < TP::FC; ++j)
#pragma unroll
      for (int i = 0; i < TP::FR; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (cb + j * 16 < cols && rb + i * 16 + e < rows)
            Y[(cb + j * 16) * ldy + rb + i * 16 + e] = from_f32<O>(f(tp.acc[i][j][e], i, j, e));
  }
}

// A tile's sums as they are to parts[c][r .. r + 3], rows ldp (a multiple of four,
// at least `rows`) 4-byte words apart, 16-byte aligned.
template <class TP>
__device__ inline void store_sums(const TP& tp, int64_t r0, int64_t c0, int64_t cols, void* parts,
                                  int64_t ldp) {
  const int lane = threadIdx.x & 63;
  const int64_t rb = r0 + tp.wave_r() + 4 * (lane >> 4), cb = c0 + tp.wave_c() + (lane & 15);
#pragma unroll
  for (int j = 0; j < TP::FC; ++j) {
    if (cb + j * 16 >= cols) continue;
#pragma unroll
    for (int i = 0; i < TP::FR; ++i)
      if (rb + i * 16 < ldp)
        *(typename TP::acc_t*)((int*)parts + (cb + j * 16) * ldp + rb + i * 16) = tp.acc[i][j];
  }
}

// The sums of a k that was split: four words of each range, `stride` words apart, added in
// range order. Bound by memory where there are many outputs and by latency where there are
// few, so four ranges are on their way at once, and with S > 1 the workgroup of 256 has S
// threads to each group of four words (`at`), thread y of them taking ranges y, y + S, ...,
// whose sums meet in `red` in the order of y. True for the thread that holds the result.
template <int S>
struct JoinAt {
  static constexpr int kGroups = 256 / S;
  __device__ static inline int64_t at() {
    return (int64_t)blockIdx.x * kGroups + threadIdx.x % kGroups;
  }
};
template <int S, typename V>
__device__ inline bool join_ranges(const void* first, int64_t stride, int splits, bool inside, V& a,
                                   V* red) {
  const int y = threadIdx.x / JoinAt<S>::kGroups;
  const int* p = (const int*)first;
  auto range = [&](int k) { return *(const V*)(p + k * stride); };
  a = V{0, 0, 0, 0};
  if (inside) {
    int k = y;
    for (; k + 3 * S < splits; k += 4 * S) {
      V b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = range(k + i * S);
#pragma unroll
      for (int i = 0; i < 4; ++i) a += b[i];
    }
    if (k + 2 * S < splits) {
      const V b = range(k), c = range(k + S), d = range(k + 2 * S);
      a = a + b + c + d;
    } else if (k + S < splits) {
      const V b = range(k), c = range(k + S);
      a = a + b + c;
    } else if (k < splits) {
      a += range(k);
    }
  }
  if (S == 1) return inside;
  red[threadIdx.x] = a;
  __syncthreads();
  if (y > 0 || !inside) return false;
#pragma unroll
  for (int i = 1; i < S; ++i) a += red[i * JoinAt<S>::kGroups + threadIdx.x];
  return true;
}
// Threads to a group. Input gradients, one against eight: 1 x 40000 x 64 bfloat16 in 256
// ranges 40.7 and 25.7 us, in 16 37.1 and 36.4; 200 x 14336 x 512 in 24 30.8 and 29.8; 16 x
// 14336 x 4096 in 12 56.2 and 55.7. With few ranges of many outputs one is as fast or
// faster (512 x 14336 x 1024 float32 in 4: 108.2 and 109.3).
inline int join_slices(int splits) { return splits < 12 ? 1 : 8; }

// The tile of a product, and the ranges its k is split into. 256 x 256 tiles
// (one workgroup a CU) need the fewest bytes and are taken where they fill the
// chip without more than a quarter of empty rows and columns beyond those of 128 x 128
// (131072 x 2048 int8, us with 256 and without: 20 columns 61 and 45, 128 71 and 59, 300 143
// and 132; 256 85 and 86; float32 input gradient 1 x 1024 x 65536 108 and 96, the cross
// entropy's of 1 x 512 x 128256 521 and 457). Otherwise the choice is by an estimate of the
// time in us, of 128 x 128 tiles (two workgroups a CU) and 64 x 64 tiles (four):
// - with c workgroups on each CU a step takes step + share c (bound by the L2), and
//   at least `alone` (bound by latency); k-major operands 0.15 more of the
//   small tile; filling the ring and the epilogue take `fill`;
// - k split into n ranges, each summed apart: `join` for the kernel that joins
//   them, `range` for each of them, and their sums, written and read again, at `rate` bytes a ps.
// The constants are fitted to measurements: of int8 products over 1000 x 1504 to
// 28672 x 4096 with 20 to 800 columns, the 128 and 64 tiles of each with up to 16 ranges,
// weights from memory (of those the choice is within 0.6% of the best one on average; fitted to
// fewer it was 5%). For several pairs of planes, which read the same planes again and
// again, they are of float32 gradients: with the other constants the cross entropy's of 333 x
// 1000 x 10007 takes 237 us, not 214, and that of 2048 x 512 x 8000 382, not 354, though that of
// 512 x 1024 x 32000 takes 663, not 701. Every division that may be taken is compared: over
// 60 sizes each, a search that gave a tile up once it was twice as slow as the other tile's best
// cost int8 products 1.2 % on average (304 x 113 x 14592: 11.1 us, now 9.2), float32 input
// gradients 3 % (1 x 9664 x 256: 17.0, now 14.3), the float32 cross entropy gradient 1.5 %.
struct TileCost {
  double step, share, alone, fill;
};
struct PlanCosts {
  TileCost tile[2];  // 128 x 128, 64 x 64
  double join, range, rate;
};
constexpr PlanCosts kCostsOne = {{{0.15, 0.48, 0.61, 2.2}, {0.1, 0.26, 0.29, 1.5}}, 2.2, 0.02, 2.2};
constexpr PlanCosts kCostsPairs = {{{0.28, 0.4, 0.5, 3}, {0.19, 0.175, 0.35, 1}}, 3, 0.02, 3.5};
// Products with block scales (block_tile.hpp), fitted to 28 sizes of 1024 x 2048 to 14336 x 4096 with
// 100 to 2048 rows: 8-bit and 16-bit instructions, and 8-bit codes on 16-bit ones.
constexpr PlanCosts kCostsBlocks = {{{0.26, 0.47, 0.72, 3}, {0.15, 0.19, 0.5, 2.5}}, 6, 0.02, 4};
constexpr PlanCosts kCostsExact = {{{0.4, 0.9, 1.2, 3}, {0.25, 0.36, 0.6, 2.5}}, 6, 0.02, 4};
struct TilePlan {
  int tile, splits;
};
inline int64_t tiles_of(int64_t M, int64_t N, int64_t tile) {
  return ((M + tile - 1) / tile) * ((N + tile - 1) / tile);
}
// Whether tiles of 128 or 64 may have their k in n ranges: all at once on the chip, two steps
// of all pairs each at least.
inline bool plan_fits(int64_t M, int64_t N, int64_t steps, bool may_split, int tile, int64_t n) {
  return n == 1 || (may_split && n * tiles_of(M, N, tile) <= (tile == 64 ? 1024 : 512) && n <= steps / 2);
}
// The numbers of ranges: every one for a single pair; 1, 2 and multiples of three for three or
// six pairs, whose ranges then meet the same k at the same time, in different planes or the
// same (input gradient 64 x 14336 x 1024: 20 ranges 38.4 us, 24 32.7, 28 36.6; dX of 333 x 1000 x
// 10007: 16 158 us, 18 142, 20 156, 21 139; of 512 x 1024 x 32000: 14 523, 15 476, 16 514).
inline int plan_next(int pairs, int n) { return n + (pairs > 1 && n >= 3 ? 3 : 1); }
inline bool plan_allowed(int64_t M, int64_t N, int64_t steps, int pairs, bool may_split, int tile,
                         int64_t n) {
  return (pairs == 1 || n < 3 || n % 3 == 0) && plan_fits(M, N, steps, may_split, tile, n);
}
// The estimate, for `steps` of all pairs; `joining`: the part of it that grows with n.
inline double plan_us(int64_t M, int64_t N, int64_t steps, int pairs, bool kmajor, int tile, int64_t n,
                      double* joining = nullptr, const PlanCosts* own = nullptr) {
  const PlanCosts& costs = own ? *own : pairs > 1 ? kCostsPairs : kCostsOne;
  const bool small = tile == 64;
  const TileCost& cost = costs.tile[small];
  const int64_t work = n * tiles_of(M, N, tile), slots = small ? 1024 : 512;
  const int64_t rounds = (work + slots - 1) / slots;
  const double c = (double)(rounds > 1 ? slots : work) / 256;
  double each = cost.step + cost.share * c;
  if (each < cost.alone) each = cost.alone;
  if (small && kmajor) each += 0.15;
  const double sums = (double)M * (double)N * 8 / (costs.rate * 1e6);
  const double join = cost.fill + (n > 1 ? costs.join + (double)n * (sums + costs.range) : 0);
  if (joining) *joining = join;
  return (double)rounds * each * (double)((steps + n - 1) / n) + join;
}
// steps: of one pair.
inline TilePlan plan_tiles(int64_t M, int64_t N, int64_t steps, int pairs, bool kmajor,
                           bool may_split, const PlanCosts* own = nullptr) {
  TilePlan best = {128, 1};
  if (M <= 0 || N <= 0) return best;
  const int64_t large = tiles_of(M, N, 256);
  if (large >= 192 && 32 * large <= 10 * tiles_of(M, N, 128)) return {256, 1};
  steps *= pairs;
  double least = 1e300;
  for (int tile : {128, 64})
    for (int n = 1; plan_fits(M, N, steps, may_split, tile, n); n = plan_next(pairs, n)) {
      double joining;
      const double t = plan_us(M, N, steps, pairs, kmajor, tile, n, &joining, own);
      if (t < least) {
        least = t;
        best = {tile, n};
      }
      if (joining > least) break;  // and so for every larger n
    }
  return best;
}
// words of the ranges' sums, rows of M padded to four
inline int64_t split_words(int64_t M, int64_t N, int splits) {
  return splits > 1 ? splits * N * ((M + 3) / 4 * 4) : 0;
}

// ---- planes -----------------------------------------------------------------
// How a matrix is held for the 16-bit instructions: as one bfloat16 plane, as three (a
// float32 value with all of its 24 bits), or as float16.
enum Split { kBF16x1, kBF16x3, kF16x1 };
constexpr int kPlanes[] = {1, 3, 1};

// The planes' 16-bit words of x. The first ones are truncated, so that each
// rest is exact and no finite x overflows; an infinity or a NaN stands in the
// first plane alone.
template <int KIND>
__device__ inline void split16(float x, unsigned short* w) {
  if (KIND == kF16x1) {
    w[0] = __builtin_bit_cast(unsigned short, (_Float16)x);
  } else if (KIND == kBF16x1) {
    w[0] = from_f32<BF16>(x).v;
  } else {
    const unsigned u = __float_as_uint(x);
    if ((u & 0x7f800000u) == 0x7f800000u) {
      w[0] = from_f32<BF16>(x).v;
      w[1] = w[2] = 0;
      return;
    }
    w[0] = (unsigned short)(u >> 16);
    const float r = x - __uint_as_float(u & 0xffff0000u);
    const unsigned v = __float_as_uint(r);
    w[1] = (unsigned short)(v >> 16);
    w[2] = from_f32<BF16>(r - __uint_as_float(v & 0xffff0000u)).v;
  }
}

// ---- rows ---------------------------------------------------------------------
// Eight elements of a row from column c on, zero past `cols`; `vec` (load8_ok):
// groups of eight are aligned to their size, or to 16 bytes.
template <typename X> struct Eight {
  X v[8];
};
template <typename X> constexpr int kLoadBytes = 8 * sizeof(X) < 16 ? 8 * sizeof(X) : 16;
template <typename X>
__device__ inline Eight<X> load8(const X* row, int64_t c, int64_t cols, bool vec) {
  Eight<X> t;
  if (vec && c + 8 <= cols) {
    constexpr int kPer = kLoadBytes<X> / sizeof(X);
#pragma unroll
    for (int i = 0; i < 8; i += kPer)
      __builtin_memcpy(t.v + i, __builtin_assume_aligned(row + c + i, kLoadBytes<X>),
                       kLoadBytes<X>);
  } else {
    __builtin_memset(&t, 0, sizeof t);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) t.v[i] = row[c + i];
  }
  return t;
}
template <typename X>
inline bool load8_ok(const X* x, int64_t ld) {
  return (uintptr_t)x % kLoadBytes<X> == 0 && ld * sizeof(X) % kLoadBytes<X> == 0;
}

// A workgroup of 256 threads on one row: groups of eight elements, group k of
// thread t at column 8 (256 k + t). The first NV groups of each thread stay in
// registers, so that a row is read once for its maximum and what follows.
template <typename X, int NV>
struct RowOf {
  Eight<X> keep[NV > 0 ? NV : 1];
  const X* row;
  int64_t cols;
  bool vec;

  __device__ inline RowOf(const X* r, int64_t n, bool v) : row(r), cols(n), vec(v) {
#pragma unroll
    for (int k = 0; k < NV; ++k) keep[k] = load8(row, at(k), cols, vec);
  }
  __device__ static inline int64_t at(int64_t k) { return 8 * (256 * k + threadIdx.x); }
  // f(column, eight elements) for every group with columns below `upto`
  template <typename F> __device__ inline void each(int64_t upto, F f) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (at(k) < upto) f(at(k), keep[k]);
    for (int64_t k = NV; at(k) < upto; ++k) f(at(k), load8(row, at(k), cols, vec));
  }
};
// Eight factors of the columns from c on (0 past `cols`).
__device__ inline void factors8(const float* cs, int64_t c, int64_t cols, bool vec, float* f) {
  const Eight<float> t = load8(cs, c, cols, vec);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = t.v[i];
}
// The largest of the workgroup's values (256 threads).
__device__ inline unsigned max_of_256(unsigned top, unsigned* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const unsigned u = __shfl_xor(top, o, 64);
    top = u > top ? u : top;
  }
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) top = red[w] > top ? red[w] : top;
  return top;
}
// Groups a thread keeps for rows of n columns: the row, if 8 groups hold it
// (16384 columns, at most 64 registers).
inline int row_groups(int64_t n) {
  const int64_t g = (n + 2047) / 2048;
  return g <= 1 ? 1 : g <= 2 ? 2 : g <= 4 ? 4 : g <= 8 ? 8 : 0;
}

}  // namespace bk
