// product_tile.h -- a workgroup's part of the product d = epilogue(a b^T) on the
// matrix cores: a tile of sums, or a strip for up to 64 rows.
#pragma once

#include "product_epilogue.h"

namespace hf {

typedef __attribute__((address_space(3))) char lds_char;

// A view of an operand from a byte on, as the buffer loads want it: they
// return zeros past the operand's end, so ragged edges need no branch.
__device__ __forceinline__ i32x4 view(const char *p, int64_t left) {
  const uint64_t at = (uint64_t)p;
  // in 32-bit halves, so that it stays in scalar instructions
  const int hi = (int)(left >> 32), lo = (int)(uint32_t)left;
  i32x4 r;
  r[0] = (int)(uint32_t)at;
  r[1] = (int)(uint32_t)(at >> 32) & 0xffff;
  r[2] = hi < 0 ? 0 : (hi > 0 || lo < 0) ? 0x7fffffff : lo;
  r[3] = 0x00020000;
  return r;
}

// 16 bytes a lane from `r` at byte v + at (past its end: zeros) into LDS, lane
// l at lds + 16 l.  The load has no register result; it is counted by vmcnt alone,
// and whoever reads the bytes waits for the count first and then meets the
// other waves at a barrier.  It is written as assembly because the compiler
// makes every LDS read after the builtin wait for all loads in flight.  m0,
// which the compiler gives to nothing (no LDS access of this target needs it),
// holds the LDS address.
__device__ __forceinline__ void load_to_lds(uint32_t lds, i32x4 r, uint32_t v, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(v), "s"(r), "s"(at)
               : "memory");
}

// The same with 4 bytes a lane.
__device__ __forceinline__ void load_to_lds4(uint32_t lds, i32x4 r, uint32_t v) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(v), "s"(r)
               : "memory");
}
__device__ __forceinline__ float lds_float(uint32_t at) {
  return *(const __attribute__((address_space(3))) float *)(uintptr_t)at;
}

// All loads but the newest N have arrived, and this wave's LDS reads (but the
// newest READS of them).
template <int N, int READS = 0>
__device__ __forceinline__ void arrived() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(%1)" : : "n"(N), "n"(READS) : "memory");
}

// A barrier that nothing is moved across; it waits for no memory by itself.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// One half (R rows of the operand's tile, 128 bytes of the contraction) of a
// stage in LDS, and how it gets there.
//
// LDS has 64 banks of 4 bytes, and 16 lanes of a 16-byte read (32 of an 8-byte
// one) go at once.
//
// By row (the contraction lies along the operand's rows): LDS row r holds the
// 8 16-byte chunks of tile row r, chunk c at slot c ^ (r / 2 % 8).  Two rows
// fill the banks, and the lanes of one turn (rows 0-3 and 12-15 of one chunk,
// 4-11 of the next, or the others) meet 8 different slots in each of the two.
// By column (the contraction runs over the operand's rows; 16-bit types):
// LDS row k holds R columns of contraction step k in units of 16 columns (32
// bytes), unit u at u ^ f(k).  The lanes of one turn read steps k .. k + 3 and
// k + 8 .. k + 11 of one unit, and f tells those apart: 3 bits of k where a
// row fills the banks, 2 where two rows do.  ds_read_b64_tr_b16 turns the
// unit.
//
// The loads write LDS directly, 1 KiB a wave: lane l of a wave fills bytes
// 16 l .. of its kilobyte, so the swizzle is in which global bytes it asks
// for.
template <int R, bool COL, int WAVES>
struct Half {
  static constexpr int kBytes = R * 128;
  static constexpr int kLoads = kBytes / (WAVES * 1024);  // 16-byte loads a thread

  static __device__ __forceinline__ int f(int k) {
    return R == 128 ? (k & 3) | ((k >> 3) & 1) << 2 : ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
  }

  // The global offsets of this thread's loads, from the tile's first row (by
  // row) or first column (by column) at the stage's first contraction byte.
  static __device__ __forceinline__ void offsets(int64_t ld, uint32_t (&v)[kLoads]) {
    const int w = threadIdx.x / 64, l = threadIdx.x % 64;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int piece = w + WAVES * i;
      if (!COL) {
        const int row = piece * 8 + l / 8;
        v[i] = (uint32_t)(row * ld) + (uint32_t)(chunk() * 16);
      } else {
        constexpr int per = R * 2 / 16;  // lanes a step
        const int k = piece * (64 / per) + l / per, slot = l % per;
        v[i] = (uint32_t)(k * ld) + (uint32_t)((((slot >> 1) ^ f(k)) * 32) + (slot & 1) * 16);
      }
    }
  }
  // by row: the chunk that this thread loads, the same in all its pieces (as
  // WAVES is even), and whether it lies past `left` contraction bytes
  static __device__ __forceinline__ int chunk() {
    const int l = threadIdx.x % 64, w = threadIdx.x / 64;
    return (l & 7) ^ ((w & 1) * 4 + (l >> 4));
  }
  static __device__ __forceinline__ uint32_t past(int left) { return !COL && chunk() * 16 >= left ? 0x80000000u : 0u; }
  // into LDS from `lds` on (this wave's first kilobyte)
  static __device__ __forceinline__ void load(uint32_t lds, i32x4 r, const uint32_t (&v)[kLoads], uint32_t at,
                                              uint32_t past) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_to_lds(lds + i * (WAVES * 1024), r, COL ? v[i] : v[i] | past, at);
  }

  // This lane's LDS addresses for the fragments of T tiles of 16 rows
  // (columns) from row `base` of the half on: by row one for each half of the
  // contraction bytes, by column one for each tile.  Everything else is a
  // constant.
  template <int T>
  static constexpr int kAddr = COL ? T : 2;
  template <int T>
  static __device__ __forceinline__ void addresses(uint32_t lds, int base, uint32_t (&p)[kAddr<T>]) {
    const int l = threadIdx.x % 64, g = l >> 4, i = l & 15;
#pragma unroll
    for (int t = 0; t < kAddr<T>; ++t) {
      const int k = g * 8 + (i >> 2);
      p[t] = lds + (COL ? k * (R * 2) + (((base / 16 + t) ^ f(k)) * 32) + (i & 3) * 8
                        : (base + i) * 128 + (((4 * t + g) ^ (i >> 1)) * 16));
    }
  }
  // The fragment of tile t, rows (columns) base + 16 t + l % 16: piece h holds
  // this lane's 16 of the 64 bytes h of the contraction's 128.
  template <int T>
  static __device__ __forceinline__ void read(const uint32_t (&p)[kAddr<T>], uint32_t at, int t, i32x4 (&v)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!COL) {
        v[h] = *(const __attribute__((address_space(3))) i32x4 *)(uintptr_t)(p[h] + at + t * 2048);
      } else {
        typedef __attribute__((address_space(3))) i16x4 tr;
        const uint32_t q = p[t % kAddr<T>] + at + h * (R * 64);
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr *)(uintptr_t)q);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr *)(uintptr_t)(q + R * 8));
        v[h] = __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  }
};

// Tile number `id`: columns of 4 tile rows.
__device__ __forceinline__ void tile_at(int id, int tiles_m, int tiles_n, int &tm, int &tn) {
  constexpr int G = 4;
  const int group = id / (G * tiles_n), first = group * G, size = tiles_m - first < G ? tiles_m - first : G;
  tm = first + (id - group * G * tiles_n) % size;
  tn = (id - group * G * tiles_n) / size;
}

// A workgroup computes 2 HM x 2 HN sums, 128 contraction bytes a stage, two
// stages in LDS: 256 x 256 with 8 waves, one workgroup a compute unit, or
// 128 x 128 with 4 waves, two of them.  A wave has HM/2 x 32 sums in each
// quarter of the tile; gated, the second half of the columns is the up half
// of the first, so a lane holds gate and up of the same element.
// Measured: 8192 x 8192 x 8192 bf16 730 us, 1.51 PFLOP/s; 4096 x 4096 x 16384
// e4m3 187 us, 2.9 PFLOP/s; 8191 x 22528 x 4096 gated bf16 with both halves
// kept 1092 us.  The matrix cores are busy 74 - 81% of the cycles and the
// power limit holds the clock at 1.6 - 1.9 GHz; a tile's end (sums out, the
// next tile's first loads in) is 10 us.  With block scales 4096 x 4096 x 16384
// e4m3 takes 234 us, 2.35 PFLOP/s: a matrix instruction comes with 5.8 others of
// the vector unit, 4 of them the additions of its block's sums and the rest
// scales and addresses, and the matrix cores are busy 63% of the cycles at 1.92
// GHz.
template <int HM, int HN>
struct Shape {
  static constexpr int kWaves = 2 * (HN / 32), kThreads = kWaves * 64;
  static constexpr int kStage = 256 * (HM + HN);
  // the sums on their way out: rows of 2 HN with a pad of 16 bytes
  static constexpr int kPitch = 2 * HN + 4, kOut = HM * kPitch * 4;
  // block scales: of four stages in turn, 4 bytes a thread, behind the stages
  static constexpr int kScale = kThreads * 4;
  static constexpr int lds(bool block) {
    return block ? 2 * kStage + 4 * kScale : 2 * kStage > kOut ? 2 * kStage : kOut;
  }
};

// EXPERT: `a` is one expert's part of a product by experts, whose tiles are
// numbered from 0 and are a workgroup's each (kWhole), or that of every one of
// the splits (kSplit: piece a.piece, whose sums go to a.partial on).  They are
// kernels of their own: with the choice made in one, small products of the
// whole contraction take 1 us more.
enum { kDense = 0, kWhole = 1, kSplit = 2 };
template <class Step, bool ACOL, bool BCOL, int HM, int HN, int EXPERT = kDense>
__device__ __forceinline__ void product_tile(const ProductArgs &a, int block, char *lds) {
  typedef Shape<HM, HN> S;
  constexpr int WN = HN / 32, WAVES = S::kWaves, THREADS = S::kThreads, kStage = S::kStage, kPitch = S::kPitch;
  typedef Half<HM, ACOL, WAVES> HA;
  typedef Half<HN, BCOL, WAVES> HB;
  constexpr int TM = HM / 32, TN = 2;  // 16 x 16 tiles of a wave in a quarter
  static_assert(kStage == 2 * HA::kBytes + 2 * HB::kBytes, "two halves of both operands");

  const bool gated = a.e.gated;
  const int tile_n = gated ? HN : 2 * HN;
  const int tiles_m = (a.m + 2 * HM - 1) / (2 * HM), tiles_n = (a.n + tile_n - 1) / tile_n;
  // The first tiles_full tiles are a workgroup's each; the rest, which would
  // leave most of the chip idle for a whole tile's time, are shared by
  // `splits` workgroups each, one part of the contraction a workgroup.
  const int tiles = tiles_m * tiles_n, rest = EXPERT ? 0 : tiles - a.tiles_full;
  const bool part = !EXPERT && block >= a.tiles_full;
  // Consecutive workgroups go to different XCDs; each XCD takes a contiguous
  // run of tiles, in columns of 4 tile rows, so that the tiles it works on at
  // a time share rows and columns in its L2.
  int id = part ? block - a.tiles_full : block;
  if (!EXPERT) {
    const int count = part ? rest * a.splits : a.tiles_full;
    const int xcd = id % 8, q = count / 8, r = count % 8;
    id = xcd * q + (xcd < r ? xcd : r) + id / 8;
  }
  const int piece = EXPERT == kSplit ? a.piece : part ? id / rest : 0, local = part ? id % rest : 0;
  int tm, tn;
  tile_at(part ? a.tiles_full + local : id, tiles_m, tiles_n, tm, tn);
  const int m0 = tm * 2 * HM, n0 = tn * tile_n;

  const int w = threadIdx.x / 64, wm = w / WN, wn = w % WN;
  constexpr int kStep = 128 / Step::kBytes;  // elements of the contraction a stage
  const int all = (a.k + kStep - 1) / kStep;
  const int k0 = piece * a.k_tiles_per_split;
  const int kn = !(EXPERT == kSplit || part) || all - k0 < a.k_tiles_per_split ? all - k0 : a.k_tiles_per_split;

  // the operands' first bytes for this tile and what is left of them
  const int64_t a0 = ACOL ? (int64_t)m0 * Step::kBytes + (int64_t)k0 * kStep * a.lda
                          : (int64_t)m0 * a.lda + (int64_t)k0 * 128;
  const int64_t a_half = ACOL ? (int64_t)HM * Step::kBytes : (int64_t)HM * a.lda;
  const int64_t b0 = BCOL ? (int64_t)n0 * Step::kBytes + (int64_t)k0 * kStep * a.ldb
                          : (int64_t)n0 * a.ldb + (int64_t)k0 * 128;
  const int64_t b_half = gated ? a.b_half : BCOL ? (int64_t)HN * Step::kBytes : (int64_t)HN * a.ldb;
  const int64_t a_step = ACOL ? kStep * a.lda : 128, b_step = BCOL ? kStep * a.ldb : 128;
  uint32_t va[HA::kLoads], vb[HB::kLoads];
  HA::offsets(a.lda, va);
  HB::offsets(a.ldb, vb);

  typename Step::Acc acc[2][2][TM][TN];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int x = 0; x < TM; ++x)
#pragma unroll
        for (int y = 0; y < TN; ++y) acc[i][j][x][y] = typename Step::Acc{0, 0, 0, 0};

  // half h of a's (b's) stage kt into its place; past the last stage zeros are
  // written, so that the counts below always hold.  By row the two halves'
  // views stay and the offset moves; by column the halves share a view, whose
  // base moves, as the whole operand may be beyond an offset's 32 bits.
  const uint32_t base = (uint32_t)(uintptr_t)(lds_char *)lds;
  const uint32_t mine = base + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x / 64) * 1024;
  const int k_end = (k0 + kn) * kStep < a.k ? kn * kStep : a.k - k0 * kStep;  // elements of this split
  const i32x4 ra[2] = {view((const char *)a.a + a0, a.a_bytes - a0),
                       view((const char *)a.a + a0 + a_half, a.a_bytes - a0 - a_half)};
  const i32x4 rb[2] = {view((const char *)a.b + b0, a.b_bytes - b0),
                       view((const char *)a.b + b0 + b_half, a.b_bytes - b0 - b_half)};
  auto fetch_a = [&](int kt, int odd, int h) {
    const uint32_t to = mine + odd * kStage + h * HA::kBytes;
    if (!ACOL) {
      HA::load(to, ra[h], va, kt * 128, HA::past((k_end - kt * kStep) * Step::kBytes));
    } else {
      const int64_t at = a0 + kt * a_step;
      HA::load(to, view((const char *)a.a + at, kt < kn ? a.a_bytes - at : 0), va, h * HM * 2, 0);
    }
  };
  auto fetch_b = [&](int kt, int odd, int h) {
    const uint32_t to = mine + odd * kStage + 2 * HA::kBytes + h * HB::kBytes;
    if (!BCOL) {
      HB::load(to, rb[h], vb, kt * 128, HB::past((k_end - kt * kStep) * Step::kBytes));
    } else {
      const int64_t at = b0 + kt * b_step;
      HB::load(to, view((const char *)a.b + at, kt < kn ? a.b_bytes - at : 0), vb, h * HN * 2, 0);
    }
  };
  // Block scales: the lower half of the waves asks for the rows' of a stage, a
  // row a lane, the next quarters for the one of b's half 0 and of half 1.
  // Past the last stage they are zeros, as the operands are.
  constexpr bool BLOCK = Step::kBlock;
  const uint32_t scales = base + 2 * kStage;
  // Where a wave's lie is chosen here: the loop has no branch, or the compiler
  // moves products past the barriers.
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const char *scale_from = nullptr;
  int64_t scale_step = 0;
  int scale_bytes = 0;
  const uint32_t scale_lane = wave < WAVES / 2 ? threadIdx.x * 4 : 0;
  if constexpr (BLOCK) {
    if (wave < WAVES / 2) {
      scale_from = (const char *)(a.a_scale + (int64_t)k0 * a.lda_scale + m0);
      scale_step = a.lda_scale * 4;
      scale_bytes = min(a.m - m0, 2 * HM) * 4;  // the tile's rows: all those left may pass 2^31 bytes
    } else {
      const int half = (wave - WAVES / 2) / (WAVES / 4), n = gated ? n0 : n0 + half * HN;
      scale_from = (const char *)(a.b_scale + (min(n, a.n - 1) / 128 + (gated ? half * a.b_scale_half : 0)) * a.ldb_scale + k0);
      scale_step = scale_bytes = 4;
    }
  }
  auto fetch_scales = [&](int kt) {
    if constexpr (BLOCK)
      load_to_lds4(scales + (kt & 3) * S::kScale + wave * 256, view(scale_from + kt * scale_step, kt < kn ? scale_bytes : 0),
                   scale_lane);
  };
  // A quarter's scales are read from LDS a quarter ahead, and made into factors
  // between that quarter's products.  One address serves all: b's scale lies
  // there once for every lane.
  typename ScaleOf<Step>::Type scale[TM], next[TM];
  float rows_scale[BLOCK ? TM : 1], b_scale = 0.f;
  const uint32_t scale_at = scales + (wm * (HM / 2) + (threadIdx.x & 15)) * 4;
  auto ask_scales = [&](int kt, int h, int j) {
    if constexpr (BLOCK) {
      const uint32_t at = scale_at + (kt & 3) * S::kScale;
      b_scale = lds_float(at + (WAVES / 2 + j * (WAVES / 4)) * 256);
#pragma unroll
      for (int x = 0; x < TM; ++x) rows_scale[x] = lds_float(at + (h * HM + x * 16) * 4);
    }
  };
  // the second stage is beyond the 16 bits of a read's constant offset: its
  // addresses are registers of their own (which the compiler must not know,
  // or it makes one for every constant)
  constexpr int NA = HA::template kAddr<TM>, NB = HB::template kAddr<TN>;
  uint32_t pa[2][NA], pb[2][NB];
#pragma unroll
  for (int odd = 0; odd < 2; ++odd) {
    HA::template addresses<TM>(base + odd * kStage, wm * (HM / 2), pa[odd]);
    HB::template addresses<TN>(base + odd * kStage + 2 * HA::kBytes, wn * 32, pb[odd]);
#pragma unroll
    for (int i = 0; i < NA; ++i) asm volatile("" : "+v"(pa[odd][i]));
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(pb[odd][i]));
  }
  i32x4 fa[TM][2], fb[2][TN][2];
  auto read_a = [&](int odd, int h) {
#pragma unroll
    for (int x = 0; x < TM; ++x) HA::template read<TM>(pa[odd], h * HA::kBytes, x, fa[x]);
  };
  auto read_b = [&](int odd, int h) {
#pragma unroll
    for (int y = 0; y < TN; ++y) HB::template read<TN>(pb[odd], h * HB::kBytes, y, fb[h][y]);
  };
  // Block scales: the sum of block n of a quarter is added after kLate more are
  // asked for, by when it is there; the last ones' while the other wave has its
  // turn.  (A matrix instruction takes 32 cycles, 34 with two vector
  // instructions behind it and 40 with four, so a quarter's additions are
  // divided between the two sections.)
  constexpr int kBlocks = TM * TN, kLate = 3;
  f32x4 late[BLOCK ? kLate : 1];
  auto add_block = [&](int i, int j, int n) {
    if constexpr (BLOCK) {
      const int x = n % TM, y = n / TM;
      acc[i][j][x][y] = Step::add(acc[i][j][x][y], late[n % kLate], scale[x]);
    }
  };
  auto settle = [&](int i, int j) {
#pragma unroll
    for (int n = kBlocks - kLate; n < kBlocks; ++n) add_block(i, j, n);
  };
  auto multiply = [&](int i, int j) {
    if constexpr (BLOCK) {
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) {
        if (n >= kLate) add_block(i, j, n - kLate);
        if (n > 0 && n < kLate) {
#pragma unroll
          for (int x = (n - 1) * TM / (kLate - 1); x < n * TM / (kLate - 1); ++x) next[x] = Step::scale(rows_scale[x], b_scale);
        }
        __builtin_amdgcn_sched_barrier(0);
        late[n % kLate] = Step::block(fa[n % TM], fb[j][n / TM], scale[n % TM]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int k = 0; k < Step::kSteps; ++k)
#pragma unroll
        for (int y = 0; y < TN; ++y)
#pragma unroll
          for (int x = 0; x < TM; ++x) acc[i][j][x][y] = Step::step(fa[x], fb[j][y], acc[i][j][x][y], k);
      __builtin_amdgcn_s_setprio(0);
    }
  };

  // The stages run through a pipeline of quarters.  The two waves of a SIMD
  // (w and w + 4) take turns: in one section a wave reads the next quarter's
  // fragments from LDS and asks for a half of a later stage, in the next it
  // multiplies while the other wave reads; a barrier ends every section, and
  // waves 4 .. 7 start one section late.  (With 4 waves the other wave of a
  // SIMD is another workgroup's, and the two fall into step by themselves.)  A
  // stage's quarters go
  //   (a0, b0) (a0, b1) (a1, b1) (a1, b0)   in even stages,
  //   (a0, b1) (a0, b0) (a1, b0) (a1, b1)   in odd ones,
  // so each quarter but the last brings in one new half, and the last, which
  // brings none, reads the b half that the next stage begins with.  A half's
  // place is free once both waves have read it (their reads have arrived
  // before the barrier), so the same half of two stages on is asked for one
  // quarter later and has six quarters to arrive: kAhead loads are younger
  // than the ones that the next quarter reads.
  // (With block scales every stage asks for one more, at its first quarter: six
  // quarters hold one or two of those.)
  constexpr int kAhead = 3 * (HA::kLoads + HB::kLoads) + (BLOCK ? 1 : 0);
  // The next quarter's scales, read last, need not be there yet: the compiler
  // reads at most two of them at a time.
  constexpr int kScaleReads = BLOCK ? (TM + 2) / 2 : 0;
  // was_i, was_j: the quarter before; kt, next_i, next_j: the one after
  auto quarter = [&](auto read, auto fetch, int was_i, int was_j, int i, int j, int kt, int next_i, int next_j) {
    // with block scales the wave that reads goes first: both have vector work
    if (BLOCK) __builtin_amdgcn_s_setprio(1);
    read();
    if constexpr (BLOCK) {
      __builtin_amdgcn_sched_barrier(0);
      settle(was_i, was_j);
#pragma unroll
      for (int x = 0; x < TM; ++x) scale[x] = next[x];
      ask_scales(kt, next_i, next_j);
    }
    fetch();
    if (BLOCK) __builtin_amdgcn_s_setprio(0);
    arrived<kAhead, kScaleReads>();
    meet();
    multiply(i, j);
    meet();
  };
  if (kn > 0) {
    fetch_scales(0);
    fetch_b(0, 0, 0), fetch_a(0, 0, 0), fetch_b(0, 0, 1), fetch_a(0, 0, 1);
    fetch_scales(1);
    fetch_b(1, 1, 1), fetch_a(1, 1, 0), fetch_b(1, 1, 0), fetch_a(1, 1, 1);
    arrived<kAhead>();
    meet();
    read_b(0, 0);
    ask_scales(0, 0, 0);
    if constexpr (BLOCK) {  // no quarter was before the first
#pragma unroll
      for (int n = 0; n < kLate; ++n) late[n] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < TM; ++x) {
        scale[x] = Step::scale(0.f, 0.f);
        next[x] = Step::scale(rows_scale[x], b_scale);
      }
    }
    arrived<kAhead>();
    meet();
    if (WAVES == 8 && wm) meet();
    for (int kt = 0; kt < kn; kt += 2) {
      quarter([&] { read_a(0, 0); }, [&] { fetch_scales(kt + 2), fetch_b(kt + 2, 0, 0); }, 1, 1, 0, 0, kt, 0, 1);
      quarter([&] { read_b(0, 1); }, [&] { fetch_a(kt + 2, 0, 0); }, 0, 0, 0, 1, kt, 1, 1);
      quarter([&] { read_a(0, 1); }, [&] { fetch_b(kt + 2, 0, 1); }, 0, 1, 1, 1, kt, 1, 0);
      quarter([&] { read_b(1, 1); }, [&] { fetch_a(kt + 2, 0, 1); }, 1, 1, 1, 0, kt + 1, 0, 1);
      // an odd number of stages: the last is all zeros and adds nothing
      quarter([&] { read_a(1, 0); }, [&] { fetch_scales(kt + 3), fetch_b(kt + 3, 1, 1); }, 1, 0, 0, 1, kt + 1, 0, 0);
      quarter([&] { read_b(1, 0); }, [&] { fetch_a(kt + 3, 1, 0); }, 0, 1, 0, 0, kt + 1, 1, 0);
      quarter([&] { read_a(1, 1); }, [&] { fetch_b(kt + 3, 1, 0); }, 0, 0, 1, 0, kt + 1, 1, 1);
      quarter([&] { read_b(0, 0); }, [&] { fetch_a(kt + 3, 1, 1); }, 1, 0, 1, 1, kt + 2, 0, 0);
    }
    settle(1, 1);
    if (WAVES == 8 && !wm) meet();
    // nothing may still be on its way to LDS when its bytes are used again
    arrived<0>();
  }

  // Out: the sums of HM rows at a time go through LDS, so that a thread has 8
  // consecutive columns of a row and a row's stores are contiguous.  A lane's
  // four sums are 16 bytes; the pad keeps neighbouring rows in different banks.
  const int l = threadIdx.x % 64;
  const bool shared = EXPERT == kSplit || (part && a.splits > 1);
  float *out = (float *)lds;
  const int shift = __builtin_ctz(tile_n / 8), per = 1 << shift;  // threads a row
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    __syncthreads();
#pragma unroll
    for (int x = 0; x < TM; ++x)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int y = 0; y < TN; ++y)
          *(f32x4 *)(out + (wm * (HM / 2) + x * 16 + (l & 15)) * kPitch + j * HN + wn * 32 + y * 16 + (l >> 4) * 4) =
              shared ? Step::bits(acc[i][j][x][y]) : Step::sums(acc[i][j][x][y]);
    __syncthreads();
#pragma unroll 1
    for (int at = threadIdx.x; at < HM * per; at += THREADS) {
      const int r = at >> shift, c = (at & (per - 1)) * 8, m = m0 + i * HM + r, n = n0 + c;
      float v[8], u[8];
      load8<F32>(out + r * kPitch + c, v);
      if (gated) load8<F32>(out + r * kPitch + HN + c, u);
      if (EXPERT == kSplit) {
        if (m < a.m && n < a.n) {
          float *p = a.partial + m * a.ldp + n;
          store8<F32>(p, v);
          if (gated) store8<F32>(p + a.ldp / 2, u);
        }
      } else if (shared) {
        if (i * HM + r < a.part_rows && c < (gated ? a.part_cols / 2 : a.part_cols)) {
          float *p = a.partial + (((int64_t)piece * rest + local) * a.part_rows + i * HM + r) * a.part_cols + c;
          store8<F32>(p, v);
          if (gated) store8<F32>(p + a.part_cols / 2, u);
        }
      } else {
        finish<8>(a.e, m, n, v, u);
      }
    }
  }
}

// The product for up to 64 rows, bound by reading b: a strip of 128 columns
// (gated: 64 and their up half) a workgroup of 8 waves, 16 columns a wave, all
// rows.  Both operands go through LDS in whole 128-byte lines, a once for 128
// columns.  Five stages of 24 KiB, four of them in flight: twice what the
// memory's latency times its rate a compute unit needs.  24 x 22528 x 4096
// gated bf16 takes 37 us (5.0 TB/s), 64 rows 42; with strips of 256 columns,
// which have to share the contraction of such a layer to fill the chip, 41 and
// 47; from registers, as the skinny product does it, 51 and 75.
template <class Step>
struct Strip {
  static constexpr int kStage = 3 * 64 * 128, kStages = 5;
  // block scales: of each stage, every wave its own: 64 rows', then b's
  static constexpr int kScale = Step::kBlock ? 8 * 512 : 0;
  static constexpr int kLds = kStages * (kStage + kScale);
};

// Strip number `strip`, part number `piece` of the contraction, whose sums go to
// a.partial on; `seed` staggers the workgroups.
template <class Step>
__device__ __forceinline__ void strip_tile(const ProductArgs &a, int strip, int piece, uint32_t seed, char *lds) {
  constexpr int HN = 64;
  typedef Half<64, false, 8> HA;
  typedef Half<HN, false, 8> HB;
  constexpr int TM = 4;  // 16 x 16 tiles of a wave
  constexpr int kStage = Strip<Step>::kStage, kStages = Strip<Step>::kStages;
  constexpr int kPitch = 2 * HN + 4;
  static_assert(kStage == HA::kBytes + 2 * HB::kBytes, "both operands");
  static_assert(64 * kPitch * 4 <= kStages * kStage, "the sums go out through the stages");

  const bool gated = a.e.gated;
  const int width = gated ? HN : 2 * HN;
  const int n0 = strip * width;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64;
  constexpr int kStep = 128 / Step::kBytes;
  const int k0 = piece * a.k_tiles_per_split;
  const int all = (a.k + kStep - 1) / kStep;
  const int kn = all - k0 < a.k_tiles_per_split ? all - k0 : a.k_tiles_per_split;
  const int left = (k0 + kn) * kStep < a.k ? kn * 128 : (a.k - k0 * kStep) * Step::kBytes;
  const int64_t a0 = (int64_t)k0 * 128, b0 = (int64_t)n0 * a.ldb + (int64_t)k0 * 128;
  const int64_t b_half = gated ? a.b_half : HN * a.ldb;
  const i32x4 ra = view((const char *)a.a + a0, a.a_bytes - a0);
  const i32x4 rb[2] = {view((const char *)a.b + b0, a.b_bytes - b0),
                       view((const char *)a.b + b0 + b_half, a.b_bytes - b0 - b_half)};
  uint32_t va[HA::kLoads], vb[HB::kLoads];
  HA::offsets(a.lda, va);
  HB::offsets(a.ldb, vb);
  const uint32_t base = (uint32_t)(uintptr_t)(lds_char *)lds;
  // Workgroups begin at stages of their own and go round, so that rows a
  // power of two apart do not keep all of them on the same memory channels.
  const int turn = kn > 0 ? (int)(seed % (uint32_t)kn) : 0;
  constexpr bool BLOCK = Step::kBlock;
  const int half = w / 4, col = (w % 4) * 16;  // this wave's columns
  const float *b_scale = nullptr;
  if (BLOCK) b_scale = a.b_scale + (min(gated ? n0 : n0 + half * HN, a.n - 1) / 128 + (gated ? half * a.b_scale_half : 0)) * a.ldb_scale;
  const uint32_t scales = base + kStages * kStage + w * 512;
  auto fetch_scales = [&](int kt, int t, int stage) {
    if constexpr (BLOCK) {
      const uint32_t to = scales + stage * Strip<Step>::kScale;
      load_to_lds4(to, view((const char *)(a.a_scale + (int64_t)(k0 + t) * a.lda_scale), kt < kn ? a.m * 4 : 0), l * 4);
      load_to_lds4(to + 256, view((const char *)(b_scale + k0 + t), kt < kn ? 4 : 0), l * 4);
    }
  };
  auto fetch = [&](int kt, int stage) {
    int t = kt + turn;
    t = t >= kn ? t - kn : t;
    const uint32_t past = kt < kn ? HA::past(left - t * 128) : 0x80000000u;
    const uint32_t to = base + stage * kStage + w * 1024;
    HA::load(to, ra, va, t * 128, past);
#pragma unroll
    for (int h = 0; h < 2; ++h) HB::load(to + HA::kBytes + h * HB::kBytes, rb[h], vb, t * 128, past);
    fetch_scales(kt, t, stage);
  };
  typename Step::Acc acc[TM];
#pragma unroll
  for (int x = 0; x < TM; ++x) acc[x] = typename Step::Acc{0, 0, 0, 0};
  uint32_t pa[2], pb[2];
  HA::addresses<TM>(base, 0, pa);
  HB::addresses<1>(base + HA::kBytes + half * HB::kBytes, col, pb);
  auto add = [&](int stage) {
    const uint32_t at = stage * kStage;
    i32x4 fb[2];
    HB::read<1>(pb, at, 0, fb);
    const float sb = BLOCK ? lds_float(scales + stage * Strip<Step>::kScale + 256) : 0.f;
#pragma unroll
    for (int x = 0; x < TM; ++x) {
      if (x * 16 >= a.m) break;
      i32x4 fa[2];
      HA::read<TM>(pa, at, x, fa);
      if constexpr (BLOCK)
        acc[x] = mma_block<Step>(fa, fb, lds_float(scales + stage * Strip<Step>::kScale + (x * 16 + (l & 15)) * 4), sb, acc[x]);
      else
        acc[x] = mma<Step>(fa, fb, acc[x]);
    }
  };
  // A stage's loads have arrived when only those of the stages after it are
  // left; after the barrier every wave's have, and every wave is done with the
  // stage before it, whose place the newest stage then takes.
  constexpr int kLoads = HA::kLoads + 2 * HB::kLoads + (BLOCK ? 2 : 0);
  if (kn > 0) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i, i);
    for (int kt = 0; kt < kn; kt += kStages) {
#pragma unroll
      for (int i = 0; i < kStages; ++i) {
        arrived<kLoads *(kStages - 2)>();
        meet();
        fetch(kt + i + kStages - 1, (i + kStages - 1) % kStages);
        if (kt + i < kn) add(i);
      }
    }
    arrived<0>();
  }
  float *out = (float *)lds;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < TM; ++x)
    *(f32x4 *)(out + (x * 16 + (l & 15)) * kPitch + half * HN + col + (l >> 4) * 4) =
        a.splits > 1 ? Step::bits(acc[x]) : Step::sums(acc[x]);
  __syncthreads();
  const int shift = __builtin_ctz(width / 8), per = 1 << shift;
#pragma unroll 1
  for (int at = threadIdx.x; at < a.m * per; at += 512) {
    const int m = at >> shift, c = (at & (per - 1)) * 8, n = n0 + c;
    if (n >= a.n) continue;
    float v[8], u[8];
    load8<F32>(out + m * kPitch + c, v);
    if (gated) load8<F32>(out + m * kPitch + HN + c, u);
    if (a.splits > 1) {
      float *p = a.partial + m * a.ldp + n;
      store8<F32>(p, v);
      if (gated) store8<F32>(p + a.ldp / 2, u);
    } else {
      finish<8>(a.e, m, n, v, u);
    }
  }
}

// ---- products by expert ------------------------------------------------
// The rows of expert e are offsets[e] .. offsets[e + 1] - 1.  Tiles of `size`
// rows, `per` of them side by side: which expert's tile this workgroup has,
// and its number there; false where there are no more tiles.  The offsets are
// the caller's data: whatever they hold, rows stay within 0 .. m - 1.
//
// Every wave counts the tiles for itself, an expert a lane, and adds them up:
// about 1 us, against 10 us and more that a tile takes, and no launch or wait
// of a kernel that would write a list.  As in product_tile, each XCD takes a
// contiguous run of tiles.
//
// CUT: the last tiles, which would leave more than half of the 256 compute
// units without one, are cut into an upper and a lower half, a workgroup's
// each.
struct ExpertTile {
  int expert, row, rows, local;
  int half;  // 0 or 1: that half of the tile's rows, -1: all
};
__device__ __forceinline__ int xcd_run(int block, int count) {
  const int xcd = block % 8, q = count / 8, r = count % 8;
  return xcd * q + min(xcd, r) + block / 8;
}
template <bool CUT>
__device__ __forceinline__ bool expert_tile(const int32_t *offsets, int experts, int m, int size, int per, int block,
                                            ExpertTile &t) {
  const int l = threadIdx.x % 64;
  constexpr int kMost = 1 << 24;  // tiles of an expert: a launch holds no more
  auto tiles = [&](int e, int &lo, int &hi) {
    lo = hi = 0;
    if (e < experts) {
      lo = min(max(offsets[e], 0), m);
      hi = min(max(offsets[e + 1], lo), m);
    }
    return (int)min((int64_t)((hi - lo + size - 1) / size) * per, (int64_t)kMost);
  };
  auto scan = [&](int n) {  // the sum of the lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(n, d);
      n += l >= d ? o : 0;
    }
    return n;
  };
  // the first 64 experts' counts stay for the search
  int lo, hi;
  int n = tiles(l, lo, hi), sum = scan(n);
  int64_t all = __builtin_amdgcn_readlane(sum, 63);
  for (int first = 64; first < experts; first += 64) {
    int a, b;
    all += __builtin_amdgcn_readlane(scan(tiles(first + l, a, b)), 63);
  }
  const int total = (int)min(all, (int64_t)0x7fffffff);
  const int cut = CUT && total % 256 <= 128 ? total % 256 : 0, whole = total - cut;
  if (block >= whole + 2 * cut) return false;
  int id;
  t.half = -1;
  if (block < whole) {
    id = xcd_run(block, whole);
  } else {
    id = xcd_run(block - whole, 2 * cut);
    t.half = id % 2;
    id = whole + id / 2;
  }
  for (int first = 0; first < experts; first += 64) {
    if (first > 0) n = tiles(first + l, lo, hi), sum = scan(n);
    const uint64_t hit = __ballot(id < sum);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      t.expert = first + at;
      t.row = __builtin_amdgcn_readlane(lo, at);
      t.rows = __builtin_amdgcn_readlane(hi, at) - t.row;
      t.local = __builtin_amdgcn_readfirstlane(id) - __builtin_amdgcn_readlane(sum - n, at);
      return true;
    }
    id -= __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

// One expert's part of a product whose rows are sorted: rows `row` .. of a and
// d, the expert's weight.
__device__ __forceinline__ ProductArgs part_of(const ProductArgs &a, int expert, int row, int rows) {
  ProductArgs p = a;
  const int64_t out = a.e.out_dtype == HF_F32 ? 4 : 2, wide = a.e.gated ? 2 * (int64_t)a.n : a.n;
  p.a = (const char *)a.a + row * a.lda;
  p.a_bytes = a.a_bytes - row * a.lda;
  p.b = (const char *)a.b + expert * a.b_expert;
  p.m = p.e.m = rows;
  p.partial = a.partial + ((int64_t)a.piece * a.m + row) * a.ldp;
  p.e.d = (char *)a.e.d + row * a.e.ldd * out;
  if (a.e.z) p.e.z = (char *)a.e.z + row * a.e.ldz * out;
  if (a.e.a_scale) p.e.a_scale = a.e.a_scale + row, p.e.b_scale = a.e.b_scale + expert * wide;
  if (a.a_scale) {
    p.a_scale = a.a_scale + row;
    p.b_scale = a.b_scale + expert * (int64_t)(a.e.gated ? 2 : 1) * a.b_scale_half * a.ldb_scale;
  }
  return p;
}

// A tile of 256 x 256 of an expert, or, where it has no more than 128 rows or
// is cut, a half or two of them of 128 x 256, which take about 0.6 of its time.
template <class Step, bool ACOL, bool BCOL>
__device__ __forceinline__ void large_tile(const ProductArgs &a, const ExpertTile &t, int tiles_n, char *lds) {
  int tm, tn;
  tile_at(t.local, (t.rows + 255) / 256, tiles_n, tm, tn);
  const int from = tm * 256 + (t.half > 0 ? 128 : 0), left = t.rows - from;
  if (left <= 0) return;
  if (t.half >= 0 || left <= 128)
    product_tile<Step, ACOL, BCOL, 64, 128, kWhole>(part_of(a, t.expert, t.row + from, min(left, 128)), tn, lds);
  else
    product_tile<Step, ACOL, BCOL, 128, 128, kWhole>(part_of(a, t.expert, t.row, t.rows), t.local, lds);
}

}  // namespace hf
