// product.hip -- the tiled product d = epilogue(a b^T) on the matrix cores.
#include "product_epilogue.h"

namespace hf {
namespace {

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

// All loads but the newest N have arrived, and this wave's LDS reads.
template <int N>
__device__ __forceinline__ void arrived() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
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
// next tile's first loads in) is 10 us.
template <int HM, int HN>
struct Shape {
  static constexpr int kWaves = 2 * (HN / 32), kThreads = kWaves * 64;
  static constexpr int kStage = 256 * (HM + HN);
  // the sums on their way out: rows of 2 HN with a pad of 16 bytes
  static constexpr int kPitch = 2 * HN + 4, kOut = HM * kPitch * 4;
  static constexpr int kLds = 2 * kStage > kOut ? 2 * kStage : kOut;
};

template <class Step, bool ACOL, bool BCOL, int HM, int HN>
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
  const int tiles = tiles_m * tiles_n, rest = tiles - a.tiles_full;
  const bool part = block >= a.tiles_full;
  // Consecutive workgroups go to different XCDs; each XCD takes a contiguous
  // run of tiles, in columns of 4 tile rows, so that the tiles it works on at
  // a time share rows and columns in its L2.
  int id = part ? block - a.tiles_full : block;
  {
    const int count = part ? rest * a.splits : a.tiles_full;
    const int xcd = id % 8, q = count / 8, r = count % 8;
    id = xcd * q + (xcd < r ? xcd : r) + id / 8;
  }
  const int piece = part ? id / rest : 0, local = part ? id % rest : 0;
  int tm, tn;
  tile_at(part ? a.tiles_full + local : id, tiles_m, tiles_n, tm, tn);
  const int m0 = tm * 2 * HM, n0 = tn * tile_n;

  const int w = threadIdx.x / 64, wm = w / WN, wn = w % WN;
  constexpr int kStep = 128 / Step::kBytes;  // elements of the contraction a stage
  const int all = (a.k + kStep - 1) / kStep;
  const int k0 = piece * a.k_tiles_per_split;
  const int kn = !part || all - k0 < a.k_tiles_per_split ? all - k0 : a.k_tiles_per_split;

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
  auto multiply = [&](int i, int j) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int k = 0; k < Step::kSteps; ++k)
#pragma unroll
      for (int y = 0; y < TN; ++y)
#pragma unroll
        for (int x = 0; x < TM; ++x) acc[i][j][x][y] = Step::step(fa[x], fb[j][y], acc[i][j][x][y], k);
    __builtin_amdgcn_s_setprio(0);
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
  constexpr int kAhead = 3 * (HA::kLoads + HB::kLoads);
  auto quarter = [&](auto read, auto fetch, int i, int j) {
    read();
    fetch();
    arrived<kAhead>();
    meet();
    multiply(i, j);
    meet();
  };
  if (kn > 0) {
    fetch_b(0, 0, 0), fetch_a(0, 0, 0), fetch_b(0, 0, 1), fetch_a(0, 0, 1);
    fetch_b(1, 1, 1), fetch_a(1, 1, 0), fetch_b(1, 1, 0), fetch_a(1, 1, 1);
    arrived<kAhead>();
    meet();
    read_b(0, 0);
    arrived<kAhead>();
    meet();
    if (WAVES == 8 && wm) meet();
    for (int kt = 0; kt < kn; kt += 2) {
      quarter([&] { read_a(0, 0); }, [&] { fetch_b(kt + 2, 0, 0); }, 0, 0);
      quarter([&] { read_b(0, 1); }, [&] { fetch_a(kt + 2, 0, 0); }, 0, 1);
      quarter([&] { read_a(0, 1); }, [&] { fetch_b(kt + 2, 0, 1); }, 1, 1);
      quarter([&] { read_b(1, 1); }, [&] { fetch_a(kt + 2, 0, 1); }, 1, 0);
      // an odd number of stages: the last is all zeros and adds nothing
      quarter([&] { read_a(1, 0); }, [&] { fetch_b(kt + 3, 1, 1); }, 0, 1);
      quarter([&] { read_b(1, 0); }, [&] { fetch_a(kt + 3, 1, 0); }, 0, 0);
      quarter([&] { read_a(1, 1); }, [&] { fetch_b(kt + 3, 1, 0); }, 1, 0);
      quarter([&] { read_b(0, 0); }, [&] { fetch_a(kt + 3, 1, 1); }, 1, 1);
    }
    if (WAVES == 8 && !wm) meet();
    // nothing may still be on its way to LDS when its bytes are used again
    arrived<0>();
  }

  // Out: the sums of HM rows at a time go through LDS, so that a thread has 8
  // consecutive columns of a row and a row's stores are contiguous.  A lane's
  // four sums are 16 bytes; the pad keeps neighbouring rows in different banks.
  const int l = threadIdx.x % 64;
  const bool shared = part && a.splits > 1;
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
      if (shared) {
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

template <class Step, int HM, int HN>
__global__ __launch_bounds__(HM == 128 ? 512 : 256, 2) void product_kernel(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<HM, HN>::kLds];
  product_tile<Step, false, false, HM, HN>(a, blockIdx.x, lds);
}

// The two products of a gradient, da = dz b and db = dz^T a, in one launch:
// neither needs the other, small ones fill the chip together and large ones
// share their last round.
template <class Step, int HM, int HN>
__global__ __launch_bounds__(HM == 128 ? 512 : 256, 2) void gradient_kernel(ProductArgs da, ProductArgs db, int first) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<HM, HN>::kLds];
  if ((int)blockIdx.x < first)
    product_tile<Step, false, true, HM, HN>(da, blockIdx.x, lds);
  else
    product_tile<Step, true, true, HM, HN>(db, blockIdx.x - first, lds);
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
__global__ __launch_bounds__(512, 2) void strip_kernel(ProductArgs a) {
  constexpr int HN = 64;
  typedef Half<64, false, 8> HA;
  typedef Half<HN, false, 8> HB;
  constexpr int TM = 4;  // 16 x 16 tiles of a wave
  constexpr int kStage = HA::kBytes + 2 * HB::kBytes, kStages = 5;
  constexpr int kPitch = 2 * HN + 4;
  __shared__ __attribute__((aligned(1024))) char lds[kStages * kStage];
  static_assert(64 * kPitch * 4 <= kStages * kStage, "the sums go out through the stages");

  const bool gated = a.e.gated;
  const int width = gated ? HN : 2 * HN;
  const int n0 = (int)block_number<512>(blockIdx.x, blockIdx.z) * width;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64;
  constexpr int kStep = 128 / Step::kBytes;
  const int k0 = blockIdx.y * a.k_tiles_per_split;
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
  const int turn = kn > 0 ? (int)((blockIdx.x * 7u + blockIdx.y) % (uint32_t)kn) : 0;
  auto fetch = [&](int kt, int stage) {
    int t = kt + turn;
    t = t >= kn ? t - kn : t;
    const uint32_t past = kt < kn ? HA::past(left - t * 128) : 0x80000000u;
    const uint32_t to = base + stage * kStage + w * 1024;
    HA::load(to, ra, va, t * 128, past);
#pragma unroll
    for (int h = 0; h < 2; ++h) HB::load(to + HA::kBytes + h * HB::kBytes, rb[h], vb, t * 128, past);
  };
  typename Step::Acc acc[TM];
#pragma unroll
  for (int x = 0; x < TM; ++x) acc[x] = typename Step::Acc{0, 0, 0, 0};
  const int half = w / 4, col = (w % 4) * 16;  // this wave's columns
  uint32_t pa[2], pb[2];
  HA::addresses<TM>(base, 0, pa);
  HB::addresses<1>(base + HA::kBytes + half * HB::kBytes, col, pb);
  auto add = [&](int stage) {
    const uint32_t at = stage * kStage;
    i32x4 fb[2];
    HB::read<1>(pb, at, 0, fb);
#pragma unroll
    for (int x = 0; x < TM; ++x) {
      if (x * 16 >= a.m) break;
      i32x4 fa[2];
      HA::read<TM>(pa, at, x, fa);
      acc[x] = mma<Step>(fa, fb, acc[x]);
    }
  };
  // A stage's loads have arrived when only those of the stages after it are
  // left; after the barrier every wave's have, and every wave is done with the
  // stage before it, whose place the newest stage then takes.
  constexpr int kLoads = HA::kLoads + 2 * HB::kLoads;
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
      float *p = a.partial + ((int64_t)blockIdx.y * a.m + m) * a.ldp + n;
      store8<F32>(p, v);
      if (gated) store8<F32>(p + a.ldp / 2, u);
    } else {
      finish<8>(a.e, m, n, v, u);
    }
  }
}

// The splits' partial sums, added in order, through the epilogue.
template <bool WHOLE>
__global__ __launch_bounds__(256) void product_fold_kernel(const float *partial, int splits, int64_t ldp, Epilogue e) {
  const int n = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (n >= e.n) return;
  for (int m = blockIdx.y; m < e.m; m += gridDim.y) {
    float v[8], u[8], x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
    for (int s = 0; s < splits; ++s) {
      const float *p = partial + ((int64_t)s * e.m + m) * ldp + n;
      load8<F32>(p, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) add_part<WHOLE>(v[i], x[i]);
      if (e.gated) {
        load8<F32>(p + ldp / 2, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) add_part<WHOLE>(u[i], x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = whole_sum<WHOLE>(v[i]), u[i] = whole_sum<WHOLE>(u[i]);
    finish<8>(e, m, n, v, u);
  }
}

// The same for the shared tiles: 1/8 of a tile's rows a workgroup.
template <bool WHOLE>
__device__ __forceinline__ void fold_tile(const ProductArgs &a, int size, int block) {
  const bool gated = a.e.gated;
  const int tile_n = gated ? size / 2 : size, shift = __builtin_ctz(tile_n / 8), per = 1 << shift;
  const int tiles_m = (a.m + size - 1) / size, tiles_n = (a.n + tile_n - 1) / tile_n;
  const int rest = tiles_m * tiles_n - a.tiles_full;
  int tm, tn;
  tile_at(a.tiles_full + block, tiles_m, tiles_n, tm, tn);
  for (int at = threadIdx.x; at < size / 8 * per; at += 256) {
    const int r = blockIdx.y * (size / 8) + (at >> shift), c = (at & (per - 1)) * 8, m = tm * size + r, n = tn * tile_n + c;
    if (m >= a.m || n >= a.n) continue;
    float v[8], u[8], x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
      const float *p = a.partial + (((int64_t)s * rest + block) * a.part_rows + r) * a.part_cols + c;
      load8<F32>(p, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) add_part<WHOLE>(v[i], x[i]);
      if (gated) {
        load8<F32>(p + a.part_cols / 2, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) add_part<WHOLE>(u[i], x[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = whole_sum<WHOLE>(v[i]), u[i] = whole_sum<WHOLE>(u[i]);
    finish<8>(a.e, m, n, v, u);
  }
}

template <bool WHOLE>
__global__ __launch_bounds__(256) void product_tile_fold_kernel(ProductArgs a, ProductArgs b, int first, int size) {
  if ((int)blockIdx.x < first)
    fold_tile<WHOLE>(a, size, blockIdx.x);
  else
    fold_tile<WHOLE>(b, size, blockIdx.x - first);
}

// The tiles that are shared by workgroups, and the workgroups of a product.
int64_t shared_tiles(const ProductArgs &a) {
  const int64_t tile = a.tile == 0 ? 256 : 128, tile_n = a.e.gated ? tile / 2 : tile;
  return ((a.m + tile - 1) / tile) * ((a.n + tile_n - 1) / tile_n) - a.tiles_full;
}
unsigned groups_of(const ProductArgs &a) { return (unsigned)(a.tiles_full + shared_tiles(a) * a.splits); }

// b may be empty (m = 0)
hipError_t fold_shared(const ProductArgs &a, const ProductArgs &b, hipStream_t s) {
  const int64_t x = a.splits > 1 ? shared_tiles(a) : 0, y = b.splits > 1 ? shared_tiles(b) : 0;
  if (x + y == 0) return hipSuccess;
  return launch(a.dtype == HF_S8 ? product_tile_fold_kernel<true> : product_tile_fold_kernel<false>,
                dim3((unsigned)(x + y), 8), 256, s, a, b, (int)x, a.tile == 0 ? 256 : 128);
}

template <class Step>
hipError_t go(const ProductArgs &a, hipStream_t s) {
  hipError_t e = hipErrorInvalidValue;
  if (a.tile == 1) {
    e = launch(product_kernel<Step, 64, 64>, dim3(groups_of(a)), 256, s, a);
  } else if constexpr (!Step::kWide) {  // never planned with kWide
    e = launch(product_kernel<Step, 128, 128>, dim3(groups_of(a)), 512, s, a);
  }
  return e != hipSuccess ? e : fold_shared(a, ProductArgs{}, s);
}

template <class Step>
hipError_t go_gradient(const ProductArgs &da, const ProductArgs &db, hipStream_t s) {
  const unsigned x = groups_of(da), y = groups_of(db);
  if (x + y == 0) return hipSuccess;
  const hipError_t e = da.tile == 0 ? launch(gradient_kernel<Step, 128, 128>, dim3(x + y), 512, s, da, db, (int)x)
                                    : launch(gradient_kernel<Step, 64, 64>, dim3(x + y), 256, s, da, db, (int)x);
  return e != hipSuccess ? e : fold_shared(da, db, s);
}

template <class Step>
hipError_t go_strip(const ProductArgs &a, hipStream_t s) {
  const int width = a.e.gated ? 64 : 128;
  const dim3 strips = grid_of<512>((a.n + width - 1) / width), grid(strips.x, (unsigned)a.splits, strips.y);
  const hipError_t e = launch(strip_kernel<Step>, grid, 512, s, a);
  return e != hipSuccess || a.splits == 1 ? e : launch_product_fold(a, s);
}

template <class Step>
hipError_t either(const ProductArgs &a, hipStream_t s) {
  return a.tile == 2 ? go_strip<Step>(a, s) : go<Step>(a, s);
}

}  // namespace

hipError_t launch_product(const ProductArgs &a, hipStream_t s) {
  if (a.dtype == HF_BF16) return either<StepBF16>(a, s);
  if (a.dtype == HF_F16) return either<StepF16>(a, s);
  if (a.dtype == HF_F8E4M3) return f8_wide(a.e.out_dtype, a.k) ? either<StepF8Wide>(a, s) : either<StepF8>(a, s);
  return either<StepS8>(a, s);
}

hipError_t launch_gradient(const ProductArgs &da, const ProductArgs &db, hipStream_t s) {
  return da.dtype == HF_BF16 ? go_gradient<StepBF16>(da, db, s) : go_gradient<StepF16>(da, db, s);
}

hipError_t launch_product_fold(const ProductArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.e.n + 2047) / 2048), (unsigned)(a.e.m < 65535 ? a.e.m : 65535));
  return launch(a.dtype == HF_S8 ? product_fold_kernel<true> : product_fold_kernel<false>, grid, 256, s, a.partial,
                a.splits, a.ldp, a.e);
}

}  // namespace hf
