// skinny.hip -- the product for few rows (single tokens, small decode
// batches), bound by reading the weights.
#include "product_epilogue.h"

namespace hf {
namespace {

// A workgroup computes 16 columns of d (gated: 16 and their up half) for all
// rows: the matrix instructions take 16, the plan gives it up to 8.  Its WAVES waves share out the contraction in blocks and join
// their sums through LDS at the end, so that enough loads are in flight for
// the memory though a layer has only a few hundred column groups.  Operands go
// from memory straight to the registers in which the matrix instructions take
// them: a lane reads 16 bytes of one row, 4 lanes 64 bytes of it, and the next
// load the next 64.  b is read once by the whole launch; a comes from L2, once
// for every 16 columns, which is why more than 8 rows are the strips' (there a
// is read once for 128 columns): 16 x 4096 x 16384 bf16 takes 36 us here and
// 32 us there, 1 row 26 us here (5.2 TB/s) and 30 us there.
template <class Step, bool GATED, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void skinny_kernel(SkinnyArgs s) {
  const ProductArgs &a = s.p;
  constexpr int NB = GATED ? 2 : 1;
  constexpr int Q = 2, kBlock = Q * 128;  // steps and bytes of a block
  typedef typename Step::Acc Acc;
  __shared__ __attribute__((aligned(16))) Acc part[WAVES / 2][NB][64];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64;
  const int n0 = blockIdx.x * 16;
  const int bytes = a.k * Step::kBytes;
  const int first = blockIdx.y * s.blocks_per_split * 512;
  const int last = min(bytes, first + s.blocks_per_split * 512);
  // rows past the edge read the last row: their sums are not stored
  const char *pb[NB], *pa;
#pragma unroll
  for (int h = 0; h < NB; ++h)
    pb[h] = (const char *)a.b + (int64_t)min(n0 + (l & 15), a.n - 1) * a.ldb + h * a.b_half + (l >> 4) * 16;
  pa = (const char *)a.a + (int64_t)min(l & 15, a.m - 1) * a.lda + (l >> 4) * 16;
  Acc acc[NB];
#pragma unroll
  for (int h = 0; h < NB; ++h) acc[h] = Acc{0, 0, 0, 0};
  struct Block {
    i32x4 b[NB][Q][2], a[Q][2];
  };
  auto load = [&](int k, Block &f) {
#pragma unroll
    for (int q = 0; q < 2 * Q; ++q) {
#pragma unroll
      for (int h = 0; h < NB; ++h) f.b[h][q / 2][q % 2] = __builtin_nontemporal_load((const i32x4 *)(pb[h] + k + q * 64));
    }
#pragma unroll
    for (int q = 0; q < 2 * Q; ++q) f.a[q / 2][q % 2] = *(const i32x4 *)(pa + k + q * 64);
  };
  auto add = [&](const Block &f) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int h = 0; h < NB; ++h) acc[h] = mma<Step>(f.a[q], f.b[h][q], acc[h]);
  };
  // A workgroup's blocks begin at a place of its own and go round: with all
  // of them at the same place of rows that are a power of two apart, only
  // some of the memory's channels would be busy at a time (1 x 4096 x 16384:
  // 38 us without, 26 us with).  A block's loads are issued while the block
  // before it is multiplied; left to itself, the compiler keeps 5 loads in
  // flight.
  const int blocks = (last - first) / kBlock;
  const int turn = blocks > 0 ? (int)(blockIdx.x * 11u % (uint32_t)blocks) : 0;
  auto at = [&](int j) {
    const int b = j + turn;
    return first + (b >= blocks ? b - blocks : b) * kBlock;
  };
  if (w < blocks) {
    const int n = (blocks - w + WAVES - 1) / WAVES;  // this wave's
    Block x, y;
    load(at(w), x);
    int i = 0;
    for (; i + 2 < n; i += 2) {
      load(at(w + (i + 1) * WAVES), y);
      __builtin_amdgcn_sched_barrier(0);
      add(x);
      load(at(w + (i + 2) * WAVES), x);
      __builtin_amdgcn_sched_barrier(0);
      add(y);
    }
    if (i + 1 < n) {
      load(at(w + (i + 1) * WAVES), y);
      __builtin_amdgcn_sched_barrier(0);
      add(x);
      add(y);
    } else {
      add(x);
    }
  }
  const int k = w == blocks % WAVES ? first + blocks * kBlock : last;
  if (k < last) {  // the contraction's ragged end: chunks past it are zero
    for (int c = k; c < last; c += 128) {
      i32x4 fb[NB][2], fa[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool in = c + q * 64 + (l >> 4) * 16 < last;
#pragma unroll
        for (int h = 0; h < NB; ++h) fb[h][q] = in ? *(const i32x4 *)(pb[h] + c + q * 64) : i32x4{0, 0, 0, 0};
        fa[q] = in ? *(const i32x4 *)(pa + c + q * 64) : i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int h = 0; h < NB; ++h) acc[h] = mma<Step>(fa, fb[h], acc[h]);
    }
  }
  // join: the upper half of the waves hands its sums to the lower half, until
  // one is left
#pragma unroll
  for (int half = WAVES / 2; half; half /= 2) {
    if (w >= half && w < 2 * half) {
#pragma unroll
      for (int h = 0; h < NB; ++h) part[w - half][h][l] = acc[h];
    }
    __syncthreads();
    if (w < half) {
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        const Acc o = part[w][h][l];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[h][i] += o[i];
      }
    }
    __syncthreads();
  }
  if (w) return;
  const int m = l & 15, n = n0 + (l >> 4) * 4;
  if (a.splits > 1) {
    if (m < a.m && n < a.n) {
      float *p = a.partial + ((int64_t)blockIdx.y * a.m + m) * a.ldp + n;
      *(f32x4 *)p = Step::bits(acc[0]);
      if (GATED) *(f32x4 *)(p + a.ldp / 2) = Step::bits(acc[NB - 1]);
    }
  } else {
    const f32x4 gate = Step::sums(acc[0]), other = Step::sums(acc[NB - 1]);
    float v[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = gate[i], u[i] = other[i];
    finish<4>(a.e, m, n, v, u);
  }
}

template <class Step, bool GATED>
hipError_t go(const SkinnyArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.p.n + 15) / 16), (unsigned)a.p.splits);
  hipError_t e = hipErrorInvalidValue;
  // kWide is always planned with 8 waves; a gated product otherwise never, as
  // its 64 strips at most are no more than 256 groups of columns
  if constexpr (Step::kWide || !GATED) {
    if (a.waves == 8) e = launch(skinny_kernel<Step, GATED, 8>, grid, 512, s, a);
  }
  if constexpr (!Step::kWide) {
    if (a.waves == 16) e = launch(skinny_kernel<Step, GATED, 16>, grid, 1024, s, a);
  }
  return e != hipSuccess || a.p.splits == 1 ? e : launch_product_fold(a.p, s);
}

template <class Step>
hipError_t either(const SkinnyArgs &a, hipStream_t s) {
  return a.p.e.gated ? go<Step, true>(a, s) : go<Step, false>(a, s);
}

}  // namespace

hipError_t launch_skinny(const SkinnyArgs &a, hipStream_t s) {
  if (a.p.dtype == HF_BF16) return either<StepBF16>(a, s);
  if (a.p.dtype == HF_F16) return either<StepF16>(a, s);
  if (a.p.dtype == HF_F8E4M3)
    return f8_wide(a.p.e.out_dtype, a.p.k) ? either<StepF8Wide>(a, s) : either<StepF8>(a, s);
  return either<StepS8>(a, s);
}

}  // namespace hf
