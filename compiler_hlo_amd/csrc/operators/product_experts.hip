// product_experts.hip -- products by expert: the rows of a are sorted by
// expert, and each expert multiplies its own by its own weight.
#include "product_tile.h"

namespace hf {
namespace {

// Tiles of 256 or of 128 rows of one expert.  How many there are is in the
// offsets on the GPU: the grid holds as many as any offsets can ask for, and a
// workgroup without a tile ends at once.  Bound by the matrix cores and by what
// the experts' ragged ends and the last round leave of the chip: 8198 rows of 8
// experts, gated 4096 x 4096 bf16, 462 us, 1.19 PFLOP/s, where the last round has
// up to 128 tiles and is cut; 485 where it has 160, which are whole.
template <class Step>
__global__ __launch_bounds__(512, 2) void experts_large_kernel(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<128, 128>::lds(Step::kBlock)];
  const int width = a.e.gated ? 128 : 256, tiles_n = (a.n + width - 1) / width;
  ExpertTile t;
  if (expert_tile<true>(a.offsets, a.experts, a.m, 256, tiles_n, blockIdx.x, t)) large_tile<Step, false, false>(a, t, tiles_n, lds);
}

template <class Step, int PARTS>
__global__ __launch_bounds__(256, 2) void experts_small_kernel(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<64, 64>::lds(Step::kBlock)];
  const int width = a.e.gated ? 64 : 128;
  a.piece = blockIdx.y;
  ExpertTile t;
  if (!expert_tile<false>(a.offsets, a.experts, a.m, 128, (a.n + width - 1) / width, blockIdx.x, t)) return;
  product_tile<Step, false, false, 64, 64, PARTS>(part_of(a, t.expert, t.row, t.rows), t.local, lds);
}

// Strips for up to 64 rows of an expert, bound by reading the weights.  An
// expert with more has several; those of the same columns are neighbours and
// run at the same time on one XCD, so that its L2 has the weights for all but
// the first.  128 rows of 32 experts, gated 1408 x 4096 e4m3 with block scales:
// 74 us, 365 MB, 4.9 TB/s.
template <class Step>
__global__ __launch_bounds__(512, 2) void experts_strip_kernel(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[Strip<Step>::kLds];
  const int width = a.e.gated ? 64 : 128;
  a.piece = blockIdx.y;
  ExpertTile t;
  if (!expert_tile<false>(a.offsets, a.experts, a.m, 64, (a.n + width - 1) / width, blockIdx.x, t)) return;
  const int units = (t.rows + 63) / 64, strip = t.local / units, from = (t.local - strip * units) * 64;
  strip_tile<Step>(part_of(a, t.expert, t.row + from, min(64, t.rows - from)), strip, a.piece,
                   blockIdx.x / 8 * 7u + blockIdx.y, lds);
}

// The splits' partial sums, added in order, through the epilogue; with offsets,
// of the rows that are an expert's.
__global__ __launch_bounds__(256) void experts_fold_kernel(const float *partial, int splits, int64_t ldp, Epilogue e,
                                                           const int32_t *offsets, int experts) {
  // rows of any length side by side: eight columns a thread
  const int per = (e.n + 7) / 8;
  const int64_t id = block_number<256>(blockIdx.x, blockIdx.y) * 256 + threadIdx.x;
  const int m = (int)min(id / per, (int64_t)e.m), n = (int)(id % per) * 8;
  const int from = offsets ? max(offsets[0], 0) : 0, to = offsets ? min(offsets[experts], e.m) : e.m;
  if (m < from || m >= to) return;
  float v[8], u[8], x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.f;
  for (int s = 0; s < splits; ++s) {
    const float *p = partial + ((int64_t)s * e.m + m) * ldp + n;
    load8<F32>(p, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += x[i];
    if (e.gated) {
      load8<F32>(p + ldp / 2, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += x[i];
    }
  }
  finish<8>(e, m, n, v, u);
}

template <class Step>
hipError_t go(const ProductArgs &a, hipStream_t s) {
  const auto groups = [&](int64_t rows, int64_t cols) {
    const int64_t width = a.e.gated ? cols / 2 : cols;
    return dim3((unsigned)expert_tiles(a.m, a.experts, rows, (a.n + width - 1) / width), (unsigned)a.splits);
  };
  if (a.tile > 0) {
    hipError_t e = hipErrorInvalidValue;
    if (a.tile == 2) {
      e = launch(experts_strip_kernel<Step>, groups(64, 128), 512, s, a);
    } else if (a.splits == 1) {
      e = launch(experts_small_kernel<Step, kWhole>, groups(128, 128), 256, s, a);
    } else if constexpr (Step::kBlock || Step::kBytes == 2) {  // else never planned
      e = launch(experts_small_kernel<Step, kSplit>, groups(128, 128), 256, s, a);
    }
    return e != hipSuccess || a.splits == 1 ? e : launch_experts_fold(a, a.offsets, s);
  }
  if constexpr (!Step::kWide) {
    dim3 grid = groups(256, 256);
    grid.x += 128;  // the halves of as many tiles
    return launch(experts_large_kernel<Step>, grid, 512, s, a);
  }
  return hipErrorInvalidValue;  // never planned with kWide
}

}  // namespace

int64_t expert_tiles(int64_t m, int64_t experts, int64_t size, int64_t per) {
  return (m + (m < experts ? m : experts) * (size - 1)) / size * per;
}

hipError_t launch_experts_fold(const ProductArgs &a, const int32_t *offsets, hipStream_t s) {
  const int64_t threads = (int64_t)a.e.m * ((a.e.n + 7) / 8);
  return launch(experts_fold_kernel, grid_of<256>((threads + 255) / 256), 256, s, a.partial, a.splits, a.ldp, a.e, offsets, a.experts);
}

hipError_t launch_experts(const ProductArgs &a, hipStream_t s) {
  const bool wide = a.dtype == HF_F8E4M3 && f8_wide(a.e.out_dtype, a.k);
  if (a.a_scale) return wide ? go<StepF8BlockWide>(a, s) : go<StepF8Block>(a, s);
  if (a.dtype == HF_BF16) return go<StepBF16>(a, s);
  if (a.dtype == HF_F16) return go<StepF16>(a, s);
  if (a.dtype == HF_F8E4M3) return wide ? go<StepF8Wide>(a, s) : go<StepF8>(a, s);
  return go<StepS8>(a, s);
}

}  // namespace hf
