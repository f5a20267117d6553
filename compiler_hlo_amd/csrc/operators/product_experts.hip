// product_experts.hip -- products by expert: the rows of a are sorted by
// expert, and each expert multiplies its own by its own weight.
#include "product_tile.h"

namespace hf {
namespace {

// A tile of 256 x 256 of an expert, or, where it has no more than 128 rows or
// is cut, a half or two of them of 128 x 256, which take about 0.6 of its time.
template <class Step, bool ACOL, bool BCOL>
__device__ __forceinline__ void large_tile(const ProductArgs &a, const ExpertTile &t, int tiles_n, char *lds) {
  int tm, tn;
  tile_at(t.local, (t.rows + 255) / 256, tiles_n, tm, tn);
  const int from = tm * 256 + (t.half > 0 ? 128 : 0), left = t.rows - from;
  if (left <= 0) return;
  if (t.half >= 0 || left <= 128)
    product_tile<Step, ACOL, BCOL, 64, 128, true>(part_of(a, t.expert, t.row + from, min(left, 128)), tn, lds);
  else
    product_tile<Step, ACOL, BCOL, 128, 128, true>(part_of(a, t.expert, t.row, t.rows), t.local, lds);
}

// Tiles of 256 or of 128 rows of one expert.  How many there are is in the
// offsets on the GPU: the grid holds as many as any offsets can ask for, and a
// workgroup without a tile ends at once.  Bound by the matrix cores and by what
// the experts' ragged ends and the last round leave of the chip: 8198 rows of 8
// experts, gated 4096 x 4096 bf16, 469 us, 1.17 PFLOP/s (up to 550 where the
// last round has more than 128 tiles).
template <class Step>
__global__ __launch_bounds__(512, 2) void experts_large_kernel(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<128, 128>::lds(Step::kBlock)];
  const int width = a.e.gated ? 128 : 256, tiles_n = (a.n + width - 1) / width;
  ExpertTile t;
  if (expert_tile<true>(a.offsets, a.experts, a.m, 256, tiles_n, blockIdx.x, t)) large_tile<Step, false, false>(a, t, tiles_n, lds);
}

template <class Step>
__global__ __launch_bounds__(256, 2) void experts_small_kernel(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<64, 64>::lds(Step::kBlock)];
  const int width = a.e.gated ? 64 : 128;
  ExpertTile t;
  if (!expert_tile<false>(a.offsets, a.experts, a.m, 128, (a.n + width - 1) / width, blockIdx.x, t)) return;
  product_tile<Step, false, false, 64, 64, true>(part_of(a, t.expert, t.row, t.rows), t.local, lds);
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
  ExpertTile t;
  if (!expert_tile<false>(a.offsets, a.experts, a.m, 64, (a.n + width - 1) / width, blockIdx.x, t)) return;
  const int units = (t.rows + 63) / 64, strip = t.local / units, from = (t.local - strip * units) * 64;
  strip_tile<Step>(part_of(a, t.expert, t.row + from, min(64, t.rows - from)), strip, 0, blockIdx.x / 8 * 7u, lds);
}

// db's tiles are as long as their expert has rows, so an XCD does not take a
// contiguous run of them (one or two experts' all): they are dealt out in
// chunks of up to four tile rows, which share their operands in an L2, and the
// first XCD moves on by one with every eight chunks.  (16 experts of 1024 rows
// on average, some with three times as many as others, 16384 x 4096 x 1408 bf16:
// 501 us with contiguous runs.)
__device__ __forceinline__ int dealt(int block, int chunk) {
  const int xcd = block % 8, j = block / 8, turn = j / chunk;
  return (turn * 8 + (xcd + turn) % 8) * chunk + j % chunk;
}
__host__ __device__ __forceinline__ int chunk_of(int all, int tiles_n) { return max(1, min(4 * tiles_n, all / 128)); }

// The expert with the `place`-th most rows (of equal ones the lower first), so
// that the longest tiles begin first; of more than 64 experts the place itself.
__device__ __forceinline__ ExpertTile by_rows(const int32_t *offsets, int experts, int m, int place) {
  const int l = threadIdx.x % 64, at = experts > 64 ? place : min(l, experts - 1);
  const int lo = min(max(offsets[at], 0), m), hi = min(max(offsets[at + 1], lo), m), rows = hi - lo;
  int lane = 0;
  if (experts <= 64) {
    int before = 0;
    for (int e = 0; e < experts; ++e) {
      const int r = __builtin_amdgcn_readlane(rows, e);
      before += r > rows || (r == rows && e < l) ? 1 : 0;
    }
    lane = __builtin_ctzll(__ballot(l < experts && before == place));
  }
  ExpertTile t{};
  t.expert = experts > 64 ? place : lane;
  t.row = __builtin_amdgcn_readlane(lo, lane);
  t.rows = __builtin_amdgcn_readlane(rows, lane);
  return t;
}

// The gradient: da as the products above, with b's rows as the contraction,
// and db[e] = dz^T a over the expert's rows (zeros where it has none), in one
// launch.  16384 rows of 16 experts, 4096 x 1408 bf16: 401 us, 0.94 PFLOP/s.
// db's contraction is an expert's rows, 16 stages on average there, and a
// tile's end is as long as 8 of them.
template <class Step, int HM, int HN>
__global__ __launch_bounds__(HM == 128 ? 512 : 256, 2) void experts_gradient_kernel(ProductArgs da, ProductArgs db, int first) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<HM, HN>::lds(false)];
  const int tiles_n = (max(da.n, db.n) + 2 * HN - 1) / (2 * HN);  // of one that may be empty
  if ((int)blockIdx.x < first) {
    ExpertTile t;
    if (!expert_tile<false>(da.offsets, da.experts, da.m, 2 * HM, tiles_n, blockIdx.x, t)) return;
    if constexpr (HM == 128)
      large_tile<Step, false, true>(da, t, tiles_n, lds);
    else
      product_tile<Step, false, true, HM, HN, true>(part_of(da, t.expert, t.row, t.rows), t.local, lds);
    return;
  }
  const int tiles = (db.m + 2 * HM - 1) / (2 * HM) * tiles_n, all = tiles * db.experts;
  const int id = dealt(blockIdx.x - first, chunk_of(all, tiles_n));
  if (id >= all) return;
  const ExpertTile t = by_rows(db.offsets, db.experts, db.k, id / tiles);
  const int row = t.row, rows = t.rows;
  ProductArgs p = db;
  p.a = (const char *)db.a + row * db.lda;
  p.b = (const char *)db.b + row * db.ldb;
  p.a_bytes = rows > 0 ? (rows - 1) * db.lda + db.a_bytes : 0;
  p.b_bytes = rows > 0 ? (rows - 1) * db.ldb + db.b_bytes : 0;
  p.k = rows;
  p.e.d = (char *)db.e.d + t.expert * (int64_t)db.m * db.e.ldd * 2;
  product_tile<Step, true, true, HM, HN, true>(p, id % tiles, lds);
}

template <class Step>
hipError_t go(const ProductArgs &a, hipStream_t s) {
  const auto groups = [&](int64_t rows, int64_t cols) {
    const int64_t width = a.e.gated ? cols / 2 : cols;
    return dim3((unsigned)expert_tiles(a.m, a.experts, rows, (a.n + width - 1) / width));
  };
  if (a.tile == 2) return launch(experts_strip_kernel<Step>, groups(64, 128), 512, s, a);
  if (a.tile == 1) return launch(experts_small_kernel<Step>, groups(128, 128), 256, s, a);
  if constexpr (!Step::kWide) {
    dim3 grid = groups(256, 256);
    grid.x += 128;  // the halves of as many tiles
    return launch(experts_large_kernel<Step>, grid, 512, s, a);
  }
  return hipErrorInvalidValue;  // never planned with kWide
}

template <class Step>
hipError_t go_gradient(const ProductArgs &da, const ProductArgs &db, hipStream_t s) {
  const int64_t size = da.tile == 0 ? 256 : 128, across = ((da.n > db.n ? da.n : db.n) + size - 1) / size;
  // a multiple of 8, so that db's tiles begin at the first XCD too
  const int64_t first = (expert_tiles(da.m, da.experts, size, across) + 7) / 8 * 8;
  // whole turns of eight chunks
  const int64_t all = db.experts * ((db.m + size - 1) / size) * across, turn = 8 * chunk_of((int)all, (int)across);
  const dim3 grid((unsigned)(first + (all + turn - 1) / turn * turn));
  if (grid.x == 0) return hipSuccess;
  return da.tile == 0 ? launch(experts_gradient_kernel<Step, 128, 128>, grid, 512, s, da, db, (int)first)
                      : launch(experts_gradient_kernel<Step, 64, 64>, grid, 256, s, da, db, (int)first);
}

}  // namespace

int64_t expert_tiles(int64_t m, int64_t experts, int64_t size, int64_t per) {
  return (m + (m < experts ? m : experts) * (size - 1)) / size * per;
}

hipError_t launch_experts(const ProductArgs &a, hipStream_t s) {
  const bool wide = a.dtype == HF_F8E4M3 && f8_wide(a.e.out_dtype, a.k);
  if (a.a_scale) return wide ? go<StepF8BlockWide>(a, s) : go<StepF8Block>(a, s);
  if (a.dtype == HF_BF16) return go<StepBF16>(a, s);
  if (a.dtype == HF_F16) return go<StepF16>(a, s);
  if (a.dtype == HF_F8E4M3) return wide ? go<StepF8Wide>(a, s) : go<StepF8>(a, s);
  return go<StepS8>(a, s);
}

hipError_t launch_experts_gradient(const ProductArgs &da, const ProductArgs &db, hipStream_t s) {
  return da.dtype == HF_BF16 ? go_gradient<StepBF16>(da, db, s) : go_gradient<StepF16>(da, db, s);
}

}  // namespace hf
