// product_experts_grad.hip -- the gradient of products by expert.
#include "product_tile.h"

namespace hf {
namespace {

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
template <class Step, int HM, int HN, int DA, int DB>
__global__ __launch_bounds__(HM == 128 ? 512 : 256, 2) void experts_gradient_kernel(ProductArgs da, ProductArgs db, int first,
                                                                                    int second) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<HM, HN>::lds(false)];
  const int tiles_n = (max(da.n, db.n) + 2 * HN - 1) / (2 * HN);  // of one that may be empty
  int block = blockIdx.x;
  const int pieces = DA == kSplit ? da.splits : 1;
  if (block < first * pieces) {
    da.piece = DA == kSplit ? block / first : 0;
    ExpertTile t;
    if (!expert_tile<false>(da.offsets, da.experts, da.m, 2 * HM, tiles_n, block - da.piece * first, t)) return;
    if constexpr (HM == 128)
      large_tile<Step, false, true>(da, t, tiles_n, lds);
    else
      product_tile<Step, false, true, HM, HN, DA>(part_of(da, t.expert, t.row, t.rows), t.local, lds);
    return;
  }
  block -= first * pieces;
  const int piece = DB == kSplit ? block / second : 0;
  const int tiles = (db.m + 2 * HM - 1) / (2 * HM) * tiles_n, all = tiles * db.experts;
  const int id = dealt(block - piece * second, chunk_of(all, tiles_n));
  if (id >= all) return;
  const ExpertTile t = by_rows(db.offsets, db.experts, db.k, id / tiles);
  const int row = t.row, rows = t.rows;
  ProductArgs p = db;
  p.a = (const char *)db.a + row * db.lda;
  p.b = (const char *)db.b + row * db.ldb;
  p.a_bytes = rows > 0 ? (rows - 1) * db.lda + db.a_bytes : 0;
  p.b_bytes = rows > 0 ? (rows - 1) * db.ldb + db.b_bytes : 0;
  p.k = rows;
  p.piece = piece;
  // an expert's own share of its rows, in stages of 64
  p.k_tiles_per_split = max(1, ((rows + 63) / 64 + db.splits - 1) / db.splits);
  p.partial = db.partial + ((int64_t)piece * db.experts + t.expert) * db.m * db.ldp;
  p.e.d = (char *)db.e.d + t.expert * (int64_t)db.m * db.e.ldd * 2;
  product_tile<Step, true, true, HM, HN, DB>(p, id % tiles, lds);
}

template <class Step>
hipError_t go_gradient(const ProductArgs &da, const ProductArgs &db, hipStream_t s) {
  const int64_t size = da.tile == 0 ? 256 : 128, across = ((da.n > db.n ? da.n : db.n) + size - 1) / size;
  // a multiple of 8, so that db's tiles begin at the first XCD too
  const int64_t first = (expert_tiles(da.m, da.experts, size, across) + 7) / 8 * 8;
  // whole turns of eight chunks
  const int64_t all = db.experts * ((db.m + size - 1) / size) * across, turn = 8 * chunk_of((int)all, (int)across);
  const int64_t second = (all + turn - 1) / turn * turn;
  const dim3 grid((unsigned)(first * da.splits + second * db.splits));
  if (grid.x == 0) return hipSuccess;
  const auto go = [&](auto kernel, unsigned block) { return launch(kernel, grid, block, s, da, db, (int)first, (int)second); };
  hipError_t e;
  if (da.tile == 0) e = go(experts_gradient_kernel<Step, 128, 128, kWhole, kWhole>, 512);  // never split
  else if (da.splits == 1 && db.splits == 1) e = go(experts_gradient_kernel<Step, 64, 64, kWhole, kWhole>, 256);
  else if (db.splits == 1) e = go(experts_gradient_kernel<Step, 64, 64, kSplit, kWhole>, 256);
  else if (da.splits == 1) e = go(experts_gradient_kernel<Step, 64, 64, kWhole, kSplit>, 256);
  else e = go(experts_gradient_kernel<Step, 64, 64, kSplit, kSplit>, 256);
  if (e == hipSuccess && da.splits > 1) e = launch_experts_fold(da, da.offsets, s);
  if (e == hipSuccess && db.splits > 1) {
    ProductArgs whole = db;  // all experts' rows
    whole.e.m = db.experts * db.m;
    e = launch_experts_fold(whole, nullptr, s);
  }
  return e;
}

}  // namespace

hipError_t launch_experts_gradient(const ProductArgs &da, const ProductArgs &db, hipStream_t s) {
  return da.dtype == HF_BF16 ? go_gradient<StepBF16>(da, db, s) : go_gradient<StepF16>(da, db, s);
}

}  // namespace hf
