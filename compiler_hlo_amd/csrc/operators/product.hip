// product.hip -- the tiled product d = epilogue(a b^T) on the matrix cores.
#include "product_tile.h"

namespace hf {
namespace {

template <class Step, int HM, int HN>
__global__ __launch_bounds__(HM == 128 ? 512 : 256, 2) void product_kernel(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<HM, HN>::lds(Step::kBlock)];
  product_tile<Step, false, false, HM, HN>(a, blockIdx.x, lds);
}

// The two products of a gradient, da = dz b and db = dz^T a, in one launch:
// neither needs the other, small ones fill the chip together and large ones
// share their last round.
template <class Step, int HM, int HN>
__global__ __launch_bounds__(HM == 128 ? 512 : 256, 2) void gradient_kernel(ProductArgs da, ProductArgs db, int first) {
  __shared__ __attribute__((aligned(1024))) char lds[Shape<HM, HN>::lds(Step::kBlock)];
  if ((int)blockIdx.x < first)
    product_tile<Step, false, true, HM, HN>(da, blockIdx.x, lds);
  else
    product_tile<Step, true, true, HM, HN>(db, blockIdx.x - first, lds);
}

template <class Step>
__global__ __launch_bounds__(512, 2) void strip_kernel(ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char lds[Strip<Step>::kLds];
  a.partial += (int64_t)blockIdx.y * a.m * a.ldp;
  strip_tile<Step>(a, (int)block_number<512>(blockIdx.x, blockIdx.z), blockIdx.y, blockIdx.x * 7u + blockIdx.y, lds);
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
  if (a.a_scale)
    return f8_wide(a.e.out_dtype, a.k) ? either<StepF8BlockWide>(a, s) : either<StepF8Block>(a, s);
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
