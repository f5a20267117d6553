// skinny.hip -- the product for few rows (single tokens, decode batches),
// bound by reading the weights.
#include "product_epilogue.h"

namespace hf {
namespace {

// A workgroup computes 16 columns of d (gated: 16 and their up half) for all
// m <= 16 MT rows.  Its WAVES waves share out the contraction in blocks of
// 512 bytes and join their sums through LDS at the end, so that enough loads
// are in flight for the memory though a layer has only a few hundred column
// groups.  Operands go from memory straight to the registers in which the
// matrix instructions take them: a lane reads 16 bytes of one row, 4 lanes 64
// bytes of it, and the next load the next 64.  b is read once by the whole
// launch; a (m rows) comes from L2.
template <class Step, int MT, bool GATED, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void skinny_kernel(SkinnyArgs s) {
  const ProductArgs &a = s.p;
  constexpr int NB = GATED ? 2 : 1;
  typedef typename Step::Acc Acc;
  __shared__ __attribute__((aligned(16))) f32x4 part[WAVES / 2][NB * MT][64];
  const int w = threadIdx.x / 64, l = threadIdx.x % 64;
  const int n0 = blockIdx.x * 16;
  const int bytes = a.k * Step::kBytes;
  const int first = blockIdx.y * s.blocks_per_split * 512;
  const int last = min(bytes, first + s.blocks_per_split * 512);
  // rows past the edge read the last row: their sums are not stored
  const char *pb[NB], *pa[MT];
#pragma unroll
  for (int h = 0; h < NB; ++h)
    pb[h] = (const char *)a.b + (int64_t)min(n0 + (l & 15), a.n - 1) * a.ldb + h * a.b_half + (l >> 4) * 16;
#pragma unroll
  for (int t = 0; t < MT; ++t)
    pa[t] = (const char *)a.a + (int64_t)min(t * 16 + (l & 15), a.m - 1) * a.lda + (l >> 4) * 16;
  Acc acc[NB][MT];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[h][t] = Acc{0, 0, 0, 0};
  int k = first + w * 512;
  for (; k + 512 <= last; k += WAVES * 512) {
    i32x4 fb[NB][4][2], fa[MT][4][2];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
#pragma unroll
      for (int h = 0; h < NB; ++h) fb[h][q / 2][q % 2] = __builtin_nontemporal_load((const i32x4 *)(pb[h] + k + q * 64));
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
#pragma unroll
      for (int t = 0; t < MT; ++t) fa[t][q / 2][q % 2] = *(const i32x4 *)(pa[t] + k + q * 64);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < NB; ++h) acc[h][t] = Step::mma(fa[t][q], fb[h][q], acc[h][t]);
  }
  if (k < last) {  // the contraction's ragged end: chunks past it are zero
    for (int c = k; c < last; c += 128) {
      i32x4 fb[NB][2], fa[MT][2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool in = c + q * 64 + (l >> 4) * 16 < last;
#pragma unroll
        for (int h = 0; h < NB; ++h) fb[h][q] = in ? *(const i32x4 *)(pb[h] + c + q * 64) : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < MT; ++t) fa[t][q] = in ? *(const i32x4 *)(pa[t] + c + q * 64) : i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < NB; ++h) acc[h][t] = Step::mma(fa[t], fb[h], acc[h][t]);
    }
  }
  // join: the upper half of the waves hands its sums to the lower half, until
  // one is left
  f32x4 sum[NB][MT];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int t = 0; t < MT; ++t) sum[h][t] = Step::sums(acc[h][t]);
#pragma unroll
  for (int half = WAVES / 2; half; half /= 2) {
    if (w >= half && w < 2 * half) {
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int t = 0; t < MT; ++t) part[w - half][h * MT + t][l] = sum[h][t];
    }
    __syncthreads();
    if (w < half) {
#pragma unroll
      for (int h = 0; h < NB; ++h)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const f32x4 o = part[w][h * MT + t][l];
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[h][t][i] += o[i];
        }
    }
    __syncthreads();
  }
  if (w) return;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = t * 16 + (l & 15), n = n0 + (l >> 4) * 4;
    if (a.splits > 1) {
      if (m < a.m && n < a.n) {
        float *p = a.partial + ((int64_t)blockIdx.y * a.m + m) * a.ldp + n;
        *(f32x4 *)p = sum[0][t];
        if (GATED) *(f32x4 *)(p + a.ldp / 2) = sum[NB - 1][t];
      }
    } else {
      float v[4], u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = sum[0][t][i], u[i] = sum[NB - 1][t][i];
      finish<4>(a.e, m, n, v, u);
    }
  }
}

template <class Step, int MT, bool GATED>
hipError_t go(const SkinnyArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)((a.p.n + 15) / 16), (unsigned)a.p.splits);
  if constexpr (MT <= 2) {
    if (a.waves == 16) {
      skinny_kernel<Step, MT, GATED, 16><<<grid, 1024, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  skinny_kernel<Step, MT, GATED, 8><<<grid, 512, 0, s>>>(a);
  return hipGetLastError();
}

template <class Step>
hipError_t by_rows(const SkinnyArgs &a, hipStream_t s) {
  if (a.p.e.gated) {
    if (a.p.m <= 16) return go<Step, 1, true>(a, s);
    if (a.p.m <= 32) return go<Step, 2, true>(a, s);
    return go<Step, 4, true>(a, s);
  }
  if (a.p.m <= 16) return go<Step, 1, false>(a, s);
  if (a.p.m <= 32) return go<Step, 2, false>(a, s);
  return go<Step, 4, false>(a, s);
}

}  // namespace

hipError_t launch_skinny(const SkinnyArgs &a, hipStream_t s) {
  if (a.p.dtype == HF_BF16) return by_rows<StepBF16>(a, s);
  if (a.p.dtype == HF_F16) return by_rows<StepF16>(a, s);
  if (a.p.dtype == HF_F8E4M3)
    return f8_wide(a.p.e.out_dtype, a.p.k) ? by_rows<StepF8Wide>(a, s) : by_rows<StepF8>(a, s);
  return by_rows<StepS8>(a, s);
}

}  // namespace hf
