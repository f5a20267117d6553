// product.hip -- the tiled product d = epilogue(a b^T) on the matrix cores.
#include "product_epilogue.h"

namespace hf {
namespace {

typedef __attribute__((address_space(3))) char lds_char;

// A view of an operand from a byte on, as the buffer loads want it: they
// return zeros past the operand's end, so ragged edges need no branch.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t view(const char *p, int64_t left) {
  const int64_t n = left < 0 ? 0 : left > 0x7fffffff ? 0x7fffffff : left;
  return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)n, 0x00020000);
}

// One half (R rows of the operand's tile, 128 bytes of the contraction) of a
// stage in LDS, and how it gets there.
//
// By row (the contraction lies along the operand's rows): LDS row r holds the
// 8 16-byte chunks of tile row r, chunk c at slot c ^ (r % 8), so that the 8
// lanes that read one chunk of 8 rows meet 8 different slots.
// By column (the contraction runs over the operand's rows; 16-bit types):
// LDS row k holds R columns of contraction step k in units of 16 columns (32
// bytes), unit u at u ^ f(k) with f(k) = k % 4 + 4 (k / 8 % 2) (R = 64:
// k % 4), so that the 16 lanes that read 4 steps of one unit, and the next 16
// lanes 8 steps on, meet different banks; ds_read_b64_tr_b16 turns the unit.
//
// The loads write LDS directly, 1 KiB a wave: lane l of a wave fills bytes
// 16 l .. of its kilobyte, so the swizzle is in which global bytes it asks
// for.
template <int R, bool COL>
struct Half {
  static constexpr int kBytes = R * 128;
  static constexpr int kLoads = kBytes / 8192;  // 16-byte loads a thread

  // The global offsets of this thread's loads, from the tile's first row (by
  // row) or first column (by column) at the stage's first contraction byte.
  static __device__ __forceinline__ void offsets(int64_t ld, uint32_t (&v)[kLoads]) {
    const int w = threadIdx.x / 64, l = threadIdx.x % 64;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int piece = w + 8 * i;
      if (!COL) {
        const int row = piece * 8 + l / 8;
        v[i] = (uint32_t)(row * ld) + (uint32_t)(((l & 7) ^ (l >> 3)) * 16);
      } else {
        constexpr int per = R * 2 / 16;  // lanes a step
        const int k = piece * (64 / per) + l / per, slot = l % per;
        const int f = (k & 3) | (R == 128 ? ((k >> 3) & 1) << 2 : 0);
        v[i] = (uint32_t)(k * ld) + (uint32_t)((((slot >> 1) ^ f) * 32) + (slot & 1) * 16);
      }
    }
  }
  // by row: set where this thread's chunk lies past `left` contraction bytes
  static __device__ __forceinline__ uint32_t past(int left) {
    const int l = threadIdx.x % 64;
    return !COL && ((l & 7) ^ (l >> 3)) * 16 >= left ? 0x80000000u : 0u;
  }
  static __device__ __forceinline__ void load(lds_char *lds, __amdgpu_buffer_rsrc_t r, const uint32_t (&v)[kLoads],
                                              uint32_t past) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          r, (__attribute__((address_space(3))) void *)(lds + ((threadIdx.x / 64) + 8 * i) * 1024), 16, v[i] | past, 0,
          0, 0);
  }

  // The fragment of rows (by column: columns) base + 16 t + l % 16.
  static __device__ __forceinline__ void read(const lds_char *lds, int base, int t, i32x4 (&f)[2]) {
    const int l = threadIdx.x % 64;
    if (!COL) {
      const lds_char *p = lds + (base + t * 16 + (l & 15)) * 128;
      f[0] = *(const __attribute__((address_space(3))) i32x4 *)(p + (((l >> 4) ^ (l & 7)) * 16));
      f[1] = *(const __attribute__((address_space(3))) i32x4 *)(p + (((l >> 4) ^ (l & 7) ^ 4) * 16));
    } else {
      const int g = l >> 4, i = l & 15, s = (i >> 2) | (R == 128 ? (g & 1) << 2 : 0);
      const lds_char *p = lds + (g * 8 + (i >> 2)) * (R * 2) + (((base / 16 + t) ^ s) * 32) + (i & 3) * 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        typedef __attribute__((address_space(3))) i16x4 tr;
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr *)(p + (h * 32) * (R * 2)));
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr *)(p + (h * 32 + 4) * (R * 2)));
        f[h] = __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  }
};

// A workgroup of 8 waves computes 2 HM x 2 HN sums (HM = HN = 128: 256 x 256;
// 64: 128 x 128), 128 contraction bytes a stage, two stages in LDS.  A wave
// has, in each quarter of the tile, HM/2 x HN/4 sums; gated, the second half
// of the columns is the up half of the first, so a lane holds gate and up of
// the same element.
template <class Step, bool ACOL, bool BCOL, int HM, int HN>
__global__ __launch_bounds__(512, HM == 128 ? 2 : 4) void product_kernel(ProductArgs a) {
  typedef Half<HM, ACOL> HA;
  typedef Half<HN, BCOL> HB;
  constexpr int TM = HM / 32, TN = HN / 64;  // 16 x 16 tiles of a wave in a quarter
  constexpr int kStage = 2 * HA::kBytes + 2 * HB::kBytes;
  // the stages, then rows of 2 HN sums with a pad of 16 bytes (Out)
  constexpr int kPitch = 2 * HN + 4;
  constexpr int kOut = HM * kPitch * 4;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage > kOut ? 2 * kStage : kOut];
  char *lds0 = lds, *lds1 = lds + kStage;

  const bool gated = a.e.gated;
  const int tile_n = gated ? HN : 2 * HN;
  const int tiles_m = (a.m + 2 * HM - 1) / (2 * HM), tiles_n = (a.n + tile_n - 1) / tile_n;
  // Consecutive workgroups go to different XCDs; each XCD takes a contiguous
  // run of tiles, in columns of 4 tile rows, so that the tiles it works on at
  // a time share rows and columns in its L2.
  const int tiles = tiles_m * tiles_n;
  int id = blockIdx.x;
  {
    const int xcd = id % 8, q = tiles / 8, r = tiles % 8;
    id = xcd * q + (xcd < r ? xcd : r) + id / 8;
  }
  constexpr int G = 4;
  const int group = id / (G * tiles_n), first = group * G, size = tiles_m - first < G ? tiles_m - first : G;
  const int tm = first + (id - group * G * tiles_n) % size, tn = (id - group * G * tiles_n) / size;
  const int m0 = tm * 2 * HM, n0 = tn * tile_n;

  const int w = threadIdx.x / 64, wm = w / 4, wn = w % 4;
  const int k0 = blockIdx.y * a.k_tiles_per_split;
  constexpr int kStep = 128 / Step::kBytes;  // elements of the contraction a stage
  const int all = (a.k + kStep - 1) / kStep;
  const int kn = all - k0 < a.k_tiles_per_split ? all - k0 : a.k_tiles_per_split;

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

  auto fetch = [&](int kt, char *stage) {
    const char *pa = (const char *)a.a + a0 + kt * a_step, *pb = (const char *)a.b + b0 + kt * b_step;
    const int64_t la = a.a_bytes - a0 - kt * a_step, lb = a.b_bytes - b0 - kt * b_step;
    const int left = (a.k - (k0 + kt) * kStep) * Step::kBytes;
    lds_char *s = (lds_char *)stage;
    HA::load(s, view(pa, la), va, HA::past(left));
    HA::load(s + HA::kBytes, view(pa + a_half, la - a_half), va, HA::past(left));
    HB::load(s + 2 * HA::kBytes, view(pb, lb), vb, HB::past(left));
    HB::load(s + 2 * HA::kBytes + HB::kBytes, view(pb + b_half, lb - b_half), vb, HB::past(left));
  };
  auto compute = [&](const char *stage) {
    const lds_char *s = (const lds_char *)stage;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      i32x4 fb[TN][2];
#pragma unroll
      for (int y = 0; y < TN; ++y) HB::read(s + 2 * HA::kBytes + j * HB::kBytes, wn * (HN / 4), y, fb[y]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < TM; ++x) {
          i32x4 fa[2];
          HA::read(s + i * HA::kBytes, wm * (HM / 2), x, fa);
#pragma unroll
          for (int y = 0; y < TN; ++y) acc[i][j][x][y] = Step::mma(fa, fb[y], acc[i][j][x][y]);
        }
    }
  };

  // A stage's loads are in flight while the other stage is worked on.  The
  // barrier at the top of a step stands between the reads of a stage and the
  // loads that write over it.
  if (kn > 0) fetch(0, lds0);
  for (int kt = 0; kt < kn; kt += 2) {
    __syncthreads();
    if (kt + 1 < kn) fetch(kt + 1, lds1);
    compute(lds0);
    if (kt + 1 < kn) {
      __syncthreads();
      if (kt + 2 < kn) fetch(kt + 2, lds0);
      compute(lds1);
    }
  }

  // Out: the sums of HM rows at a time go through LDS, so that a thread has 8
  // consecutive columns of a row and a row's stores are contiguous.  A lane's
  // four sums are 16 bytes; the pad keeps the 16 rows of a tile in different
  // banks.
  const int l = threadIdx.x % 64;
  float *out = (float *)lds;
  const int per = tile_n / 8;  // threads a row
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    __syncthreads();
#pragma unroll
    for (int x = 0; x < TM; ++x)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int y = 0; y < TN; ++y)
          *(f32x4 *)(out + (wm * (HM / 2) + x * 16 + (l & 15)) * kPitch + j * HN + wn * (HN / 4) + y * 16 +
                     (l >> 4) * 4) = Step::sums(acc[i][j][x][y]);
    __syncthreads();
#pragma unroll 1
    for (int at = threadIdx.x; at < HM * per; at += 512) {
      const int r = at / per, c = at % per * 8, m = m0 + i * HM + r, n = n0 + c;
      float v[8], u[8];
      load8<F32>(out + r * kPitch + c, v);
      if (gated) load8<F32>(out + r * kPitch + HN + c, u);
      if (a.splits > 1) {
        // partial sums: rows of ldp floats, the up half in their second half
        if (m < a.m && n < a.n) {
          float *p = a.partial + ((int64_t)blockIdx.y * a.m + m) * a.ldp + n;
          store8<F32>(p, v);
          if (gated) store8<F32>(p + a.ldp / 2, u);
        }
      } else {
        finish<8>(a.e, m, n, v, u);
      }
    }
  }
}

// The splits' partial sums, added in order, through the epilogue.
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
      for (int i = 0; i < 8; ++i) v[i] += x[i];
      if (e.gated) {
        load8<F32>(p + ldp / 2, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] += x[i];
      }
    }
    finish<8>(e, m, n, v, u);
  }
}

template <class Step, bool ACOL, bool BCOL>
hipError_t go(const ProductArgs &a, hipStream_t s) {
  const int64_t tile = a.tile == 0 ? 256 : 128, tile_n = a.e.gated ? tile / 2 : tile;
  const dim3 grid((unsigned)(((a.m + tile - 1) / tile) * ((a.n + tile_n - 1) / tile_n)), (unsigned)a.splits);
  if (a.tile == 0)
    product_kernel<Step, ACOL, BCOL, 128, 128><<<grid, 512, 0, s>>>(a);
  else
    product_kernel<Step, ACOL, BCOL, 64, 64><<<grid, 512, 0, s>>>(a);
  return hipGetLastError();
}

template <class Step>
hipError_t by_layout(const ProductArgs &a, hipStream_t s) {
  if (!a.a_by_col && !a.b_by_col) return go<Step, false, false>(a, s);
  if constexpr (Step::kBytes == 2) {
    if (!a.a_by_col) return go<Step, false, true>(a, s);
    if (a.b_by_col) return go<Step, true, true>(a, s);
  }
  return hipErrorInvalidValue;  // not planned: only 16-bit gradients run over rows
}

}  // namespace

hipError_t launch_product(const ProductArgs &a, hipStream_t s) {
  if (a.dtype == HF_BF16) return by_layout<StepBF16>(a, s);
  if (a.dtype == HF_F16) return by_layout<StepF16>(a, s);
  if (a.dtype == HF_F8E4M3)
    return f8_wide(a.e.out_dtype, a.k) ? by_layout<StepF8Wide>(a, s) : by_layout<StepF8>(a, s);
  return by_layout<StepS8>(a, s);
}

hipError_t launch_product_fold(const float *partial, int splits, int64_t ldp, const Epilogue &e, hipStream_t s) {
  const dim3 grid((unsigned)((e.n + 2047) / 2048), (unsigned)(e.m < 65535 ? e.m : 65535));
  product_fold_kernel<<<grid, 256, 0, s>>>(partial, splits, ldp, e);
  return hipGetLastError();
}

}  // namespace hf
