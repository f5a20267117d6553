// rows.hip -- the operators that are bound by memory: the root-mean-square
// norm and its gradient, dropout, the activation's gradient, and the copies
// that lay out an operand.
#include "device.h"

namespace hf {
namespace {

// Where element i of a thread's vector j lies in a row.  VEC: eight
// consecutive elements a thread, so that each access is 16 bytes.  Otherwise
// (rows that are not 16-byte aligned, or a length that is no multiple of 8)
// consecutive threads take consecutive elements, one by one: RmsNorm of 4099 x
// 4097 bf16 with a residual takes 117 us, of 4099 x 4096 21.
template <int T, bool VEC>
__device__ __forceinline__ int column(int t, int j, int i) {
  return VEC ? (j * T + t) * 8 + i : (j * 8 + i) * T + t;
}

// One vector of a row; elements past the row's end are 0.
template <class E, int T, bool VEC>
__device__ __forceinline__ void load_row(const typename E::Store *row, int t, int j, int cols, float (&v)[8]) {
  if (VEC) {
    const int c = column<T, VEC>(t, j, 0);
    if (c < cols) {
      load8<E>(row + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<T, VEC>(t, j, i);
      v[i] = c < cols ? E::load(row[c]) : 0.f;
    }
  }
}

template <class E, int T, bool VEC>
__device__ __forceinline__ void store_row(typename E::Store *row, int t, int j, int cols, const float (&v)[8]) {
  if (VEC) {
    const int c = column<T, VEC>(t, j, 0);
    if (c < cols) store8<E>(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<T, VEC>(t, j, i);
      if (c < cols) row[c] = E::store(v[i]);
    }
  }
}

// The same in two parts: the bits as they come from memory, asked for a row
// ahead, and their values.
template <class E, int T, bool VEC>
struct Raw {
  u32x4 v[E::kBytes / 2];        // VEC
  typename E::Store one[VEC ? 1 : 8];
  __device__ __forceinline__ void load(const typename E::Store *row, int t, int j, int cols) {
    if (VEC) {
      const int c = column<T, VEC>(t, j, 0);
#pragma unroll
      for (int i = 0; i < E::kBytes / 2; ++i) v[i] = c < cols ? ((const u32x4 *)(row + c))[i] : u32x4{0, 0, 0, 0};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = column<T, VEC>(t, j, i);
        one[VEC ? 0 : i] = c < cols ? row[c] : (typename E::Store)0;
      }
    }
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!VEC) f[i] = E::load(one[VEC ? 0 : i]);
      else if (E::kBytes == 4) f[i] = __uint_as_float(v[i / 4 % (E::kBytes / 2)][i % 4]);
      else f[i] = E::load((typename E::Store)(uint16_t)(v[0][i / 2] >> (i % 2 * 16)));
    }
  }
};

// The weight, in f32 or in the rows' type.
template <class E, int T, bool VEC>
__device__ __forceinline__ void load_weight(const void *w, bool wide, int t, int j, int cols, float (&v)[8]) {
  if (wide)
    load_row<F32, T, VEC>((const float *)w, t, j, cols, v);
  else
    load_row<E, T, VEC>((const typename E::Store *)w, t, j, cols, v);
}

// One step of a wave's reduction: the value of the lane that CTRL (a data
// parallel primitive's control) names, 0 where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, true);
}

// Over a wave: within rows of 16 lanes by shifts of 1, 2, 4 and 8, then row 0
// into 1 and 2 into 3, then the first half into the second; lane 63 has it
// all.  0 is neutral to both operations.
__device__ __forceinline__ float wave_sum(float v) {
  v += __uint_as_float(moved<0x111, 0xf>(__float_as_uint(v)));
  v += __uint_as_float(moved<0x112, 0xf>(__float_as_uint(v)));
  v += __uint_as_float(moved<0x114, 0xf>(__float_as_uint(v)));
  v += __uint_as_float(moved<0x118, 0xf>(__float_as_uint(v)));
  v += __uint_as_float(moved<0x142, 0xa>(__float_as_uint(v)));
  v += __uint_as_float(moved<0x143, 0xc>(__float_as_uint(v)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, moved<0x111, 0xf>(v));
  v = max(v, moved<0x112, 0xf>(v));
  v = max(v, moved<0x114, 0xf>(v));
  v = max(v, moved<0x118, 0xf>(v));
  v = max(v, moved<0x142, 0xa>(v));
  v = max(v, moved<0x143, 0xc>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Over the T threads of a row.  `slots`: T/64 floats of this call's own (no
// second barrier is needed before the next call, which takes other slots).
template <int T>
__device__ __forceinline__ float row_sum(float v, float *slots) {
  v = wave_sum(v);
  if (T == 64) return v;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x / 64] = v;
  __syncthreads();
  v = slots[0];
#pragma unroll
  for (int i = 1; i < T / 64; ++i) v += slots[i];
  return v;
}

// The largest magnitude of a row.  Magnitudes are compared as the integers
// that their bits are: the same order, and a NaN is above infinity, so a row
// that holds one gets it.
template <int T>
__device__ __forceinline__ float row_top(uint32_t v, uint32_t *slots) {
  v = wave_max(v);
  if (T != 64) {
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x / 64] = v;
    __syncthreads();
    v = slots[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) v = max(v, slots[i]);
  }
  return __uint_as_float(v);
}

// y / scale, rounded once, for every element of a row: r is the rounded
// reciprocal, q = y r is within two ulps of the quotient and the remainder
// y - q scale, exact in one fma, corrects it.  Where r or the remainder
// could overflow (scales near the ends of the range, infinite or NaN) the
// division itself is taken.
struct Quotient {
  float s, r;
  bool slow;
  __device__ __forceinline__ explicit Quotient(float scale) : s(scale), r(1.0f / scale), slow(!(scale > 1e-30f && scale < 1e30f)) {}
  __device__ __forceinline__ float operator()(float y) const {
    if (slow) return s == 0.f ? 0.f : y / s;
    const float q = y * r;
    return __builtin_fmaf(__builtin_fmaf(-q, s, y), r, q);
  }
};

// Eight quotients as e4m3 or s8, each rounded to nearest even and clamped.
// NaN stays NaN in e4m3 and is 0 in s8, which has none.
template <int OUT>
__device__ __forceinline__ u32x2 pack8(const float (&v)[8]) {
  u32x2 r;
  if (OUT == HF_F8E4M3) {
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = v[i] != v[i] ? v[i] : __builtin_fminf(__builtin_fmaxf(v[i], -448.f), 448.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * h], c[4 * h + 1], 0, false);
      r[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * h + 2], c[4 * h + 3], w, true);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = v[4 * h + i];
        const int q = f != f ? 0 : (int)__builtin_rintf(__builtin_fminf(__builtin_fmaxf(f, -127.f), 127.f));
        w |= (uint32_t)(q & 0xff) << (8 * i);
      }
      r[h] = w;
    }
  }
  return r;
}

template <int OUT, int T, bool VEC>
__device__ __forceinline__ void store_row8(uint8_t *row, int t, int j, int cols, const float (&v)[8]) {
  const u32x2 p = pack8<OUT>(v);
  if (VEC) {
    const int c = column<T, VEC>(t, j, 0);
    if (c < cols) __builtin_nontemporal_store(p, (u32x2 *)(row + c));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<T, VEC>(t, j, i);
      if (c < cols) row[c] = (uint8_t)(p[i / 4] >> (8 * (i % 4)));
    }
  }
}

// RmsNorm.  h = x + residual in f32; rstd = (mean h^2 + eps)^-1/2;
// y = h rstd weight, rounded once; in 8 bits, scale = max|y| / Q of the row
// and q = y / scale.  The row stays in registers between its sum, its largest
// magnitude and its store, so x and residual are read once: the kernel is
// bound by memory (4099 x 4096 bf16 to e4m3 with a residual: 20 us, 118 MB,
// 5.9 TB/s; a single such row 4.2 us, a launch and two reductions).  T threads
// a row; a row of 1024 elements or fewer is one
// wave's, and a workgroup then takes four.
// NV = 0: rows too long for registers, read again for each of the steps.
template <class E, int OUT, int T, int NV, bool VEC>
__global__ __launch_bounds__(T == 64 ? 256 : T) void norm_kernel(NormArgs a) {
  __shared__ float slots[T == 64 ? 1 : T / 64];
  __shared__ uint32_t top_slots[T == 64 ? 1 : T / 64];
  __shared__ float far_slots[T == 64 ? 1 : T / 64];
  __shared__ uint32_t far_top_slots[T == 64 ? 1 : T / 64];
  constexpr int ROWS = T == 64 ? 4 : 1;
  const int t = threadIdx.x % T;
  const int64_t row = block_number<T * ROWS>(blockIdx.x, blockIdx.y) * ROWS + threadIdx.x / T;
  if (row >= a.rows) return;  // whole waves, and no barrier follows where ROWS > 1
  typedef typename E::Store S;
  const S *x = (const S *)a.x + row * a.ldx;
  const S *r = a.residual ? (const S *)a.residual + row * a.ldr : nullptr;
  S *stream = a.stream ? (S *)a.stream + row * a.lds : nullptr;
  const int n = NV ? NV : (a.cols + 8 * T - 1) / (8 * T);
  float keep[NV ? NV : 1][8];
  float sum = 0.f;
  auto input = [&](int j, float (&h)[8]) {
    load_row<E, T, VEC>(x, t, j, a.cols, h);
    if (r) {
      float o[8];
      load_row<E, T, VEC>(r, t, j, a.cols, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] += o[i];
    }
  };
  auto take = [&](int j, float (&h)[8]) {
    if (stream) store_row<E, T, VEC>(stream, t, j, a.cols, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(h[i], h[i], sum);
  };
  // The weight is asked for together with the row, not after its sum: with a
  // single row the two latencies would add up.
  const bool wide = a.weight_dtype == HF_F32;
  float w[NV ? NV : 1][8];
  if (NV) {
#pragma unroll
    for (int j = 0; j < NV; ++j) input(j, keep[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) load_weight<E, T, VEC>(a.weight, wide, t, j, a.cols, w[j]);
#pragma unroll
    for (int j = 0; j < NV; ++j) take(j, keep[j]);
  } else {
    for (int j = 0; j < n; ++j) {
      input(j, keep[0]);
      take(j, keep[0]);
    }
  }
  sum = row_sum<T>(sum, slots);
  const float m = sum / (float)a.cols + a.eps;
  // v_rsq is within one ulp; the step brings it to half an ulp and a bit
  float rstd = __builtin_amdgcn_rsqf(m);
  if (m > 1e-30f && m < 1e37f) {
    const float e = __builtin_fmaf(-m * rstd, rstd, 1.f);
    rstd = __builtin_fmaf(0.5f * rstd, e, rstd);
  } else {
    // The squares may have left the range of 32 bits though rstd is in it:
    // once more, with the row scaled by a power of two that brings its
    // largest magnitude (or sqrt(eps), where that is larger) to 1 .. 2.
    uint32_t top = 0;
    auto widen = [&](const float (&h)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(h[i]) & 0x7fffffffu);
    };
    if (NV) {
#pragma unroll
      for (int j = 0; j < NV; ++j) widen(keep[j]);
    } else {
      for (int j = 0; j < n; ++j) {
        input(j, keep[0]);
        widen(keep[0]);
      }
    }
    float root = a.root;
    const float largest = __builtin_fmaxf(row_top<T>(top, far_top_slots), root);
    int power = 0;
    (void)frexpf(largest, &power);
    const bool far = largest > 0.f && largest < __builtin_inff();
    float again = 0.f;
    auto add = [&](const float (&h)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = ldexpf(h[i], 1 - power);
        again = __builtin_fmaf(v, v, again);
      }
    };
    if (NV) {
#pragma unroll
      for (int j = 0; j < NV; ++j) add(keep[j]);
    } else {
      for (int j = 0; j < n; ++j) {
        input(j, keep[0]);
        add(keep[0]);
      }
    }
    again = row_sum<T>(again, far_slots);
    root = ldexpf(root, 1 - power);
    rstd = far ? ldexpf(1.0f / sqrtf(again / (float)a.cols + root * root), 1 - power) : 1.0f / sqrtf(m);
  }
  if (a.rstd && t == 0) a.rstd[row] = rstd;
  auto scaled = [&](int j, float (&h)[8]) {
    if (!NV) load_weight<E, T, VEC>(a.weight, wide, t, j, a.cols, w[0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = h[i] * rstd * w[NV ? j : 0][i];
  };
  if (OUT < 0) {
    S *y = (S *)a.y + row * a.ldy;
    if (NV) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        scaled(j, keep[j]);
        store_row<E, T, VEC>(y, t, j, a.cols, keep[j]);
      }
    } else {
      for (int j = 0; j < n; ++j) {
        input(j, keep[0]);
        scaled(j, keep[0]);
        store_row<E, T, VEC>(y, t, j, a.cols, keep[0]);
      }
    }
  } else {
    uint32_t top = 0;
    auto widen = [&](const float (&h)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(h[i]) & 0x7fffffffu);
    };
    if (NV) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        scaled(j, keep[j]);
        widen(keep[j]);
      }
    } else {
      for (int j = 0; j < n; ++j) {
        input(j, keep[0]);
        scaled(j, keep[0]);
        widen(keep[0]);
      }
    }
    const float scale = row_top<T>(top, top_slots) / (OUT == HF_F8E4M3 ? 448.f : 127.f);
    if (t == 0) a.scale[row] = scale;
    const Quotient q(scale);
    uint8_t *y = (uint8_t *)a.y + row * a.ldy;
    auto out = [&](int j, float (&h)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = q(h[i]);
      store_row8<OUT, T, VEC>(y, t, j, a.cols, h);
    };
    if (NV) {
#pragma unroll
      for (int j = 0; j < NV; ++j) out(j, keep[j]);
    } else {
      for (int j = 0; j < n; ++j) {
        input(j, keep[0]);
        scaled(j, keep[0]);
        out(j, keep[0]);
      }
    }
  }
}

// RmsNormGrad.  With xh = h rstd and g = dy weight,
//   dx = (g - xh mean(g xh)) rstd + dstream,   dweight = sum over rows dy xh.
// A workgroup (one wave in rows of 512 or fewer) takes every groups-th row
// and keeps its columns' dweight in registers over all of them, so dweight
// costs no memory traffic but one partial row a group, written and read again
// by fold_kernel, which adds the groups in a fixed order.  (Up to
// norm_grad_groups' number of rows a group is one row, and those partial rows
// in f32 are as many bytes as the operator's own: 1024 x 4096 bf16 19 us, where
// 34 MB take 7.)  Bound by memory: dy, h and dstream read once, dx written once
// (16384 x 4096 bf16 with dstream: 113 us, 4.7 TB/s, the fold's 7 us in it).  A row's mean stands between its loads and its stores, so the
// next row is asked for before that (189 us without).
template <class E, int T, int NV, bool VEC>
__global__ __launch_bounds__(T == 64 ? 256 : T) void norm_grad_kernel(NormGradArgs a) {
  __shared__ float slots[2][T == 64 ? 1 : T / 64];
  constexpr int PER = T == 64 ? 4 : 1;
  const int t = threadIdx.x % T;
  const int group = blockIdx.x * PER + threadIdx.x / T;
  if (group >= a.groups) return;
  typedef typename E::Store S;
  const bool wide = a.weight_dtype == HF_F32, stream = a.dstream != nullptr;
  float *partial = a.partial + (int64_t)group * a.cols;
  float dw[NV][8], w[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_weight<E, T, VEC>(a.weight, wide, t, j, a.cols, w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  }
  Raw<E, T, VEC> rh[NV], rg[NV], rs[NV];
  float next_rstd = 0.f;
  auto ask = [&](int64_t row) {
    next_rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < NV; ++j) rh[j].load((const S *)a.h + row * a.ldh, t, j, a.cols);
#pragma unroll
    for (int j = 0; j < NV; ++j) rg[j].load((const S *)a.dy + row * a.lddy, t, j, a.cols);
    if (stream) {
#pragma unroll
      for (int j = 0; j < NV; ++j) rs[j].load((const S *)a.dstream + row * a.ldds, t, j, a.cols);
    }
  };
  if (group < a.rows) ask(group);
  int turn = 0;
  for (int64_t row = group; row < a.rows; row += a.groups, turn ^= 1) {
    const float rstd = next_rstd;
    float xh[NV][8], g[NV][8], o[NV][8];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      rh[j].values(xh[j]);
      rg[j].values(g[j]);
      if (stream) rs[j].values(o[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[j][i] *= rstd;
        dw[j][i] = __builtin_fmaf(g[j][i], xh[j][i], dw[j][i]);
        g[j][i] *= w[j][i];
        dot = __builtin_fmaf(g[j][i], xh[j][i], dot);
      }
    }
    if (row + a.groups < a.rows) ask(row + a.groups);
    // the slots change with each row: a thread may be one row ahead of
    // another, never two, as each row has a barrier
    const float mean = row_sum<T>(dot, slots[turn]) / (float)a.cols;
    S *dx = (S *)a.dx + row * a.lddx;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[j][i] = (g[j][i] - xh[j][i] * mean) * rstd;
        if (stream) g[j][i] += o[j][i];
      }
      store_row<E, T, VEC>(dx, t, j, a.cols, g[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) store_row<F32, T, VEC>(partial, t, j, a.cols, dw[j]);
}

// The same for rows that do not fit the registers: each is read twice, and
// dweight's partial row is kept in memory (it is this workgroup's alone).
template <class E, bool VEC>
__global__ __launch_bounds__(1024) void norm_grad_long_kernel(NormGradArgs a) {
  constexpr int T = 1024;
  __shared__ float slots[2][T / 64];
  const int t = threadIdx.x, group = blockIdx.x;
  typedef typename E::Store S;
  const bool wide = a.weight_dtype == HF_F32;
  const int n = (a.cols + 8 * T - 1) / (8 * T);
  float *partial = a.partial + (int64_t)group * a.cols;
  for (int j = 0; j < n; ++j) {
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    store_row<F32, T, VEC>(partial, t, j, a.cols, z);
  }
  int turn = 0;
  for (int64_t row = group; row < a.rows; row += a.groups, turn ^= 1) {
    const S *dy = (const S *)a.dy + row * a.lddy, *h = (const S *)a.h + row * a.ldh;
    const float rstd = a.rstd[row];
    float xh[8], g[8], w[8], o[8], dot = 0.f;
    auto take = [&](int j) {
      load_row<E, T, VEC>(h, t, j, a.cols, xh);
      load_row<E, T, VEC>(dy, t, j, a.cols, g);
      load_weight<E, T, VEC>(a.weight, wide, t, j, a.cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) xh[i] *= rstd;
    };
    for (int j = 0; j < n; ++j) {
      take(j);
      load_row<F32, T, VEC>(partial, t, j, a.cols, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = __builtin_fmaf(g[i], xh[i], o[i]);
        dot = __builtin_fmaf(g[i] * w[i], xh[i], dot);
      }
      store_row<F32, T, VEC>(partial, t, j, a.cols, o);
    }
    const float mean = row_sum<T>(dot, slots[turn]) / (float)a.cols;
    for (int j = 0; j < n; ++j) {
      take(j);
      if (a.dstream) load_row<E, T, VEC>((const S *)a.dstream + row * a.ldds, t, j, a.cols, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = (g[i] * w[i] - xh[i] * mean) * rstd;
        if (a.dstream) g[i] += o[i];
      }
      store_row<E, T, VEC>((S *)a.dx + row * a.lddx, t, j, a.cols, g);
    }
  }
}

// out[c] = sum over g of partial[g][c], always in the same order: 16 columns
// (64 bytes of a row) a workgroup, 64 threads a column, so that a few thousand
// columns already fill the chip (1024 x 4096 partial sums: 7 us; with 8 threads
// a column 33 us).
__global__ __launch_bounds__(1024) void fold_kernel(const float *partial, int groups, int64_t cols, float *out) {
  __shared__ float part[64][17];
  const int64_t c = block_number<1024>(blockIdx.x, blockIdx.y) * 16 + threadIdx.x % 16;
  const int lane = threadIdx.x / 16;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int g = lane; g < groups; g += 64) s += partial[(int64_t)g * cols + c];
  }
  part[lane][threadIdx.x % 16] = s;
#pragma unroll
  for (int half = 32; half; half /= 2) {
    __syncthreads();
    if (lane < half) part[lane][threadIdx.x % 16] += part[lane + half][threadIdx.x % 16];
  }
  if (lane == 0 && c < cols) out[c] = part[0][threadIdx.x];
}

// Dropout.  Element i of the row-major array takes 16 bits of the generator's
// call number offset + i / 8: word (i % 8) / 2, the low half for even i.  It
// is kept where they are >= cut = p 65536, so the kept share is exactly
// 1 - cut / 65536 and scale its exact inverse.  One call serves one 16-byte
// vector; nothing of the mask is stored, and the backward pass makes it again.
// The generator's 20 products a vector hide behind the memory: 16384 x 4096
// bf16 with a residual takes 69 us, 5.8 TB/s.
template <class E, bool VEC>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a) {
  typedef typename E::Store S;
  const uint64_t key = (uint64_t)a.state[0], offset = (uint64_t)a.state[1];
  const int64_t total = a.rows * a.cols, vectors = (total + 7) / 8;
  const int64_t v = block_number<256>(blockIdx.x, blockIdx.y) * 256 + threadIdx.x;
  if (v >= vectors) return;
  const u32x4 word = philox(offset + (uint64_t)v, key);
  // arrays without gaps come as one row
  int64_t row = 0, col = v * 8;
  if (a.rows > 1) {
    row = (v * 8) / a.cols;
    col = v * 8 - row * a.cols;
  }
  auto kept = [&](int i, float x) {
    const uint32_t bits = i % 2 ? word[i / 2] >> 16 : word[i / 2] & 0xffff;
    return bits >= a.cut ? x * a.scale : 0.f;
  };
  if (VEC && v * 8 + 8 <= total) {
    float x[8], r[8];
    load8<E>((const S *)a.x + row * a.ldx + col, x);
    if (a.residual) load8<E>((const S *)a.residual + row * a.ldr + col, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = kept(i, x[i]) + (a.residual ? r[i] : 0.f);
    store8<E>((S *)a.y + row * a.ldy + col, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (v * 8 + i < total) {
        float x = kept(i, E::load(((const S *)a.x)[row * a.ldx + col]));
        if (a.residual) x += E::load(((const S *)a.residual)[row * a.ldr + col]);
        ((S *)a.y)[row * a.ldy + col] = E::store(x);
        if (++col == a.cols) col = 0, ++row;
      }
    }
  }
}

// dz = dd act'(z) in the operands' type, as the matrix instructions take it (a
// second 16-bit part for the rest would double both products), and the column
// sums' partials from the values before that rounding.  In f16 dz has that
// type's range: a value from 65520 on is an infinity, one below 2^-25 zero.  256 threads take 8 columns each of every
// groups-th row.  Columns n .. lddz-1 of dz are padding and become 0, so that
// a product over them adds nothing.  Bound by memory: 8192 x 16384 bf16 with
// GELU and column sums 162 us, 5.0 TB/s.
template <class E, bool GATED, bool VEC>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradArgs a) {
  typedef typename E::Store S;
  const int64_t c0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  // GATED: both halves' columns lie side by side, so padding follows 2n
  const int64_t width = GATED ? (int64_t)a.n : (a.dz ? a.lddz : (int64_t)a.n);
  if (c0 >= width) return;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t row = blockIdx.y; row < a.m; row += a.groups) {
    const S *dd = (const S *)a.dd + row * a.lddd;
    const S *z = a.z ? (const S *)a.z + row * a.ldz : nullptr;
    S *dz = a.dz ? (S *)a.dz + row * a.lddz : nullptr;
    float d[8], g[8], u[8];
    auto get = [&](const S *p, float (&v)[8]) {
      if (VEC) {
        load8<E>(p + c0, v);
      } else if (c0 + 8 <= a.n) {
        load_any<E, 8>(p + c0, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + i < a.n ? E::load(p[c0 + i]) : 0.f;
      }
    };
    auto set = [&](S *p, int64_t extent, const float (&v)[8]) {
      if (VEC) {
        store8<E>(p + c0, v);
      } else if (c0 + 8 <= extent) {
        store_any<E, 8>(p + c0, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c0 + i < extent) p[c0 + i] = E::store(v[i]);
      }
    };
    get(dd, d);
    if (GATED) {
      get(z, g);
      get(z + a.n, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f, df;
        f = act_both(a.act, g[i], &df);
        g[i] = d[i] * u[i] * df;
        u[i] = d[i] * f;
      }
      set(dz, a.n, g);
      set(dz + a.n, a.n, u);
      if (c0 + 8 >= a.n)
        for (int64_t c = 2 * (int64_t)a.n; c < a.lddz; ++c) dz[c] = E::store(0.f);
    } else {
      if (z) {
        get(z, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float df;
          (void)act_both(a.act, g[i], &df);
          d[i] *= df;
        }
      }
      if (dz) set(dz, a.lddz, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += d[i];
    }
  }
  if (!GATED && a.partial) {
    float *p = a.partial + (int64_t)blockIdx.y * a.n;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < a.n) p[c0 + i] = sum[i];
  }
}

// Rows of any alignment into rows that start on 16 bytes, the tail zero: 16
// bytes of a row a thread, in one unaligned load where the row has them all.
// 11252 + 11252 rows of 3643 s8 take 28 us, 5.8 TB/s.
__global__ __launch_bounds__(256) void pack_kernel(const uint8_t *src, int64_t ld_src, uint8_t *dst, int64_t ld_dst,
                                                   int64_t rows, int64_t bytes) {
  const int64_t c = ((int64_t)blockIdx.x * 64 + threadIdx.x % 64) * 16;
  if (c >= ld_dst) return;
  const int valid = bytes - c < 16 ? (int)(bytes - c) : 16;
  for (int64_t r = (int64_t)blockIdx.y * 4 + threadIdx.x / 64; r < rows; r += (int64_t)gridDim.y * 4) {
    const uint8_t *from = src + r * ld_src + c;
    u32x4 v = {0, 0, 0, 0};
    if (valid == 16) {
      __builtin_memcpy(&v, from, 16);
    } else if (bytes >= 16) {
      // the row's last 16 bytes, the first of them shifted out
      u32x4 w;
      __builtin_memcpy(&w, from + valid - 16, 16);
      const int words = (16 - valid) / 4;
      uint32_t t[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        t[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + words == j) t[i] = w[j];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_alignbyte(t[i + 1], t[i], (uint32_t)(16 - valid) & 3);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < valid) v[i / 4] |= (uint32_t)from[i] << (i % 4 * 8);
    }
    *(u32x4 *)(dst + r * ld_dst + c) = v;
  }
}

template <class E, int OUT, int T, int NV>
hipError_t norm_go(const NormArgs &a, hipStream_t s) {
  constexpr int per = T == 64 ? 4 : 1, block = T * per;
  return launch(a.vec ? norm_kernel<E, OUT, T, NV, true> : norm_kernel<E, OUT, T, NV, false>,
                grid_of<block>((a.rows + per - 1) / per), block, s, a);
}

template <class E, int OUT>
hipError_t norm_by_length(const NormArgs &a, hipStream_t s) {
  if (a.cols <= 512) return norm_go<E, OUT, 64, 1>(a, s);
  if (a.cols <= 1024) return norm_go<E, OUT, 64, 2>(a, s);
  if (a.cols <= 2048) return norm_go<E, OUT, 256, 1>(a, s);
  if (a.cols <= 4096) return norm_go<E, OUT, 256, 2>(a, s);
  if (a.cols <= 8192) return norm_go<E, OUT, 256, 4>(a, s);
  if (a.cols <= 16384) return norm_go<E, OUT, 1024, 2>(a, s);
  if (a.cols <= 32768) return norm_go<E, OUT, 1024, 4>(a, s);
  return norm_go<E, OUT, 1024, 0>(a, s);
}

template <class E>
hipError_t norm_by_out(const NormArgs &a, hipStream_t s) {
  if (a.out_dtype == HF_F8E4M3) return norm_by_length<E, HF_F8E4M3>(a, s);
  if (a.out_dtype == HF_S8) return norm_by_length<E, HF_S8>(a, s);
  return norm_by_length<E, -1>(a, s);
}

template <class E, int T, int NV>
hipError_t norm_grad_go(const NormGradArgs &a, hipStream_t s) {
  const int per = T == 64 ? 4 : 1;
  const dim3 grid((unsigned)((a.groups + per - 1) / per));
  return launch(a.vec ? norm_grad_kernel<E, T, NV, true> : norm_grad_kernel<E, T, NV, false>, grid,
                T == 64 ? 256 : T, s, a);
}

// Rows of 8193 to 16384 columns stay in registers where those suffice for
// them: in 16 bits, with whole vectors (2000 x 16384 bf16: 64 us, read twice
// 121 us).
template <class E>
hipError_t norm_grad_by_length(const NormGradArgs &a, hipStream_t s) {
  if (a.cols <= 512) return norm_grad_go<E, 64, 1>(a, s);
  if (a.cols <= 2048) return norm_grad_go<E, 256, 1>(a, s);
  if (a.cols <= 4096) return norm_grad_go<E, 256, 2>(a, s);
  if (a.cols <= 8192) return norm_grad_go<E, 1024, 1>(a, s);
  if constexpr (E::kBytes == 2) {
    if (a.cols <= 16384 && a.vec) return launch(norm_grad_kernel<E, 512, 4, true>, dim3((unsigned)a.groups), 512, s, a);
  }
  return launch(a.vec ? norm_grad_long_kernel<E, true> : norm_grad_long_kernel<E, false>, dim3((unsigned)a.groups), 1024,
                s, a);
}

template <class E>
hipError_t dropout_go(const DropoutArgs &a, hipStream_t s) {
  const int64_t vectors = (a.rows * a.cols + 7) / 8;
  return launch(a.vec ? dropout_kernel<E, true> : dropout_kernel<E, false>, grid_of<256>((vectors + 255) / 256), 256, s, a);
}

template <class E>
hipError_t act_grad_go(const ActGradArgs &a, hipStream_t s) {
  const int64_t width = a.gated || !a.dz ? (int64_t)a.n : a.lddz;
  const dim3 grid((unsigned)((width + 2047) / 2048), (unsigned)a.groups);
  if (a.gated) return launch(a.vec ? act_grad_kernel<E, true, true> : act_grad_kernel<E, true, false>, grid, 256, s, a);
  return launch(a.vec ? act_grad_kernel<E, false, true> : act_grad_kernel<E, false, false>, grid, 256, s, a);
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, hipStream_t s) {
  if (a.dtype == HF_BF16) return norm_by_out<BF16>(a, s);
  if (a.dtype == HF_F16) return norm_by_out<F16>(a, s);
  return norm_by_out<F32>(a, s);
}

int norm_grad_groups(int64_t rows, int64_t cols) {
  // enough workgroups for the memory to be kept busy (4 of 256 threads a
  // compute unit, 2 of 1024, 1 of 512), and no more partial rows than that
  const int64_t most = cols <= 512 ? 4096 : cols <= 4096 ? 1024 : cols <= 8192 ? 512 : 256;
  return (int)(rows < 1 ? 1 : rows < most ? rows : most);
}

hipError_t launch_norm_grad(const NormGradArgs &a, hipStream_t s) {
  const hipError_t e = a.dtype == HF_BF16  ? norm_grad_by_length<BF16>(a, s)
                       : a.dtype == HF_F16 ? norm_grad_by_length<F16>(a, s)
                                           : norm_grad_by_length<F32>(a, s);
  return e != hipSuccess ? e : launch_column_fold(a.partial, a.groups, a.cols, a.dweight, s);
}

hipError_t launch_column_fold(const float *partial, int groups, int64_t cols, float *out, hipStream_t s) {
  return launch(fold_kernel, grid_of<1024>((cols + 15) / 16), 1024, s, partial, groups, cols, out);
}

hipError_t launch_dropout(const DropoutArgs &a, hipStream_t s) {
  if (a.dtype == HF_BF16) return dropout_go<BF16>(a, s);
  if (a.dtype == HF_F16) return dropout_go<F16>(a, s);
  return dropout_go<F32>(a, s);
}

int act_grad_groups(int64_t m, int64_t n) {
  // 4096 workgroups in all, at most 512 partial rows
  const int64_t wide = n > 0 ? (n + 2047) / 2048 : 1;
  const int64_t most = wide >= 64 ? 64 : wide >= 8 ? 4096 / wide : 512;
  return (int)(m < 1 ? 1 : m < most ? m : most);
}

hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t s) {
  return a.dtype == HF_BF16 ? act_grad_go<BF16>(a, s) : act_grad_go<F16>(a, s);
}

hipError_t launch_pack(const void *src, int64_t ld_src, void *dst, int64_t ld_dst, int64_t rows, int64_t bytes,
                       hipStream_t s) {
  const int64_t fours = (rows + 3) / 4;
  const dim3 grid((unsigned)((ld_dst / 16 + 63) / 64), (unsigned)(fours < 65535 ? fours : 65535));
  return launch(pack_kernel, grid, 256, s, (const uint8_t *)src, ld_src, (uint8_t *)dst, ld_dst, rows, bytes);
}

}  // namespace hf
