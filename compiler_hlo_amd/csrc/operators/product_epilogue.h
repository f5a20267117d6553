// product_epilogue.h -- what happens to the sums of a product on their way
// out: scales, bias, activation, the gate, the residual and the rounding.
#pragma once

#include "device.h"

namespace hf {

// W (4 or 8) consecutive elements, those below `left`.
template <class E, int W>
__device__ __forceinline__ void get(const void *base, int64_t at, int left, bool vec, float (&v)[W]) {
  const typename E::Store *p = (const typename E::Store *)base + at;
  if (vec && W == 8) {
    load8<E>(p, *(float(*)[8])v);
  } else if (vec) {
    const f32x4 x = load4<E>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i];
  } else if (left >= W) {
    load_any<E, W>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = i < left ? E::load(p[i]) : 0.f;
  }
}

template <class E, int W>
__device__ __forceinline__ void put(void *base, int64_t at, int left, bool vec, const float (&v)[W]) {
  typename E::Store *p = (typename E::Store *)base + at;
  if (vec && W == 8) {
    store8<E>(p, *(const float(*)[8])v);
  } else if (vec) {
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[i];
    store4<E>(p, x);
  } else if (left >= W) {
    store_any<E, W>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < left) p[i] = E::store(v[i]);
  }
}

template <class E, int W>
__device__ __forceinline__ void finish_as(const Epilogue &e, int m, int n, float (&v)[W], float (&up)[W]) {
  const int left = e.n - n;
  const bool vec = e.vec && left >= W;
  if (e.a_scale) {
    // from the left: the two scales' product may leave f32's range where the
    // result is in it
    const float s = e.a_scale[m];
    float c[W];
    get<F32, W>(e.b_scale, n, left, vec, c);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = v[i] * s * c[i];
    if (e.gated) {
      get<F32, W>(e.b_scale, (int64_t)e.n + n, left, vec && e.n % 4 == 0, c);
#pragma unroll
      for (int i = 0; i < W; ++i) up[i] = up[i] * s * c[i];
    }
  }
  if (e.bias) {
    float c[W];
    get<E, W>(e.bias, n, left, vec, c);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += c[i];
  }
  if (e.z) {
    put<E, W>(e.z, m * e.ldz + n, left, vec, v);
    if (e.gated) put<E, W>(e.z, m * e.ldz + e.n + n, left, vec, up);
  }
  if (e.act != HF_ACTIVATION_NONE) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = act_value<E::kBytes == 4>(e.act, v[i]);
  }
  if (e.gated) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= up[i];
  }
  if (e.residual) {
    float c[W];
    get<E, W>(e.residual, m * e.ldr + n, left, vec, c);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += c[i];
  }
  put<E, W>(e.d, m * e.ldd + n, left, vec, v);
}

// Columns n .. n+W-1 of row m (those below e.n); `up`: the up half's sums
// where the product is gated.  Everything is in f32 until the one rounding of
// each result.
template <int W>
__device__ __forceinline__ void finish(const Epilogue &e, int m, int n, float (&v)[W], float (&up)[W]) {
  if (m >= e.m || n >= e.n) return;
  if (e.out_dtype == HF_BF16) finish_as<BF16, W>(e, m, n, v, up);
  else if (e.out_dtype == HF_F16) finish_as<F16, W>(e, m, n, v, up);
  else finish_as<F32, W>(e, m, n, v, up);
}

// One step of the contraction over 128 bytes of both operands for a 16 x 16
// tile of the product.  (The 32 x 32 instructions read fewer registers for a
// multiplication, took 6% fewer cycles and drew so much more power that the
// clock fell by 10%: 1175 us against 1096 us for 8191 x 22528 x 4096.)  The operands are given in the order (b, a), so that a
// lane's four sums are four consecutive columns of one row of d: lane l holds
// row l % 16, columns (l / 16) * 4 + 0..3.  Which bytes of the 128 a lane
// holds is the same for a and b, and their order does not matter to a sum.
struct StepBF16 {
  typedef f32x4 Acc;
  static constexpr bool kWide = false;
  static constexpr int kBytes = 2;
  static constexpr int kSteps = 2;
  static __device__ __forceinline__ Acc step(const i32x4 (&a)[2], const i32x4 (&b)[2], Acc c, int i) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[i]), __builtin_bit_cast(bf16x8, a[i]), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 sums(Acc c) { return c; }
  static __device__ __forceinline__ f32x4 bits(Acc c) { return c; }
};
struct StepF16 {
  typedef f32x4 Acc;
  static constexpr bool kWide = false;
  static constexpr int kBytes = 2;
  static constexpr int kSteps = 2;
  static __device__ __forceinline__ Acc step(const i32x4 (&a)[2], const i32x4 (&b)[2], Acc c, int i) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b[i]), __builtin_bit_cast(f16x8, a[i]), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 sums(Acc c) { return c; }
  static __device__ __forceinline__ f32x4 bits(Acc c) { return c; }
};
// e4m3, for results that promise 32-bit sums: the values, exact in f16,
// through the f16 instructions at half the f8 rate.
struct StepF8Wide {
  typedef f32x4 Acc;
  static constexpr bool kWide = true;
  static constexpr int kBytes = 1;
  static __device__ __forceinline__ f16x8 widen(int lo, int hi) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const f16x2 a = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
    const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
    const f16x2 c = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
    const f16x2 d = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  }
  static constexpr int kSteps = 2;
  static __device__ __forceinline__ Acc step(const i32x4 (&a)[2], const i32x4 (&b)[2], Acc c, int i) {
#pragma unroll
    for (int h = 0; h < 4; h += 2)
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(b[i][h], b[i][h + 1]), widen(a[i][h], a[i][h + 1]), c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ f32x4 sums(Acc c) { return c; }
  static __device__ __forceinline__ f32x4 bits(Acc c) { return c; }
};
// e4m3: 32 bytes a lane, block scales of 2^0 (0x7f in e8m0).  The accumulator
// is f32, but the instruction adds its 128 products with an error of up to
// 2^-17 of the sum of their magnitudes (measured on rows whose largest value
// is 448; the 32-long f8 instruction errs the same).  That is far below the
// rounding of a 16-bit result of a long contraction, so those take it; f32
// results and contractions of one step take StepF8Wide.
struct StepF8 {
  typedef f32x4 Acc;
  static constexpr bool kWide = false;
  static constexpr int kBytes = 1;
  static constexpr int kSteps = 1;
  static __device__ __forceinline__ Acc step(const i32x4 (&a)[2], const i32x4 (&b)[2], Acc c, int) {
    const i32x8 x = __builtin_shufflevector(b[0], b[1], 0, 1, 2, 3, 4, 5, 6, 7);
    const i32x8 y = __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
  }
  static __device__ __forceinline__ f32x4 sums(Acc c) { return c; }
  static __device__ __forceinline__ f32x4 bits(Acc c) { return c; }
};
// s8: sums in 32-bit integers, exact up to contractions of 2^17.  Parts of a
// sum stay integers until they are added (bits, whole_sum): rounded to f32 one
// by one, parts of 2^30 that cancel would leave an error of 64 units.
struct StepS8 {
  typedef i32x4 Acc;
  static constexpr bool kWide = false;
  static constexpr int kBytes = 1;
  static constexpr int kSteps = 2;
  static __device__ __forceinline__ Acc step(const i32x4 (&a)[2], const i32x4 (&b)[2], Acc c, int i) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(b[i], a[i], c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 sums(Acc c) {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)c[i];
    return v;
  }
  static __device__ __forceinline__ f32x4 bits(Acc c) { return __builtin_bit_cast(f32x4, c); }
};

// Adds a part of a sum as Step::bits left it (WHOLE: s8), and the sum's value.
template <bool WHOLE>
__device__ __forceinline__ void add_part(float &sum, float part) {
  sum = WHOLE ? __int_as_float(__float_as_int(sum) + __float_as_int(part)) : sum + part;
}
template <bool WHOLE>
__device__ __forceinline__ float whole_sum(float sum) {
  return WHOLE ? (float)__float_as_int(sum) : sum;
}

template <class Step>
__device__ __forceinline__ typename Step::Acc mma(const i32x4 (&a)[2], const i32x4 (&b)[2], typename Step::Acc c) {
#pragma unroll
  for (int k = 0; k < Step::kSteps; ++k) c = Step::step(a, b, c, k);
  return c;
}

}  // namespace hf
