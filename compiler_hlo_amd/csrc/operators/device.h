// device.h -- what the operators' kernels share: element types, 16-byte
// vectors, the activations and the generator.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "operators.h"

namespace hf {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct BF16 {
  static constexpr int kBytes = 2;
  typedef uint16_t Store;
  static __device__ __forceinline__ float load(Store v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ Store store(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};
struct F16 {
  static constexpr int kBytes = 2;
  typedef uint16_t Store;
  static __device__ __forceinline__ float load(Store v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ Store store(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};
struct F32 {
  static constexpr int kBytes = 4;
  typedef float Store;
  static __device__ __forceinline__ float load(Store v) { return v; }
  static __device__ __forceinline__ Store store(float f) { return f; }
};

// Launches a kernel and returns this launch's own error.
template <class T>
struct Same {
  typedef T Type;
};
template <class... P>
inline hipError_t launch(void (*kernel)(P...), dim3 grid, unsigned block, hipStream_t s, typename Same<P>::Type... args) {
  void *pointers[] = {&args...};
  return hipLaunchKernel((const void *)kernel, grid, dim3(block), pointers, 0, s);
}

// A launch's number of threads in x stays below 2^32, so workgroups of BLOCK
// threads past 2^31 are counted on in y.  (The last row of such a grid may
// pass the end.  The width is a constant because gridDim is a load.)
template <int BLOCK>
inline dim3 grid_of(int64_t blocks) {
  const int64_t most = (int64_t(1) << 31) / BLOCK, x = blocks < most ? blocks : most;
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
template <int BLOCK>
__device__ __forceinline__ int64_t block_number(unsigned x, unsigned y) {
  return (int64_t)y * ((int64_t(1) << 31) / BLOCK) + x;
}

// Eight consecutive elements as 32-bit floats: one 16-byte access in the
// 16-bit types, two in f32.  p is 16-byte aligned.
template <class T>
__device__ __forceinline__ void load8(const typename T::Store *p, float (&v)[8]) {
  if constexpr (T::kBytes == 4) {
    const f32x4 a = ((const f32x4 *)p)[0], b = ((const f32x4 *)p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
    const u32x4 a = *(const u32x4 *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = T::load((uint16_t)(a[i] & 0xffff));
      v[2 * i + 1] = T::load((uint16_t)(a[i] >> 16));
    }
  }
}

// Results in 16 bits are stored past the caches: a kernel's end waits for the
// L2s to write back what they hold, 8 us of a norm's 30 over 4099 rows of 4096
// (bf16; 21 us so).  In f32 the two accesses of 16 bytes a lane need the cache
// to become whole lines (54 us through it, 64 past it).
template <class T>
__device__ __forceinline__ void store8(typename T::Store *p, const float (&v)[8]) {
  if constexpr (T::kBytes == 4) {
    f32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = v[i], b[i] = v[4 + i];
    ((f32x4 *)p)[0] = a;
    ((f32x4 *)p)[1] = b;
  } else {
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = (uint32_t)T::store(v[2 * i]) | (uint32_t)T::store(v[2 * i + 1]) << 16;
    __builtin_nontemporal_store(a, (u32x4 *)p);
  }
}

// W consecutive elements at any alignment, in whole accesses (the hardware's
// memory takes them unaligned).
template <class T, int W>
__device__ __forceinline__ void load_any(const typename T::Store *p, float (&v)[W]) {
  typename T::Store t[W];
  __builtin_memcpy(t, p, sizeof t);
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = T::load(t[i]);
}
template <class T, int W>
__device__ __forceinline__ void store_any(typename T::Store *p, const float (&v)[W]) {
  typename T::Store t[W];
#pragma unroll
  for (int i = 0; i < W; ++i) t[i] = T::store(v[i]);
  __builtin_memcpy(p, t, sizeof t);
}

// Four consecutive elements; p is 8-byte (16-bit types) or 16-byte (f32)
// aligned.
template <class T>
__device__ __forceinline__ f32x4 load4(const typename T::Store *p) {
  f32x4 v;
  if constexpr (T::kBytes == 4) {
    v = *(const f32x4 *)p;
  } else {
    const u32x2 a = *(const u32x2 *)p;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = T::load((uint16_t)(a[i] & 0xffff));
      v[2 * i + 1] = T::load((uint16_t)(a[i] >> 16));
    }
  }
  return v;
}

template <class T>
__device__ __forceinline__ void store4(typename T::Store *p, f32x4 v) {
  if constexpr (T::kBytes == 4) {
    *(f32x4 *)p = v;
  } else {
    u32x2 a;
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = (uint32_t)T::store(v[2 * i]) | (uint32_t)T::store(v[2 * i + 1]) << 16;
    *(u32x2 *)p = a;
  }
}

// 1 / (1 + exp(-z)) by the hardware's exp2 and reciprocal, each within one
// ulp.  exp(-z) = 2^(-z log2 e) carries the argument's rounding, so where the
// sigmoid falls off as exp(z) it is off by |z| 2^-24 of itself: ten units of
// f32 at z = -20, nothing in 16 bits.  z = -inf gives 0, +inf gives 1.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// The same within a few ulps for every z, for results in f32: the argument in
// 64 bits, its part beyond f32 as a factor 1 + lo ln 2.  Where exp2 leaves the
// range on either side there is nothing to correct.
__device__ __forceinline__ float sigmoid_fine(double z) {
  const double e = z * -1.4426950408889634;
  const float hi = (float)e;
  float x = __builtin_amdgcn_exp2f(hi);
  if (hi > -150.f && hi < 128.f) x = __builtin_fmaf(x, (float)(e - (double)hi) * 0.6931471805599453f, x);
  return __builtin_amdgcn_rcpf(1.0f + x);
}

// act(z) and act'(z).  GELU is the tanh form, 0.5 z (1 + tanh u) with
// u = sqrt(2/pi) (z + 0.044715 z^3), written as z sigmoid(2u).
// FINE: for results in f32, with GELU's cubic argument in 64 bits too; else to
// the precision that 16 bits show.
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2/pi)

template <bool FINE>
__device__ __forceinline__ float act_value(int kind, float z) {
  if (kind == HF_ACTIVATION_RELU) return z > 0.f ? z : (z == z ? 0.f : z);
  if (kind == HF_ACTIVATION_SILU) return z == -__builtin_inff() ? 0.f : z * (FINE ? sigmoid_fine((double)z) : sigmoid(z));
  if (kind == HF_ACTIVATION_GELU) {
    const double w = (double)z;
    return z == -__builtin_inff() ? 0.f
           : FINE ? z * sigmoid_fine(1.5957691216057308 * w * (1.0 + 0.044715 * w * w))
                  : z * sigmoid(kGelu2 * z * (1.f + 0.044715f * z * z));
  }
  return z;
}

// At z = -inf and +inf the derivatives are their limits, 0 and 1: there
// z * (1 - sigmoid) would be inf * 0, so z is held to +-1e4, where the
// sigmoid has long been 0 or 1 and z^3 is finite.
__device__ __forceinline__ float act_both(int kind, float z, float *d) {
  if (kind == HF_ACTIVATION_RELU) {
    *d = z > 0.f ? 1.f : 0.f;
    return act_value<false>(kind, z);
  }
  if (kind == HF_ACTIVATION_SILU || kind == HF_ACTIVATION_GELU) {
    const float c = z != z ? z : __builtin_fminf(__builtin_fmaxf(z, -1e4f), 1e4f);
    if (kind == HF_ACTIVATION_SILU) {
      const float s = sigmoid(c);
      *d = s + c * s * (1.f - s);
      return z == -__builtin_inff() ? 0.f : z * s;
    }
    const float s = sigmoid(kGelu2 * c * (1.f + 0.044715f * c * c));
    *d = s + c * s * (1.f - s) * kGelu2 * (1.f + 0.134145f * c * c);
    return z == -__builtin_inff() ? 0.f : z * s;
  }
  *d = 1.f;
  return z;
}

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as
// easy as 1, 2, 3", 2011) of a 64-bit counter and a 64-bit key.
__device__ __forceinline__ u32x4 philox(uint64_t counter, uint64_t key) {
  uint32_t a = (uint32_t)counter, b = (uint32_t)(counter >> 32), c = 0, d = 0;
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = (uint64_t)0xD2511F53u * a, q = (uint64_t)0xCD9E8D57u * c;
    a = (uint32_t)(q >> 32) ^ b ^ k0;
    b = (uint32_t)q;
    c = (uint32_t)(p >> 32) ^ d ^ k1;
    d = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  u32x4 r;
  r[0] = a, r[1] = b, r[2] = c, r[3] = d;
  return r;
}

}  // namespace hf
