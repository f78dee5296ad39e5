// arx_elem.h — element types, eight-element groups, the dropout generator and
// the activations of the layer operators (arx_rows.hip, arx_linear.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "arx_layer.h"

namespace arx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

template <typename T>
struct Vec;
template <>
struct Vec<__bf16> {
  typedef bf16x8 x8;
};
template <>
struct Vec<_Float16> {
  typedef f16x8 x8;
};
template <>
struct Vec<float> {
  typedef f32x8 x8;
};

// Eight consecutive elements from p on, the first `valid` of them read and the
// rest zero. gfx950 reads 16 bytes from any 2-byte boundary in one
// instruction, so rows of odd strides need no path of their own.
template <typename T>
__device__ __forceinline__ typename Vec<T>::x8 load8(const T* p, int valid) {
  typename Vec<T>::x8 v;
  if (valid >= 8) {
    __builtin_memcpy(&v, p, sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < valid ? p[j] : (T)0.0f;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, typename Vec<T>::x8 v, int valid) {
  if (valid >= 8) {
    __builtin_memcpy(p, &v, sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) p[j] = v[j];
  }
}

template <typename T>
__device__ __forceinline__ f32x8 widen(T v) {
  return __builtin_convertvector(v, f32x8);
}
// One rounding to nearest, ties to even (the hardware's conversion).
template <typename T>
__device__ __forceinline__ typename Vec<T>::x8 narrow(f32x8 v) {
  return __builtin_convertvector(v, typename Vec<T>::x8);
}

// ---- dropout ----------------------------------------------------------------

// Philox4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): a keyed bijection of 128-bit counters.
// The counter is (group, offset), the key the seed, so the bits of an element
// follow from its place alone: the backward pass, another launch shape and
// another rank draw the same ones, and no mask is stored. One counter serves a
// group of eight elements with 16 bits each.
__device__ __forceinline__ void philox(uint64_t group, uint64_t offset, uint64_t seed, uint32_t (&c)[4]) {
  c[0] = (uint32_t)group;
  c[1] = (uint32_t)(group >> 32);
  c[2] = (uint32_t)offset;
  c[3] = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c[0], b = (uint64_t)0xCD9E8D57u * c[2];
    c[0] = (uint32_t)(b >> 32) ^ c[1] ^ k0;
    c[1] = (uint32_t)b;
    c[2] = (uint32_t)(a >> 32) ^ c[3] ^ k1;
    c[3] = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// v with dropped elements zero (selected, so an infinity that is dropped
// leaves no NaN) and kept ones scaled.
__device__ __forceinline__ f32x8 drop8(f32x8 v, uint64_t group, const Drop& d) {
  if (d.threshold == 0) return v;
  uint32_t c[4];
  philox(group, d.offset, d.seed, c);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = (j & 1) ? c[j >> 1] >> 16 : c[j >> 1] & 0xFFFFu;
    v[j] = u >= d.threshold ? v[j] * d.scale : 0.0f;
  }
  return v;
}

// ---- activations ------------------------------------------------------------

// 1 / (1 + e^-v). The exponential's argument is rounded once (2^-24 of it) and
// the reciprocal is the hardware's, within a unit in the last place: far below
// the half precision types that the activations work for.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * v));
}

// The normal distribution's tail beyond |z|, erfc(|z| / sqrt 2) / 2, with
// e = exp(-z^2 / 2): e^(x^2) erfc(x) is close to a polynomial in 1 / (1 + 0.4 x)
// without a constant term; of degree nine, fitted here for the least relative
// error, it is within 1.6e-7 of it over all x >= 0 (the polynomial alone; its
// binary32 evaluation, the reciprocal and e add a few units of 6e-8).
__device__ __forceinline__ float normal_tail(float z, float e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.282842712f, __builtin_fabsf(z), 1.0f));
  float p = 0.0502597243f;
  p = __builtin_fmaf(p, t, -0.182892635f);
  p = __builtin_fmaf(p, t, 0.16907239f);
  p = __builtin_fmaf(p, t, -0.00559764262f);
  p = __builtin_fmaf(p, t, 0.141427338f);
  p = __builtin_fmaf(p, t, 0.168542877f);
  p = __builtin_fmaf(p, t, 0.207842603f);
  p = __builtin_fmaf(p, t, 0.225669608f);
  p = __builtin_fmaf(p, t, 0.225675866f);
  return 0.5f * e * (p * t);
}

// Values past which a slope is constant to binary32; NaN stays.
__device__ __forceinline__ float within(float z, float limit) {
  return __builtin_fabsf(z) > limit ? __builtin_copysignf(limit, z) : z;
}

template <int ACT>
__device__ __forceinline__ float act(float z) {
  if constexpr (ACT == ARX_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if constexpr (ACT == ARX_ACT_GELU) {
    const float q = normal_tail(z, __builtin_amdgcn_exp2f(-0.72134752f * z * z));
    return z * (z < 0.0f ? q : 1.0f - q);
  }
  if constexpr (ACT == ARX_ACT_GELU_TANH)   // (1 + tanh u) / 2 = sigmoid(2 u)
    return z * sigmoid(1.59576912f * __builtin_fmaf(0.044715f * z * z, z, z));
  if constexpr (ACT == ARX_ACT_SILU) return z * sigmoid(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == ARX_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == ARX_ACT_GELU) {
    z = within(z, 16.0f);
    const float e = __builtin_amdgcn_exp2f(-0.72134752f * z * z), q = normal_tail(z, e);
    return __builtin_fmaf(0.398942280f * z, e, z < 0.0f ? q : 1.0f - q);
  }
  if constexpr (ACT == ARX_ACT_GELU_TANH) {
    z = within(z, 16.0f);
    const float f = sigmoid(1.59576912f * __builtin_fmaf(0.044715f * z * z, z, z));
    return __builtin_fmaf(f * (1.0f - f), z * __builtin_fmaf(0.214064448f, z * z, 1.59576912f), f);
  }
  if constexpr (ACT == ARX_ACT_SILU) {
    z = within(z, 80.0f);
    const float f = sigmoid(z);
    return f * __builtin_fmaf(z, 1.0f - f, 1.0f);
  }
  return 1.0f;
}

}  // namespace arx
