// oz_elements.cuh -- runs of eight elements of a row in FP32, and 8-bit values with their scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "oz_internal.h"

namespace oz {

__device__ __forceinline__ void from_float(float v, float& r) { r = v; }
__device__ __forceinline__ void from_float(float v, __half& r) { r = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16& r) { r = __float2bfloat16_rn(v); }

// An element's bits, and its value.
template <class T>
struct Bits {
  typedef uint16_t Raw;
};
template <>
struct Bits<float> {
  typedef uint32_t Raw;
};
__device__ __forceinline__ float value_of(uint32_t raw, float) { return __uint_as_float(raw); }
__device__ __forceinline__ float value_of(uint32_t raw, __half) { return __half2float(__ushort_as_half(static_cast<unsigned short>(raw))); }
__device__ __forceinline__ float value_of(uint32_t raw, __nv_bfloat16) { return __uint_as_float(raw << 16); }
template <class T>
__device__ __forceinline__ float to_float(const T& v) {
  return value_of(*reinterpret_cast<const typename Bits<T>::Raw*>(&v), T());
}

// Eight elements in as many registers as they fill (16-bit ones in pairs, the first in the low half).
template <class T>
struct alignas(16) Eight {
  static constexpr int WORDS = 2 * sizeof(T);
  uint32_t w[WORDS];
  __device__ __forceinline__ float get(int e) const {
    if (sizeof(T) == 4) return __uint_as_float(w[e]);
    return value_of(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu, T());
  }
};
template <>
__device__ __forceinline__ float Eight<__nv_bfloat16>::get(int e) const {
  return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
}

// Element e is at row[e * step] where valid(e), zero otherwise.
template <class T, class V>
__device__ __forceinline__ Eight<T> gather_eight(const T* row, int step, V valid) {
  const typename Bits<T>::Raw* raw = reinterpret_cast<const typename Bits<T>::Raw*>(row);
  Eight<T> r;
  if (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < Eight<T>::WORDS; ++e) r.w[e] = valid(e) ? raw[e * step] : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = valid(2 * i) ? raw[2 * i * step] : 0u, hi = valid(2 * i + 1) ? raw[(2 * i + 1) * step] : 0u;
      r.w[i] = lo | hi << 16;
    }
  }
  return r;
}
// Eight neighbours, 16-byte aligned.
template <class T>
__device__ __forceinline__ Eight<T> load_eight(const T* p) {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < Eight<T>::WORDS / 4; ++i) {
    const uint4 x = reinterpret_cast<const uint4*>(p)[i];
    r.w[4 * i] = x.x, r.w[4 * i + 1] = x.y, r.w[4 * i + 2] = x.z, r.w[4 * i + 3] = x.w;
  }
  return r;
}
__device__ __forceinline__ uint32_t pack_two(float a, float b, __half) {
  const __half2 x = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint32_t pack_two(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&x);
}
template <class T>
__device__ __forceinline__ void store_eight(T* p, const float (&v)[8]) {
  uint4* to = reinterpret_cast<uint4*>(p);
  if constexpr (sizeof(T) == 4) {
    to[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    to[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    to[0] = make_uint4(pack_two(v[0], v[1], T()), pack_two(v[2], v[3], T()), pack_two(v[4], v[5], T()), pack_two(v[6], v[7], T()));
  }
}

// Magnitudes as ordered bits: a NaN is above Inf and Inf above all numbers, so a maximum keeps them.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The scale of a block whose largest magnitude is amax: amax / (the type's largest value), not below 2^-126
// (so that its reciprocal is finite), and 1 for a block of zeros.  A block with Inf or NaN gets one of them.
template <bool E5M2>
__device__ __forceinline__ float scale_of(uint32_t amax) {
  if (amax == 0) return 1.0f;
  const float s = __fdiv_rn(__uint_as_float(amax), E5M2 ? 57344.0f : 448.0f);
  return s < 1.17549435e-38f ? 1.17549435e-38f : s;
}

// Eight values times 1 / scale, to the nearest 8-bit ones (largest values stay finite; NaN stays NaN).  The
// product with the reciprocal is within 2^-23 of the quotient, so a value that near to the middle
// between two 8-bit ones may go to either.
template <bool E5M2>
__device__ __forceinline__ uint2 eight_bits(const float (&v)[8], float inverse) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inverse, v[2 * i + 1] * inverse), __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Whether rows of T from p on, ld apart, all start at multiples of 16 bytes.
template <class T>
bool rows_aligned(const void* p, long long ld, long long rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows <= 1 || ld * static_cast<long long>(sizeof(T)) % 16 == 0);
}

inline size_t element_bytes(int dtype) { return dtype == OZ_F32 ? 4 : dtype == OZ_BF16 || dtype == OZ_F16 ? 2 : 0; }
inline bool element_aligned(const void* p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (element_bytes(dtype) - 1)) == 0; }

}  // namespace oz
