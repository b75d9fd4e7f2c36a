// oz_elements.cuh -- runs of eight elements of a row in FP32, and 8-bit values with their scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "oz_internal.h"

namespace oz {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float v, float& r) { r = v; }
__device__ __forceinline__ void from_float(float v, __half& r) { r = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16& r) { r = __float2bfloat16_rn(v); }

// Eight neighbours, 16-byte aligned.
template <class T>
struct alignas(16) Eight {
  T e[8];
};

template <class T>
__device__ __forceinline__ Eight<T> load_eight(const T* p) {
  Eight<T> r;
  const uint4* from = reinterpret_cast<const uint4*>(p);
  uint4* to = reinterpret_cast<uint4*>(&r);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) to[i] = from[i];
  return r;
}
template <class T>
__device__ __forceinline__ void store_eight(T* p, const float (&v)[8]) {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) from_float(v[i], r.e[i]);
  const uint4* from = reinterpret_cast<const uint4*>(&r);
  uint4* to = reinterpret_cast<uint4*>(p);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) to[i] = from[i];
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
