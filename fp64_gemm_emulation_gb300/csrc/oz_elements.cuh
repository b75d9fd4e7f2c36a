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

// Elements c .. c + 7 of a row of k, zeros from k on (c is a multiple of 8), in two steps, so that other work comes
// between the loads and their first use.  ALIGNED: rows start at multiples of 16 bytes.  Otherwise the 16-byte pieces
// that hold the elements are loaded, and shifted into place when they are taken.  A piece may reach into the
// neighbouring rows or the gap between them, but not out of the matrix, whose elements lie in [first, end): at
// its two ends elements are loaded one at a time.
template <class T, bool ALIGNED>
struct Asked {
  uint32_t x[Eight<T>::WORDS + (ALIGNED ? 0 : 4)];
  int o;  // bytes before element c in x
};

template <class T, bool ALIGNED>
__device__ __forceinline__ void ask_eight(Asked<T, ALIGNED>& r, const T* row, int c, int k, const T* first, const T* end) {
  constexpr int PIECE = 16 / sizeof(T), N = Eight<T>::WORDS / 4 + (ALIGNED ? 0 : 1);
  r.o = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
  const T* from = row + c - r.o / static_cast<int>(sizeof(T));
  if (ALIGNED ? c + 8 <= k : c < k && from >= first && from + N * PIECE <= end) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(from)[i];
      r.x[4 * i] = v.x, r.x[4 * i + 1] = v.y, r.x[4 * i + 2] = v.z, r.x[4 * i + 3] = v.w;
    }
  } else {
    const Eight<T> v = gather_eight(row + c, 1, [&](int e) { return c + e < k; });
#pragma unroll
    for (int i = 0; i < Eight<T>::WORDS; ++i) r.x[i] = v.w[i];
    r.o = 0;
  }
}

template <class T, bool ALIGNED>
__device__ __forceinline__ Eight<T> take_eight(const Asked<T, ALIGNED>& r, int c, int k) {
  constexpr int W = Eight<T>::WORDS;
  Eight<T> v;
  if constexpr (ALIGNED) {
#pragma unroll
    for (int i = 0; i < W; ++i) v.w[i] = r.x[i];
  } else {
    uint32_t x[W + 4];
#pragma unroll
    for (int i = 0; i < W + 4; ++i) x[i] = r.x[i];
    if (r.o & 8) {
#pragma unroll
      for (int i = 0; i < W + 2; ++i) x[i] = x[i + 2];
    }
    if (r.o & 4) {
#pragma unroll
      for (int i = 0; i < W + 1; ++i) x[i] = x[i + 1];
    }
    if (sizeof(T) == 2 && (r.o & 2)) {
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 16);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) v.w[i] = x[i];
  }
  if (!ALIGNED && c + 8 > k) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(T) == 4) {
        if (c + i >= k) v.w[i] = 0;
      } else {
        if (c + 2 * i >= k) v.w[i] = 0;
        else if (c + 2 * i + 1 >= k) v.w[i] &= 0xFFFFu;
      }
    }
  }
  return v;
}

// Both steps at once.
template <class T, bool ALIGNED>
__device__ __forceinline__ Eight<T> fetch_eight(const T* row, int c, int k, const T* first, const T* end) {
  Asked<T, ALIGNED> r;
  ask_eight(r, row, c, k, first, end);
  return take_eight(r, c, k);
}

// v to elements c .. c + 7 of a row of k.  Called by a whole warp, whose lanes' c are 8 apart.  A row that does not start
// at a multiple of 16 bytes is written in 16-byte pieces all the same: a lane's begins with the last elements of
// the lane before it.  What no whole piece holds (at the row's and the warp's ends) goes an element at a time.
template <class T, bool ALIGNED>
__device__ __forceinline__ void store_eight_of_row(T* row, int c, int k, const float (&v)[8]) {
  const int o = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
  if (o == 0) {
    if (c + 8 <= k) {
      store_eight(row + c, v);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < k) from_float(v[e], row[c + e]);
    return;
  }
  constexpr int W = Eight<T>::WORDS, PIECE = 16 / sizeof(T);
  const int s = o / static_cast<int>(sizeof(T)), lane = threadIdx.x & 31, q = 16 - o;
  uint32_t x[W + 4];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (sizeof(T) == 4) x[4 + i] = __float_as_uint(v[i]);
    else x[4 + i] = pack_two(v[2 * i], v[2 * i + 1], T());
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __shfl_up_sync(0xFFFFFFFFu, x[W + i], 1);
  if (q & 8) {
#pragma unroll
    for (int i = 0; i < W + 2; ++i) x[i] = x[i + 2];
  }
  if (q & 4) {
#pragma unroll
    for (int i = 0; i < W + 1; ++i) x[i] = x[i + 1];
  }
  if (sizeof(T) == 2 && (q & 2)) {
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 16);
  }
  // Piece i holds elements c - s + i PIECE and on.
  auto whole = [&](int i) { return c - s + (i + 1) * PIECE <= k && (lane > 0 || i > 0); };
#pragma unroll
  for (int i = 0; i < W / 4; ++i)
    if (whole(i)) *reinterpret_cast<uint4*>(row + c - s + i * PIECE) = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  const bool next = lane < 31 && c + 8 - s + PIECE <= k;  // the next lane's first piece
  if (lane == 0 || !next || !whole(W / 4 - 1)) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < k && !(e >= 8 - s ? next : whole((e + s) / PIECE))) from_float(v[e], row[c + e]);
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

// The quotient a / b, a > 0, as y + rest: y below it by at most 6 steps, rest >= 0 what it lacks, so that v y + v rest, rounded
// once, is v a / b within 2^-40 before that.  (rest >= 0: a v of -0 stays one.)  Where y is below 2^-100, rest is below the
// normal range: then within 2^-29.  A b of Inf gives zeros, a NaN NaN.
struct Quotient {
  float y, rest;
};
// near: within 2^-23 of b / a.  (With the division's rounding 3 / 2 of that, 3 steps at most.)
__device__ __forceinline__ Quotient quotient_of(float a, float b, float near) {
  const float y = __uint_as_float(max(__float_as_uint(1.0f / near), 3u) - 3u);
  return {y, y == 0.0f ? 0.0f : fmaf(-y, b, a) * (y * (1.0f / a))};
}
// What a block's values are multiplied by: one over its scale before that was rounded, so that a 16-bit value in the middle
// between two 8-bit ones is found there.
template <bool E5M2>
__device__ __forceinline__ Quotient inverse_of(uint32_t amax, float scale) {
  constexpr float LARGEST = E5M2 ? 57344.0f : 448.0f;
  const float v = __uint_as_float(amax);
  const bool exact = v >= LARGEST * 1.17549435e-38f && v <= 3.40282347e38f;
  return quotient_of(exact ? LARGEST : 1.0f, exact ? v : scale, scale);
}

// v times the quotient r, rounded to FP32 once.
__device__ __forceinline__ float times(float v, Quotient r) { return fmaf(v, r.y, v * r.rest); }

// Eight values times quotients (r(e): of value e), to the nearest 8-bit ones (largest values stay finite; NaN stays NaN).
template <bool E5M2, class R>
__device__ __forceinline__ uint2 eight_bits(const float (&v)[8], R r) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(times(v[2 * i], r(2 * i)), times(v[2 * i + 1], r(2 * i + 1))), __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
template <bool E5M2>
__device__ __forceinline__ uint2 eight_bits(const float (&v)[8], Quotient r) {
  return eight_bits<E5M2>(v, [&](int) { return r; });
}

// Whether rows of T from p on, ld apart, all start at multiples of 16 bytes.
template <class T>
bool rows_aligned(const void* p, long long ld, long long rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows <= 1 || ld * static_cast<long long>(sizeof(T)) % 16 == 0);
}

inline size_t element_bytes(int dtype) { return dtype == OZ_F32 ? 4 : dtype == OZ_BF16 || dtype == OZ_F16 ? 2 : 0; }
inline bool element_aligned(const void* p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (element_bytes(dtype) - 1)) == 0; }

}  // namespace oz
