// oz_quantize.cu -- matrices of bfloat16, float16 or FP32 to 8-bit floating point, a scale for each block of 128.
//
// A block is 128 neighbours of a row (the operand of a forward or dgrad product), 128 rows of a column (of a
// wgrad product; anew with each group of rows) or 128 x 128 (weights): scale = max |x| / (the type's
// largest value), q = x / scale to nearest.  A gradient needs both of the first two, which one pass gives.
//
// Bound by memory: an element is read once and its one or two bytes are written once.  A CTA holds a 128 x 128
// tile in registers (a thread eight neighbours of eight rows, 16 rows apart), so that all three kinds of
// block are inside a tile: rows by shuffles among 16 lanes, columns by one exchange in shared memory.
// Three CTAs of such threads fit an SM, and what they have asked for of 16-bit tiles while they work on one does not
// keep the memory busy: 16-bit elements (FP32 tiles are twice as large) are copied into shared memory two tiles ahead,
// where each thread finds its own eight 16-byte pieces again, so that no barrier is needed.
// Measured: 8 x 2048 x 4096 FP32 in matrix blocks 53 us (6.3 TB/s); 16384 x 4096 bfloat16 in both 62 us (4.4 TB/s: the
// instructions of two conversions an element bound it; 56 us with one product a conversion instead of a product and a sum,
// which sent values in the middle between two 8-bit ones to either).
#include <atomic>
#include <type_traits>

#include "oz_elements.cuh"
#include "oz_device.cuh"
#include "oz_ragged.cuh"

namespace oz {
namespace {

constexpr int TILE = kScaleBlock, kThreads = 256;

struct QuantParams {
  int k, rows, groups, mats;
  const void* x;
  long long ldx, stride_x;
  const int32_t* offsets;
  uint8_t *q, *qc;
  long long ldq, stride_q, ldqc;
  float *s, *sc;
  long long lds, ldsc;
  int col_tiles, row_tiles, tiles;
  int* status;
};

// Eight bytes of a row from column c on, of which those below k exist.
__device__ __forceinline__ void put_bytes(uint8_t* row, int c, int k, uint2 w) {
  if (c + 8 <= k) {
    *reinterpret_cast<uint2*>(row + c) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < k) row[c + e] = static_cast<uint8_t>((e < 4 ? w.x >> (8 * e) : w.y >> (8 * (e - 4))));
  }
}

// The larger of two magnitudes, of two pairs of 16-bit ones; NaN is the largest.
template <class T>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) {
    return max(a, b);
  } else {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
}
// The bits of a magnitude in FP32.
template <class T>
__device__ __forceinline__ uint32_t raw_magnitude(uint32_t raw) {
  return magnitude(value_of(raw, T()));
}

// Where a tile lies: its matrix, block of rows, first row, how many rows it has, and this thread's first column.
struct Place {
  int mat, block, row, count, c;
};

template <bool MATRIX, bool RAGGED_POSSIBLE>
__device__ __forceinline__ Place place_of(const QuantParams& a, const int* off, int tile) {
  Place p;
  const int rt = tile / a.col_tiles;
  p.c = (tile - rt * a.col_tiles) * TILE + 8 * (threadIdx.x & 15);
  p.mat = MATRIX ? rt / a.row_tiles : 0;
  p.block = rt - p.mat * a.row_tiles;
  p.row = p.block * TILE;
  p.count = min(TILE, a.rows - p.row);
  if (RAGGED_POSSIBLE && a.offsets) {
    int lo = 0, hi = a.groups;  // the last group whose first block is not past this one
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_column_block(off[mid], mid) <= p.block) lo = mid; else hi = mid;
    }
    const int b = p.block - first_column_block(off[lo], lo);
    p.row = off[lo] + b * TILE;
    p.count = b < 0 ? 0 : max(0, min(TILE, off[lo + 1] - p.row));
  }
  return p;
}

constexpr int kAhead = 2;  // tiles on their way into shared memory
constexpr int kTileBytes16 = TILE * TILE * 2;

// BLOCK: an OZ_BLOCK_*.  ALIGNED: rows at multiples of 16 bytes.
// CTAs of an SM: three of 16-bit tiles in shared memory; two hold their tile in 128 registers a thread, but for both blocks at once and
// for shifted pieces.
constexpr int resident_ctas(int block, bool aligned, bool ahead) {
  return ahead ? 3 : block == OZ_BLOCK_BOTH || (!aligned && block != OZ_BLOCK_COLUMN) ? 1 : 2;
}
template <class T, int BLOCK, bool E5M2, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, resident_ctas(BLOCK, ALIGNED, ALIGNED && sizeof(T) == 2)) quantize_kernel(const __grid_constant__ QuantParams a) {
  constexpr bool ROW = BLOCK == OZ_BLOCK_ROW || BLOCK == OZ_BLOCK_BOTH, COLUMN = BLOCK == OZ_BLOCK_COLUMN || BLOCK == OZ_BLOCK_BOTH;
  constexpr bool MATRIX = BLOCK == OZ_BLOCK_MATRIX, AHEAD = ALIGNED && sizeof(T) == 2;
  extern __shared__ uint4 ahead[];  // [kAhead][8][kThreads]
  __shared__ int off[COLUMN ? OZ_MAX_GROUPS + 1 : 1];
  __shared__ uint32_t most[kThreads / 32][TILE];
  __shared__ __align__(16) float inverses[2][COLUMN ? TILE : 4];  // y, rest
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c8 = 8 * (threadIdx.x & 15), r0 = threadIdx.x >> 4;
  let_next_start();
  wait_for_previous();
  const bool ragged = COLUMN && a.offsets;
  if (ragged) {
    if (warp == 0 && clamp_offsets(a.offsets, a.groups, a.rows, off) && lane == 0 && blockIdx.x == 0) atomicExch(a.status, OZ_EINVAL);
    __syncthreads();
  }
  // A tile's pieces of this thread into its places of slot s; those that do not exist as zeros.
  auto send = [&](int tile, int slot) {
    if (tile < a.tiles) {
      const Place p = place_of<MATRIX, COLUMN>(a, off, tile);
      const T* from = static_cast<const T*>(a.x) + p.mat * a.stride_x + static_cast<long long>(p.row + r0) * a.ldx + p.c;
      const int bytes = max(0, min(8, a.k - p.c)) * 2;
      uint32_t to = smem_u32(ahead + slot * 8 * kThreads + threadIdx.x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool have = r0 + 16 * i < p.count && bytes;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(have ? from : static_cast<const T*>(a.x)), "r"(have ? bytes : 0)
                     : "memory");
        from += 16 * a.ldx;
        to += kThreads * 16;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int slot = 0;
  if (AHEAD) {
    for (int s = 0; s < kAhead; ++s) send(blockIdx.x + s * gridDim.x, s);
  }
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const Place place = place_of<MATRIX, COLUMN>(a, off, tile);
    const int c = place.c, mat = place.mat, block = place.block, row = place.row, count = place.count;
    Eight<T> v[8];
    if constexpr (AHEAD) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const Eight<T>*>(ahead + (slot * 8 + i) * kThreads + threadIdx.x);
    } else {
      const T *x = static_cast<const T*>(a.x) + mat * a.stride_x, *end = x + static_cast<long long>(a.rows - 1) * a.ldx + a.k;
      Asked<T, ALIGNED> asked[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        ask_eight(asked[i], x + static_cast<long long>(row + r) * a.ldx, c, r < count ? a.k : 0, x, end);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = take_eight(asked[i], c, r0 + 16 * i < count ? a.k : 0);
    }
    // Largest magnitudes: of FP32 values as bits, of 16-bit ones two at a time (in by_col both columns' in a word).
    constexpr int PAIRS = sizeof(T) == 2 ? 2 : 1;
    uint32_t by_row[8], by_col[8 / PAIRS] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      by_row[i] = 0;
#pragma unroll
      for (int e = 0; e < 8 / PAIRS; ++e) {
        by_row[i] = larger<T>(by_row[i], v[i].w[e] & (PAIRS == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu));
        if (COLUMN) by_col[e] = larger<T>(by_col[e], v[i].w[e] & (PAIRS == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu));
      }
      if (PAIRS == 2) by_row[i] = max(by_row[i] & 0xFFFFu, by_row[i] >> 16);
    }
    if constexpr (AHEAD) {  // the slot has been read (every value of it is in a maximum)
      send(tile + kAhead * gridDim.x, slot);
      slot = slot + 1 == kAhead ? 0 : slot + 1;
    }
    // What make returns for each i, to this thread's columns of row `first` + r0 + 16 i, of which `rows` exist.  Called by whole
    // warps.
    auto put_rows = [&](uint8_t* q, long long ld, long long first, int rows, auto make) {
      uint8_t* to = q + (first + r0) * ld + c;
      if (c - c8 + TILE <= a.k && rows == TILE) {
#pragma unroll
        for (int i = 0; i < 8; ++i, to += 16 * ld) *reinterpret_cast<uint2*>(to) = make(i);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i, to += 16 * ld) {
          const uint2 w = make(i);
          if (r0 + 16 * i < rows) put_bytes(to - c, c, a.k, w);
        }
      }
    };
    auto unpack = [&](int i, float (&f)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = v[i].get(e);
    };
    if (ROW) {
      // The maxima of eight rows over 16 lanes: exchanged so that after three steps a lane holds one row's over eight
      // lanes, which costs 8 shuffles instead of 32, and a lane works out one row's scale instead of eight.
#pragma unroll
      for (int half = 4; half > 0; half >>= 1) {
        const bool upper = lane & half;
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const uint32_t give = upper ? by_row[i] : by_row[i + half], keep = upper ? by_row[i + half] : by_row[i];
          by_row[i] = max(keep, __shfl_xor_sync(0xFFFFFFFFu, give, half));
        }
      }
      const uint32_t amax = raw_magnitude<T>(max(by_row[0], __shfl_xor_sync(0xFFFFFFFFu, by_row[0], 8)));
      const float scale = scale_of<E5M2>(amax);
      const Quotient inverse = inverse_of<E5M2>(amax, scale);
      const int mine = r0 + 16 * (lane & 7);  // this lane's row
      if ((lane & 8) == 0 && mine < count) a.s[c / TILE * a.lds + row + mine] = scale;
      put_rows(a.q, a.ldq, row, count, [&](int i) {
        const Quotient by = {__shfl_sync(0xFFFFFFFFu, inverse.y, (lane & 16) | i), __shfl_sync(0xFFFFFFFFu, inverse.rest, (lane & 16) | i)};
        float f[8];
        unpack(i, f);
        return eight_bits<E5M2>(f, by);
      });
    }
    if constexpr (COLUMN) {
#pragma unroll
      for (int e = 0; e < 8 / PAIRS; ++e) by_col[e] = larger<T>(by_col[e], __shfl_xor_sync(0xFFFFFFFFu, by_col[e], 16));
      if (lane < 16) {
#pragma unroll
        for (int e = 0; e < 8 / PAIRS; ++e) most[warp][c8 / PAIRS + e] = by_col[e];
      }
      __syncthreads();
      if (threadIdx.x < TILE) {  // a column's scale is one thread's
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, static_cast<uint32_t>(reinterpret_cast<const typename Bits<T>::Raw*>(most[w])[threadIdx.x]));
        m = raw_magnitude<T>(m);
        const float scale = scale_of<E5M2>(m);
        const Quotient inverse = inverse_of<E5M2>(m, scale);
        inverses[0][threadIdx.x] = inverse.y;
        inverses[1][threadIdx.x] = inverse.rest;
        const int column = c - c8 + static_cast<int>(threadIdx.x);
        if (column < a.k) a.sc[block * a.ldsc + column] = scale;
      }
      __syncthreads();
      Quotient inverse[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 y = reinterpret_cast<const float4*>(inverses[0] + c8)[i], x = reinterpret_cast<const float4*>(inverses[1] + c8)[i];
        inverse[4 * i] = {y.x, x.x}, inverse[4 * i + 1] = {y.y, x.y}, inverse[4 * i + 2] = {y.z, x.z}, inverse[4 * i + 3] = {y.w, x.w};
      }
      // The rows as they are, or the block's own 128 with zeros behind the group's last (which were read as zeros).
      put_rows(a.qc, a.ldqc, ragged ? static_cast<long long>(block) * TILE : row, ragged ? TILE : count, [&](int i) {
        float f[8];
        unpack(i, f);
        const uint2 w = eight_bits<E5M2>(f, [&](int e) { return inverse[e]; });
        return r0 + 16 * i < count ? w : make_uint2(0, 0);
      });
    }
    if (MATRIX) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, by_row[i]);
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if (lane == 0) most[0][warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) m = max(m, most[0][w]);
      __syncthreads();
      m = raw_magnitude<T>(m);
      const float scale = scale_of<E5M2>(m);
      const Quotient inverse = inverse_of<E5M2>(m, scale);
      if (threadIdx.x == 0) a.s[(static_cast<long long>(mat) * a.row_tiles + block) * a.col_tiles + c / TILE] = scale;
      put_rows(a.q + mat * a.stride_q, a.ldq, row, count, [&](int i) {
        float f[8];
        unpack(i, f);
        return eight_bits<E5M2>(f, inverse);
      });
    }
  }
  // Rows that belong to no group are in no tile: a warp a block of 128.
  if (ROW && ragged) {
    const int lo = off[0], hi = off[a.groups];
    const long long loose = static_cast<long long>(lo + a.rows - hi) * a.col_tiles;
    for (long long i = blockIdx.x * (kThreads / 32) + warp; i < loose; i += gridDim.x * (kThreads / 32)) {
      const int at = static_cast<int>(i / a.col_tiles), b = static_cast<int>(i - static_cast<long long>(at) * a.col_tiles);
      const long long r = at < lo ? at : hi + at - lo;
      const T* x = static_cast<const T*>(a.x) + r * a.ldx;
      float f[8] = {};
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = b * TILE + lane + 32 * e;
        if (c < a.k) f[e] = to_float(x[c]);
        m = max(m, magnitude(f[e]));
      }
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      const float scale = scale_of<E5M2>(m);
      const uint2 v = eight_bits<E5M2>(f, inverse_of<E5M2>(m, scale));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = b * TILE + lane + 32 * e;
        if (c < a.k) a.q[r * a.ldq + c] = static_cast<uint8_t>(v.x >> (8 * e));
      }
      if (lane == 0) a.s[b * a.lds + r] = scale;
    }
  }
}

template <class T, int BLOCK, bool E5M2, bool ALIGNED>
cudaError_t start(const QuantParams& a, cudaStream_t stream) {
  auto kernel = quantize_kernel<T, BLOCK, E5M2, ALIGNED>;
  constexpr bool AHEAD = ALIGNED && sizeof(T) == 2;
  constexpr int smem = AHEAD ? kAhead * kTileBytes16 : 0;
  int grid = 1 << 20;
  if (AHEAD) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // The shared-memory limit is the function's, in this context: set on the first launch (and again below, should a
    // launch be refused, in a new context after a device reset).
    static std::atomic<bool> ready[64] = {};
    const bool known = dev < 64 && ready[dev].load(std::memory_order_acquire);
    if (e == cudaSuccess && !known) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
    grid = 3 * sms;  // as many as run at once
    const dim3 ctas(static_cast<unsigned>(a.tiles < grid ? a.tiles : grid));
    e = launch_overlapping(kernel, ctas, kThreads, smem, stream, a);
    if (e != cudaErrorInvalidValue || !known) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return launch_overlapping(kernel, dim3(static_cast<unsigned>(a.tiles < grid ? a.tiles : grid)), kThreads, smem, stream, a);
}

template <class T, int BLOCK>
cudaError_t launch_quantize(const QuantParams& a, bool e5m2, cudaStream_t stream) {
  const bool aligned = rows_aligned<T>(a.x, a.ldx, a.rows) && (a.mats == 1 || a.stride_x * sizeof(T) % 16 == 0);
  if (aligned) return e5m2 ? start<T, BLOCK, true, true>(a, stream) : start<T, BLOCK, false, true>(a, stream);
  return e5m2 ? start<T, BLOCK, true, false>(a, stream) : start<T, BLOCK, false, false>(a, stream);
}

template <class T>
cudaError_t launch_of_type(int block, const QuantParams& a, bool e5m2, cudaStream_t stream) {
  switch (block) {
    case OZ_BLOCK_ROW: return launch_quantize<T, OZ_BLOCK_ROW>(a, e5m2, stream);
    case OZ_BLOCK_COLUMN: return launch_quantize<T, OZ_BLOCK_COLUMN>(a, e5m2, stream);
    case OZ_BLOCK_BOTH: return launch_quantize<T, OZ_BLOCK_BOTH>(a, e5m2, stream);
    default: return launch_quantize<T, OZ_BLOCK_MATRIX>(a, e5m2, stream);
  }
}

// An 8-bit output: rows at multiples of 16 bytes.
bool output_ok(const void* q, long long ldq, const float* s, long long k, long long rows) {
  return rows == 0 || (q && s && (reinterpret_cast<uintptr_t>(q) & 15) == 0 && (reinterpret_cast<uintptr_t>(s) & 3) == 0 && ldq >= k &&
         (rows <= 1 || ldq % 16 == 0));
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

int ozaki_f8_column_blocks(int rows, int groups, int ragged) {
  if (rows < 0 || groups < 1 || groups > OZ_MAX_GROUPS) return OZ_EINVAL;
  return column_blocks(rows, groups, ragged != 0);
}

int ozaki_quantize_f8(int block, int k, int rows, int groups, int dtype, const void* X, int ldx, long long strideX,
                      const int32_t* offsets, int type, void* Q, int ldq, long long strideQ, float* S, int lds, void* QC, int ldqc,
                      float* SC, int ldsc, cudaStream_t stream) {
  const bool matrix = block == OZ_BLOCK_MATRIX, row = block == OZ_BLOCK_ROW || block == OZ_BLOCK_BOTH;
  const bool column = block == OZ_BLOCK_COLUMN || block == OZ_BLOCK_BOTH;
  if (!matrix && !row && !column) return OZ_EINVAL;
  if (k < 0 || rows < 0 || k > INT32_MAX - 1024 || rows > INT32_MAX - 1024 - 128 * (OZ_MAX_GROUPS + 1) || groups < 1) return OZ_EINVAL;
  if (!matrix && (groups > OZ_MAX_GROUPS || (!offsets && groups != 1))) return OZ_EINVAL;
  if (!column && offsets) return OZ_EINVAL;
  if (!element_bytes(dtype) || (type != OZ_E4M3 && type != OZ_E5M2)) return OZ_EINVAL;
  if (ldx < (k > 1 ? k : 1)) return OZ_EINVAL;
  if (matrix && groups > 1 && (strideX < static_cast<long long>(ldx) * rows || strideQ < static_cast<long long>(ldq) * rows || strideQ % 16)) return OZ_EINVAL;
  if (k == 0 || (rows == 0 && !(column && offsets))) return OZ_OK;
  if ((!X && rows) || !element_aligned(X, dtype)) return OZ_EINVAL;
  if ((row || matrix) && !output_ok(Q, ldq, S, k, matrix ? static_cast<long long>(rows) * groups : rows)) return OZ_EINVAL;
  if (row && lds < rows) return OZ_EINVAL;
  QuantParams a{};
  a.row_tiles = matrix || !offsets ? column_blocks(rows, 1, false) : column_blocks(rows, groups, true);
  if (column && (!output_ok(QC, ldqc, SC, k, offsets ? static_cast<long long>(a.row_tiles) * TILE : rows) || ldsc < k)) return OZ_EINVAL;
  a.k = k;
  a.rows = rows;
  a.groups = groups;
  a.mats = matrix ? groups : 1;
  a.x = X ? X : QC;  // no rows: pieces are still asked for, of no bytes, from an address that has to be one
  a.ldx = ldx;
  a.stride_x = strideX;
  a.offsets = offsets;
  a.q = static_cast<uint8_t*>(Q);
  a.qc = static_cast<uint8_t*>(QC);
  a.ldq = ldq;
  a.stride_q = strideQ;
  a.ldqc = ldqc;
  a.s = S;
  a.sc = SC;
  a.lds = lds;
  a.ldsc = ldsc;
  a.col_tiles = column_blocks(k, 1, false);
  const long long tiles = static_cast<long long>(a.col_tiles) * a.row_tiles * a.mats;
  if (tiles > INT32_MAX / 2) return OZ_EINVAL;  // (2^44 elements)
  a.tiles = static_cast<int>(tiles);
  a.status = device_status_ptr();
  if (!a.status) return OZ_ECUDA;
  const bool e5m2 = type == OZ_E5M2;
  const cudaError_t e = dtype == OZ_BF16 ? launch_of_type<__nv_bfloat16>(block, a, e5m2, stream)
                        : dtype == OZ_F16 ? launch_of_type<__half>(block, a, e5m2, stream)
                                          : launch_of_type<float>(block, a, e5m2, stream);
  return e == cudaSuccess ? OZ_OK : OZ_ECUDA;
}

}  // extern "C"
