// oz_norm.cu -- root-mean-square norm of rows with the residual's addition, its result in 8 bits with a scale
// for each block of 128, and its gradients.
//
//   forward   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w   -> q, scales (of y), h, r; y if wanted
//   backward  g = dy w,  dx = dh + r (g - h r^2 mean(g h)),  dw = sum over rows of dy h r
// All in FP32, from the FP32 sum h, not from the stored one; q is rounded from the ratio of h w to its block's largest.
//
// Bound by memory: every row is read once, held in registers between its sum and its results, and written
// once.  With many rows the CTAs stay, keep w in registers, and fetch their next row while they work on one: the
// waits of a row (for its values, its sum's barrier) would otherwise follow each other (16384 rows of 4096 bfloat16 values
// with a residual: 79 us, 5.9 TB/s; 127 with a CTA a row).  Several threads share a row, eight neighbours each (a block of
// 128 is 16 threads); rows that do not start at multiples of 16 bytes are read and written in 16-byte pieces too, shifted
// (7777 rows of 2049 bfloat16 values backward: 41 us, 3.1 TB/s; 68 with an access an element).
#include <atomic>

#include "oz_elements.cuh"
#include "oz_device.cuh"
#include "oz_ragged.cuh"

namespace oz {
namespace {

struct NormParams {
  int k, rows;
  const void *x, *residual, *w;
  void *h, *y;
  uint8_t* q;
  float *s, *rstd;
  long long ldx, ldr, ldh, ldy, ldq, lds;
  float eps;
};

struct NormBackParams {
  int k, rows;
  const void *dy, *h, *w, *dh;
  const float* rstd;
  void *dx, *dw;
  long long lddy, ldh, lddh, lddx;
  float* part;  // [CTAs][k]
  int parts;
  int period;   // rows after which one starts alike against 16 bytes
};

// The sum over a row's threads (blockDim.x of them, whole warps); meet: room for 32 floats of each row.
__device__ __forceinline__ float row_sum(float v, float* meet) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) meet[warp] = v;
  __syncthreads();
  v = lane < warps ? meet[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// The first of a thread's eight columns of run j.
__device__ __forceinline__ int first_column(int j) { return 8 * static_cast<int>(threadIdx.x + j * blockDim.x); }

// A matrix that is read by eights.
template <class T, bool VEC>
struct Rows {
  const T *first, *end;
  long long ld;
  int rows, k;
  __device__ Rows(const void* p, long long ld, int rows, int k)
      : first(static_cast<const T*>(p)), end(first + (rows - 1) * ld + k), ld(ld), rows(rows), k(k) {}
  __device__ void ask(Asked<T, VEC>& r, int row, int c) const { ask_eight(r, first + row * ld, c, row < rows ? k : 0, first, end); }
  __device__ Eight<T> fetch(int row, int c) const { return fetch_eight<T, VEC>(first + row * ld, c, row < rows ? k : 0, first, end); }
};

// CTAs of 256 threads on an SM: what the registers hold; shifted pieces of two runs spill with a third (16384 x 4095 bfloat16 with a
// residual 230 us instead of 203).
__host__ __device__ constexpr int resident_ctas(bool vec, int runs) { return runs == 1 ? 4 : runs == 2 && vec ? 3 : 2; }

// q is y / scale, in which r cancels: 448 h w / (the block's largest |h w|), so that the roundings of r, of the scale and of h r
// do not come before the one to 8 bits (with two 16-bit summands h w often is exact).  h is multiplied by r's power of two
// all the same, which rounds nothing, so that h w leaves the range of FP32 only where y does.
//
// RUNS: runs of eight elements a thread holds.  blockDim (threads of a row, rows).  STAY: a CTA takes every
// gridDim.x-th group of rows, at most 256 threads; otherwise one.
template <class T, bool VEC, int RUNS, bool STAY>
__global__ void __launch_bounds__(STAY ? 256 : 1024, STAY ? resident_ctas(VEC, RUNS) : 1) norm_kernel(const __grid_constant__ NormParams a) {
  __shared__ float meet[2][32];
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, step = STAY ? gridDim.x * blockDim.y : a.rows;
  int row = blockIdx.x * blockDim.y + threadIdx.y, turn = 0;
  const Rows<T, VEC> x(a.x, a.ldx, a.rows, a.k), res(a.residual, a.ldr, a.rows, a.k);
  Asked<T, VEC> nx[RUNS], nr[RUNS];
  Eight<T> w[RUNS];
  auto ask = [&](int row) {
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      x.ask(nx[j], row, first_column(j));
      if (a.residual) res.ask(nr[j], row, first_column(j));
    }
  };
  ask(row);
#pragma unroll
  for (int j = 0; j < RUNS; ++j) w[j] = Rows<T, VEC>(a.w, 0, 1, a.k).fetch(0, first_column(j));
  for (; row < a.rows; row += step, turn ^= 1) {
    float h[RUNS][8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const int c = first_column(j);
      const Eight<T> vx = take_eight(nx[j], c, a.k);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] = vx.get(e);
      if (a.residual) {
        const Eight<T> vr = take_eight(nr[j], c, a.k);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] += vr.get(e);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = fmaf(h[j][e], h[j][e], sum);
      }
    }
    if (STAY) ask(row + step);
    sum = row_sum(sum, meet[turn]);
    const float r = 1.0f / sqrtf(sum / static_cast<float>(a.k) + a.eps);
    if (threadIdx.x == 0) a.rstd[row] = r;
    const uint32_t bits = __float_as_uint(r);
    const float power = r < __int_as_float(0x7F800000) ? __uint_as_float(bits & 0x7F800000u) : r, mantissa = __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
    // The largest |h w| of each run's block, which 16 lanes hold.
    uint32_t most[RUNS];
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const int c = first_column(j);
      if (a.h) store_eight_of_row<T, VEC>(static_cast<T*>(a.h) + row * a.ldh, c, a.k, h[j]);
      most[j] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[j][e] = h[j][e] * power * w[j].get(e);
        most[j] = max(most[j], c + e < a.k ? magnitude(h[j][e]) : 0u);
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) most[j] = max(most[j], __shfl_xor_sync(0xFFFFFFFFu, most[j], d));
    }
    // A lane works out the scale of one run's block.
    const int mine = lane & (RUNS - 1);
    uint32_t amax = most[0];
#pragma unroll
    for (int j = 1; j < RUNS; ++j) amax = mine == j ? most[j] : amax;
    const float top = __uint_as_float(amax), scale = scale_of<false>(magnitude(top * mantissa));
    const bool least = !(top >= 448.0f * 1.17549435e-38f), exact = !least && top <= 3.40282347e38f;  // least: the smallest scales, and 1; NaN too
    const Quotient inverse = quotient_of(exact ? 448.0f : 1.0f, exact ? top : scale, exact ? top * (1.0f / 448.0f) : scale);
    const bool any_least = __any_sync(0xFFFFFFFFu, least);
    const int block = 8 * ((static_cast<int>(threadIdx.x) & ~15) + mine * static_cast<int>(blockDim.x));
    if ((lane & 15) < RUNS && block < a.k) a.s[block / kScaleBlock * a.lds + row] = scale;
    uint8_t* q = a.q + row * a.ldq;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const int c = first_column(j), from = (lane & 16) | j;
      const Quotient by = {__shfl_sync(0xFFFFFFFFu, inverse.y, from), __shfl_sync(0xFFFFFFFFu, inverse.rest, from)};
      float to_y = mantissa;
      if (any_least) {
        const float f = __shfl_sync(0xFFFFFFFFu, least ? mantissa : 1.0f, from);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] *= f;
        if (f != 1.0f) to_y = 1.0f;
      }
      const uint2 v = eight_bits<false>(h[j], by);
      if (c + 8 <= a.k) {
        *reinterpret_cast<uint2*>(q + c) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < a.k) q[c + e] = static_cast<uint8_t>(e < 4 ? v.x >> (8 * e) : v.y >> (8 * (e - 4)));
      }
      if (a.y) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[j][e] *= to_y;
        store_eight_of_row<T, VEC>(static_cast<T*>(a.y) + row * a.ldy, c, a.k, h[j]);
      }
    }
  }
}

// Gradients: a CTA takes every so many rows and keeps dw's sums of its columns in registers; the CTAs' sums go to
// the workspace and are added in their order by a second launch, so results do not depend on timing.
// With one run a thread the next row is fetched into registers meanwhile (two and more leave none for it).
//
// Rows that do not start at multiples of 16 bytes: the rows whose starts lie alike against 16 bytes are every
// `period`-th, and a CTA takes only such.  Its threads' eight columns then start `shift` elements before a multiple of
// 8, so that all their accesses are of whole 16-byte pieces, and w and dw still belong to fixed threads; only a row's
// first and last piece hold elements that are not the row's (read where they are the matrix's own, never written).
// PIECES: all matrices lie alike (and one thread's eight elements are whole pieces); otherwise element by element.
template <class T, bool PIECES>
struct Columns {
  const T *at, *end;  // the next row's first element, the matrix's end
  long long step;     // elements from one of the CTA's rows to the next
  __device__ Columns(const void* p, long long ld, int rows, int k, int row, int step)
      : at(static_cast<const T*>(p) + row * ld), end(static_cast<const T*>(p) + (rows - 1) * ld + k), step(step * ld) {}
  // Eight columns of that row from c on, without a mask: what is in columns outside [0, k) may be anything.  Nothing is read
  // before the matrix's first element, which the columns before row 0 .. 6 may be (rows have a distance of at least 1).
  __device__ Eight<T> load(int c, int k, int row) const {
    const T* from = at + c;
    if (PIECES && ((c >= 0 && c + 8 <= k) || (c < k && (c >= 0 || row > 6) && from + 8 <= end))) return load_eight(from);
    return gather_eight(from, 1, [&](int e) { return c + e >= 0 && c + e < k; });
  }
};

template <class T, bool PIECES, int RUNS>
__global__ void __launch_bounds__(1024, 1) norm_back_kernel(const __grid_constant__ NormBackParams a) {
  constexpr bool EARLY = RUNS == 1;
  __shared__ float meet[2][32];
  let_next_start();
  wait_for_previous();
  const int kind = static_cast<int>(blockIdx.x) % a.period;  // rows kind, kind + period, ...
  const int shift = PIECES ? static_cast<int>((reinterpret_cast<uintptr_t>(a.dy) + kind * a.lddy * sizeof(T)) & 15) / static_cast<int>(sizeof(T)) : 0;
  const int step = a.period * ((static_cast<int>(gridDim.x) - kind + a.period - 1) / a.period);  // (CTAs of this kind)
  auto column = [&](int j) { return first_column(j) - shift; };
  auto mask = [&](int c, float (&v)[8]) {
    if (c < 0 || c + 8 > a.k) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < 0 || c + e >= a.k) v[e] = 0.0f;
    }
  };
  float dw[RUNS][8];
#pragma unroll
  for (int i = 0; i < RUNS * 8; ++i) dw[i >> 3][i & 7] = 0.0f;
  int row = kind + a.period * (static_cast<int>(blockIdx.x) / a.period), turn = 0;
  Columns<T, PIECES> rdy(a.dy, a.lddy, a.rows, a.k, row, step), rh(a.h, a.ldh, a.rows, a.k, row, step), rdh(a.dh, a.lddh, a.rows, a.k, row, step);
  T* to_row = static_cast<T*>(a.dx) + row * a.lddx;
  const float each = 1.0f / static_cast<float>(a.k);
  Eight<T> dy[RUNS] = {}, h[RUNS] = {}, dh[RUNS] = {}, w[RUNS];
  float r = 0.0f;
  auto ask = [&](int row) {
    if (row >= a.rows) return;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      dy[j] = rdy.load(column(j), a.k, row);
      h[j] = rh.load(column(j), a.k, row);
      if (EARLY && a.dh) dh[j] = rdh.load(column(j), a.k, row);
    }
    r = a.rstd[row];
    rdy.at += rdy.step;
    rh.at += rh.step;
    if (EARLY) rdh.at += rdh.step;
  };
  if (EARLY) ask(row);
#pragma unroll
  for (int j = 0; j < RUNS; ++j) w[j] = Columns<T, false>(a.w, 0, 1, a.k, 0, 0).load(column(j), a.k, 0);
  for (; row < a.rows; row += step, turn ^= 1) {
    if (!EARLY) ask(row);
    float dot = 0.0f;
    const float rs = r;
    Eight<T> dy1[EARLY ? 1 : RUNS], h1[EARLY ? 1 : RUNS], dh1[EARLY ? 1 : RUNS];  // this row's
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      dy1[j] = dy[j], h1[j] = h[j], dh1[j] = dh[j];
      float d[8], v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = dy[j].get(e), v[e] = h[j].get(e);
      mask(column(j), d);
      mask(column(j), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dot = fmaf(d[e] * w[j].get(e), v[e], dot);
        dw[j][e] = fmaf(d[e] * rs, v[e], dw[j][e]);
      }
    }
    if (EARLY) ask(row + step);
    // Two rooms in turn: a warp writes one again only after the other's barrier.
    dot = row_sum(dot, meet[turn]) * each;
    const float f = rs * rs * dot;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const int c = column(j);
      if (!EARLY && a.dh) dh1[j] = rdh.load(c, a.k, row);
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dx[e] = rs * (dy1[j].get(e) * w[j].get(e) - h1[j].get(e) * f);
        if (a.dh) dx[e] += dh1[j].get(e);
      }
      T* to = to_row + c;
      if (PIECES && c >= 0 && c + 8 <= a.k) {
        store_eight(to, dx);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e >= 0 && c + e < a.k) from_float(dx[e], to[e]);
      }
    }
    to_row += step * a.lddx;
    if (!EARLY) rdh.at += rdh.step;
  }
#pragma unroll
  for (int j = 0; j < RUNS; ++j) {
    const int c = column(j);
    float* part = a.part + static_cast<long long>(blockIdx.x) * a.k;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e >= 0 && c + e < a.k) part[c + e] = dw[j][e];
  }
}

// The same for 16-bit elements where all accesses are whole pieces, rows of at most two runs: a CTA's next two rows are on
// their way into shared memory, where each thread finds its own pieces again (so no barrier is needed), twice: for the
// sum, and behind the barrier for dx, so that a row takes no registers meanwhile.  (FP32: a thread's two pieces are
// neighbours, and copied apart they use half of each sector: 8192 x 4096 141 us instead of 108.)
// Against a row ahead in registers: 16384 x 4096 with dh 116 -> 90 us (6.0 TB/s), 4096 x 16384 288 -> 90, 7777 x 2049 46 -> 41.
// EDGES: pieces that are not whole columns of the row exist (compiled in, their code costs rows without them a fifth:
// 16384 x 4096 117 us).
constexpr int kRowsAhead = 2;
template <class T, int RUNS, bool EDGES>
__global__ void __launch_bounds__(1024, 1) norm_back_staged_kernel(const __grid_constant__ NormBackParams a) {
  static_assert(sizeof(T) == 2, "a run is one piece");
  extern __shared__ uint4 staged[];  // [kRowsAhead][dy, h, dh][RUNS][threads]
  __shared__ float meet[2][32];
  let_next_start();
  wait_for_previous();
  const int threads = blockDim.x, matrix = RUNS * threads, slot_size = (a.dh ? 3 : 2) * matrix;
  const int kind = EDGES ? static_cast<int>(blockIdx.x) % a.period : 0;  // rows kind, kind + period, ...
  const int shift = !EDGES ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(a.dy) + kind * a.lddy * sizeof(T)) & 15) / static_cast<int>(sizeof(T));
  const int step = a.period * ((static_cast<int>(gridDim.x) - kind + a.period - 1) / a.period);  // (CTAs of this kind)
  auto column = [&](int j) { return first_column(j) - shift; };
  float dw[RUNS][8];
#pragma unroll
  for (int i = 0; i < RUNS * 8; ++i) dw[i >> 3][i & 7] = 0.0f;
  Eight<T> w[RUNS];
#pragma unroll
  for (int j = 0; j < RUNS; ++j)
    w[j] = gather_eight(static_cast<const T*>(a.w) + column(j), 1, [&](int e) { return column(j) + e >= 0 && column(j) + e < a.k; });

  // This thread's piece of run j of a row into its place.  A row's first and last piece may reach into its neighbours (their
  // elements are made zeros when the piece has arrived), but not out of the matrix: before row 0 .. 6 or behind the last
  // one (rows have a distance of at least 1) it is gathered.
  auto fill = [&](const void* p, long long ld, int row, int j, uint4* to) {
    const int c = column(j);
    const T* from = static_cast<const T*>(p) + row * ld + c;
    if (EDGES ? (c >= 0 && c + 8 <= a.k) || (c < a.k && (c >= 0 || row > 6) && (a.rows - 1 - row) * ld + a.k >= c + 8) : c < a.k) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
    } else if (EDGES && c < a.k) {
      const Eight<T> v = gather_eight(from, 1, [&](int e) { return c + e >= 0 && c + e < a.k; });
      *to = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    }
  };
  auto send = [&](int row, uint4* to) {
    if (row < a.rows) {
#pragma unroll
      for (int j = 0; j < RUNS; ++j) {
        fill(a.dy, a.lddy, row, j, to + j * threads);
        fill(a.h, a.ldh, row, j, to + matrix + j * threads);
        if (a.dh) fill(a.dh, a.lddh, row, j, to + 2 * matrix + j * threads);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto take = [&](const uint4* from) {
    const uint4 x = *from;
    Eight<T> v;
    v.w[0] = x.x, v.w[1] = x.y, v.w[2] = x.z, v.w[3] = x.w;
    return v;
  };
  int row = kind + a.period * (static_cast<int>(blockIdx.x) / a.period), turn = 0;
  uint4* slot = staged + threadIdx.x;
#pragma unroll
  for (int j = 0; j < RUNS; ++j) {
    if (column(j) < a.k) continue;  // behind the rows: never filled
    for (int i = j * threads; i < kRowsAhead * slot_size; i += matrix) slot[i] = make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kRowsAhead; ++i) send(row + i * step, slot + i * slot_size);
  float r = row < a.rows ? a.rstd[row] : 0.0f;
  for (; row < a.rows; row += step, turn ^= 1) {
    const float rs = r;
    if (row + step < a.rows) r = a.rstd[row + step];
    asm volatile("cp.async.wait_group %0;" ::"n"(kRowsAhead - 1) : "memory");
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const int c = column(j);
      if (EDGES && c < a.k && (c < 0 || c + 8 > a.k)) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint4* at = slot + m * matrix + j * threads;
          Eight<T> v = take(at);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (c + 2 * i < 0 || c + 2 * i >= a.k) v.w[i] &= 0xFFFF0000u;
            if (c + 2 * i + 1 < 0 || c + 2 * i + 1 >= a.k) v.w[i] &= 0xFFFFu;
          }
          *at = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
        }
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const Eight<T> dy = take(slot + j * threads), h = take(slot + matrix + j * threads);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dot = fmaf(dy.get(e) * w[j].get(e), h.get(e), dot);
        dw[j][e] = fmaf(dy.get(e) * rs, h.get(e), dw[j][e]);
      }
    }
    // Two rooms in turn: a warp writes one again only after the other's barrier.
    dot = row_sum(dot, meet[turn]) / static_cast<float>(a.k);
    const float f = rs * rs * dot;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const int c = column(j);
      const Eight<T> dy = take(slot + j * threads), h = take(slot + matrix + j * threads);
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) dx[e] = rs * (dy.get(e) * w[j].get(e) - h.get(e) * f);
      if (a.dh) {
        const Eight<T> dh = take(slot + 2 * matrix + j * threads);
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] += dh.get(e);
      }
      T* to = static_cast<T*>(a.dx) + row * a.lddx + c;
      if (EDGES ? c >= 0 && c + 8 <= a.k : c < a.k) {
        store_eight(to, dx);
      } else if (EDGES) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e >= 0 && c + e < a.k) from_float(dx[e], to[e]);
      }
    }
    send(row + kRowsAhead * step, slot);
    slot = slot == staged + threadIdx.x ? slot + slot_size : slot - slot_size;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* part = a.part + static_cast<long long>(blockIdx.x) * a.k;
#pragma unroll
  for (int j = 0; j < RUNS; ++j) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (column(j) + e >= 0 && column(j) + e < a.k) part[column(j) + e] = dw[j][e];
  }
}

// dw: 32 columns a CTA, 8 warps each a run of parts, added in order.
template <class T>
__global__ void __launch_bounds__(256) norm_weight_kernel(const float* part, int parts, int k, T* dw) {
  __shared__ float sums[8][32];
  let_next_start();
  wait_for_previous();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  float v = 0.0f;
  if (c < k) {
#pragma unroll 4
    for (int i = warp; i < parts; i += 8) v += part[static_cast<long long>(i) * k + c];
  }
  sums[warp][threadIdx.x & 31] = v;
  __syncthreads();
  if (warp == 0 && c < k) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += sums[i][threadIdx.x];
    from_float(v, dw[c]);
  }
}

constexpr int kMaxRows = INT32_MAX - (1 << 20);  // a row's number and a step of all CTAs stay an int

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

struct Shape {
  int threads, rows, runs;  // threads of a row, rows of a CTA, runs a thread
};

// Threads of a row: one run each for few rows (latency), otherwise about 256 threads.
Shape shape_of(int k, bool spread) {
  const int runs_all = (k + 255) / 256 * 32;  // whole warps of runs
  int runs = 1;
  while (runs < 4 && (runs_all / runs > 1024 || (!spread && runs_all / runs > 256))) runs *= 2;
  const int threads = ((runs_all + runs - 1) / runs + 31) / 32 * 32;
  return {threads, threads >= 128 ? 1 : 128 / threads, runs};
}

template <class T, bool VEC>
cudaError_t launch_norm(const NormParams& a, int sms, cudaStream_t stream) {
  Shape s = shape_of(a.k, a.rows < 4 * sms);
  if (s.threads > 32) s.rows = 1;  // (several rows of one warp each need no barrier)
  const int groups = (a.rows + s.rows - 1) / s.rows, threads = s.threads * s.rows;
  const int resident = sms * (threads <= 256 ? 256 / threads : 1) * resident_ctas(VEC, s.runs);
  const bool stay = threads <= 256 && groups > resident;
  cudaError_t e = cudaErrorInvalidValue;
  auto go = [&](void (*kernel)(NormParams)) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(stay ? resident : groups);
    cfg.blockDim = dim3(s.threads, s.rows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) cudaGetLastError();
  };
  switch (s.runs) {
    case 1: go(stay ? norm_kernel<T, VEC, 1, true> : norm_kernel<T, VEC, 1, false>); break;
    case 2: go(stay ? norm_kernel<T, VEC, 2, true> : norm_kernel<T, VEC, 2, false>); break;
    default: go(stay ? norm_kernel<T, VEC, 4, true> : norm_kernel<T, VEC, 4, false>); break;
  }
  return e;
}

template <class T>
cudaError_t norm_of_type(const NormParams& a, int sms, cudaStream_t stream) {
  const bool vec = rows_aligned<T>(a.x, a.ldx, a.rows) && rows_aligned<T>(a.w, 0, 1) &&
                   (!a.residual || rows_aligned<T>(a.residual, a.ldr, a.rows)) && (!a.h || rows_aligned<T>(a.h, a.ldh, a.rows)) &&
                   (!a.y || rows_aligned<T>(a.y, a.ldy, a.rows));
  return vec ? launch_norm<T, true>(a, sms, stream) : launch_norm<T, false>(a, sms, stream);
}

// CTAs of the backward pass: 1024 threads of them an SM, of 152 (64 registers a thread), counted for k columns: rows that are shifted
// have up to 7 more, which can make a warp more (7777 rows of 2049: 288 threads, so three of the four CTAs counted run at once;
// with 56 registers all four do, which leaves the next launch's no room: 54 us a call instead of 41).
int parts_of(int rows, int k) {
  const int threads = shape_of(k, true).threads, most = 152 * (threads >= 128 ? 1024 / threads : 8);
  return rows < most ? rows : most;
}

// The shared-memory limit is the function's, in this context, for all host threads: the most that any launch takes, set once
// (and again should a launch be refused, in a new context after a device reset).
template <class T, int RUNS, bool EDGES>
cudaError_t launch_staged(const NormBackParams& a, int threads, cudaStream_t stream) {
  auto kernel = norm_back_staged_kernel<T, RUNS, EDGES>;
  constexpr int piece = kRowsAhead * RUNS * 16, most = 3 * piece * 1024;
  static std::atomic<bool> ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  for (int attempt = 0; attempt < 2 && e == cudaSuccess; ++attempt) {
    if (attempt || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) break;
      if (dev < 64) ready[dev].store(true, std::memory_order_release);
    }
    e = launch_overlapping(kernel, dim3(a.parts), threads, (a.dh ? 3 : 2) * piece * threads, stream, a);
    if (e != cudaErrorInvalidValue) return e;
    if (!attempt) e = cudaSuccess;
  }
  cudaGetLastError();
  return e;
}

template <class T, bool PIECES>
cudaError_t launch_norm_back(const NormBackParams& a, cudaStream_t stream) {
  // (one row a CTA; a shift takes up to seven columns more)
  const bool shifted = PIECES && (a.period > 1 || (reinterpret_cast<uintptr_t>(a.dy) & 15));
  const Shape s = shape_of(shifted ? a.k + 7 : a.k, true);
  if constexpr (PIECES && sizeof(T) == 2) {
    if (s.runs <= 2) {
      const bool edges = shifted || a.k % 8;
      if (s.runs == 1) return edges ? launch_staged<T, 1, true>(a, s.threads, stream) : launch_staged<T, 1, false>(a, s.threads, stream);
      return edges ? launch_staged<T, 2, true>(a, s.threads, stream) : launch_staged<T, 2, false>(a, s.threads, stream);
    }
  }
  auto kernel = norm_back_kernel<T, PIECES, 4>;
  if constexpr (!(PIECES && sizeof(T) == 2)) kernel = s.runs == 1 ? norm_back_kernel<T, PIECES, 1> : s.runs == 2 ? norm_back_kernel<T, PIECES, 2> : kernel;
  return launch_overlapping(kernel, dim3(a.parts), s.threads, 0, stream, a);
}

template <class T>
cudaError_t norm_back_of_type(NormBackParams a, cudaStream_t stream) {
  // Whether all matrices' rows lie alike against 16 bytes, and after how many rows they do so again.
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.dy) & 15;
  auto alike = [&](const void* p, long long ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == at && (a.rows == 1 || (ld - a.lddy) * static_cast<long long>(sizeof(T)) % 16 == 0);
  };
  // (The widest rows leave no room for a shift.)
  const bool pieces = alike(a.h, a.ldh) && alike(a.dx, a.lddx) && (!a.dh || alike(a.dh, a.lddh)) && a.k + 7 <= OZ_MAX_NORM_WIDTH;
  a.period = 1;
  if (pieces && a.rows > 1) {
    while (a.period < 16 && a.period * a.lddy * static_cast<long long>(sizeof(T)) % 16) a.period *= 2;
  }
  const cudaError_t e = pieces ? launch_norm_back<T, true>(a, stream) : launch_norm_back<T, false>(a, stream);
  if (e != cudaSuccess) return e;
  return launch_overlapping(norm_weight_kernel<T>, dim3((a.k + 31) / 32), 256, 0, stream, a.part, a.parts, a.k, static_cast<T*>(a.dw));
}

int check_back(int k, int rows, int dtype, long long lddy, long long ldh, long long lddh, long long lddx) {
  if (k < 0 || rows < 0 || rows > kMaxRows || k > OZ_MAX_NORM_WIDTH || !element_bytes(dtype)) return OZ_EINVAL;
  const long long least = k > 1 ? k : 1;
  return lddy < least || ldh < least || lddh < least || lddx < least ? OZ_EINVAL : OZ_OK;
}

int norm_back(int k, int rows, int dtype, const void* dY, int lddy, const void* H, int ldh, const void* W, const float* rstd,
              const void* dH, int lddh, void* dX, int lddx, void* dW, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (k == 0) return OZ_OK;
  if (!dW || !element_aligned(dW, dtype)) return OZ_EINVAL;
  if (rows == 0) return cudaMemsetAsync(dW, 0, element_bytes(dtype) * k, stream) == cudaSuccess ? OZ_OK : OZ_ECUDA;
  for (const void* p : {dY, H, W, static_cast<const void*>(dX)})
    if (!p || !element_aligned(p, dtype)) return OZ_EINVAL;
  if (!rstd || (reinterpret_cast<uintptr_t>(rstd) & 3) || !element_aligned(dH, dtype)) return OZ_EINVAL;
  const NormBackParams a{k, rows, dY, H, W, dH, rstd, dX, dW, lddy, ldh, lddh, lddx, static_cast<float*>(workspace), parts_of(rows, k), 1};
  if (!workspace || ws_bytes < sizeof(float) * static_cast<size_t>(k) * a.parts || (reinterpret_cast<uintptr_t>(workspace) & 255)) return OZ_ENOMEM;
  const cudaError_t e = dtype == OZ_BF16 ? norm_back_of_type<__nv_bfloat16>(a, stream)
                        : dtype == OZ_F16 ? norm_back_of_type<__half>(a, stream)
                                          : norm_back_of_type<float>(a, stream);
  return e == cudaSuccess ? OZ_OK : OZ_ECUDA;
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

int ozaki_rms_norm_f8(int k, int rows, int dtype, const void* X, int ldx, const void* residual, int ldr, const void* W, float eps,
                      void* Q, int ldq, float* S, int lds, void* H, int ldh, float* rstd, void* Y, int ldy, cudaStream_t stream) {
  if (k < 0 || rows < 0 || rows > kMaxRows || k > OZ_MAX_NORM_WIDTH || !element_bytes(dtype) || !(eps >= 0.0f)) return OZ_EINVAL;
  const int least = k > 1 ? k : 1;
  if (ldx < least || ldr < least || ldh < least || ldy < least || ldq < least || lds < (rows > 1 ? rows : 1)) return OZ_EINVAL;
  if (k == 0 || rows == 0) return OZ_OK;
  if (!X || !W || !Q || !S || !rstd || (reinterpret_cast<uintptr_t>(Q) & 15) || (rows > 1 && ldq % 16)) return OZ_EINVAL;
  if ((reinterpret_cast<uintptr_t>(S) & 3) || (reinterpret_cast<uintptr_t>(rstd) & 3)) return OZ_EINVAL;
  for (const void* p : {X, residual, W, static_cast<const void*>(H), static_cast<const void*>(Y)})
    if (!element_aligned(p, dtype)) return OZ_EINVAL;
  const int sms = sm_count();
  if (!sms) return OZ_ECUDA;
  const NormParams a{k, rows, X, residual, W, H, Y, static_cast<uint8_t*>(Q), S, rstd, ldx, ldr, ldh, ldy, ldq, lds, eps};
  const cudaError_t e = dtype == OZ_BF16 ? norm_of_type<__nv_bfloat16>(a, sms, stream)
                        : dtype == OZ_F16 ? norm_of_type<__half>(a, sms, stream)
                                          : norm_of_type<float>(a, sms, stream);
  return e == cudaSuccess ? OZ_OK : OZ_ECUDA;
}

size_t ozaki_rms_norm_backward_workspace_bytes(int k, int rows) {
  if (check_back(k, rows, OZ_F32, k > 1 ? k : 1, k > 1 ? k : 1, k > 1 ? k : 1, k > 1 ? k : 1)) return 0;
  return sizeof(float) * static_cast<size_t>(k) * parts_of(rows, k);
}
int ozaki_rms_norm_backward_ws(int k, int rows, int dtype, const void* dY, int lddy, const void* H, int ldh, const void* W,
                               const float* rstd, const void* dH, int lddh, void* dX, int lddx, void* dW, void* workspace,
                               size_t ws_bytes, cudaStream_t stream) {
  const int rc = check_back(k, rows, dtype, lddy, ldh, lddh, lddx);
  return rc ? rc : norm_back(k, rows, dtype, dY, lddy, H, ldh, W, rstd, dH, lddh, dX, lddx, dW, workspace, ws_bytes, stream);
}
int ozaki_rms_norm_backward(int k, int rows, int dtype, const void* dY, int lddy, const void* H, int ldh, const void* W,
                            const float* rstd, const void* dH, int lddh, void* dX, int lddx, void* dW, cudaStream_t stream) {
  int rc = check_back(k, rows, dtype, lddy, ldh, lddh, lddx);
  if (rc) return rc;
  const bool operands = dY && H && W && rstd && dX && dW;  // argument errors before any allocation
  const size_t bytes = operands ? ozaki_rms_norm_backward_workspace_bytes(k, rows) : 0;
  void* ws = nullptr;
  if (bytes) {
    keep_default_pool_cached();
    if (cudaMallocAsync(&ws, bytes, stream) != cudaSuccess) {
      cudaGetLastError();
      return OZ_ENOMEM;
    }
  }
  rc = norm_back(k, rows, dtype, dY, lddy, H, ldh, W, rstd, dH, lddh, dX, lddx, dW, ws, bytes, stream);
  if (ws && cudaFreeAsync(ws, stream) != cudaSuccess && rc == OZ_OK) rc = OZ_ECUDA;
  return rc;
}

}  // extern "C"
