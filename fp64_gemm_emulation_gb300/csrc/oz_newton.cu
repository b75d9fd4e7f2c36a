// oz_newton.cu -- Newton-Schulz orthogonalisation of matrices on the tensor cores.
//
//   X_0 = G / (|G|_F + eps),   X_{i+1} = a X_i + (b A + c A^2) X_i,   A = X_i X_i^T
// (X_i^T X_i on the right when G has more rows than columns).  Completing the square,
//   S = A + (b / 2c) I,   B = c S^2 + (a - b^2 / 4c) I,   X_{i+1} = B X_i,
// makes a step three plain products whose epilogues only scale and add to the diagonal, so no
// epilogue reads a matrix back.  (c = 0: B = b A + a I comes out of the first product.)
// S and B are symmetric: only tiles that reach the lower triangle are computed, and mirrored.
//
// All products of all steps run in ONE cooperative launch (ChainWalk): the units of the products
// follow each other in the same order on every CTA pair, and a unit's producer waits until the
// product before it is finished for its own matrix (a counter per matrix in global memory).  So the
// matrices of a batch do not wait for one another, and a product boundary costs a flag instead of
// a launch (a launch a product took 3.7 us each at 128 x 128, for 1.5 us of work).
//
// Numerics.  The products run on the FP16 tensor-core path: FP16 holds 11 bits where bf16
// holds 8, at the same rate, and every range is known beforehand: |X_0| <= 1, and a host-side
// bound on the polynomial bounds the singular values of every X_i, S and B, so each is stored
// times a power of two that fills FP16's range.  |G|_F is divided out as a power of two (exact
// on bf16 inputs); the remaining factor in [1, 2) joins the first step's scalings.  With two
// slices each matrix is h + l in FP16 (22 bits), and a product is h h' + h l' + l h'.  All sums
// are FP32; the norm's partial sums are joined in FP64.
#include <cmath>

#include "oz_newton.h"
#include "oz_products.cuh"

namespace oz {
namespace {

using namespace prod;

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

constexpr int kNormBlocks = 304;       // partial sums of a matrix's norm, at most
constexpr int kMaxParts = 160;         // parts of split tiles that a product's workspace holds
// Two slices: MMA steps (16 k) summed on the tensor core before the sum moves to FP32 registers.
// The tensor core truncates each addition, which biases long sums, so the result's relative error (five
// steps, against 64 bits) grows with the steps of a sum, while the epilogue's work shrinks:
//                  single steps        k-blocks (4 steps)    plain FP32
//   128 x 300      0.95e-6   124 us    2.0e-6     96 us      1.6e-6
//   512 x 512      1.3e-6    170 us    2.8e-6    123 us      2.1e-6
//   1023 x 2777    1.2e-6    509 us    2.3e-6    281 us      3.7e-6
//   8192 x 2048    1.4e-6   2.58 ms    2.1e-6   1.35 ms      4.5e-6
// K-blocks keep it below plain FP32's from a side of about 1000 on, and within 1.4 times that below.  Where the
// smaller side is at most 128, S^2 is taken in single steps, which alone is enough: 128 x 300 1.1e-6 and 104 us.

// The products of a step.
enum Kind { kGram = 0, kSquare = 1, kApply = 2 };

struct Product {
  CUtensorMap mapA[2], mapB[2];  // by the parity of the step (which of the two X)
  int M, N, K, bn;
  int chunk;                     // MMA steps of a sum (two slices)
  int tiles_m, tiles_n, tiles;   // of one matrix (symmetric: those that reach the lower triangle)
  int full, nsplit, units;       // tiles of the batch that are not split, parts of the others, units in all
  int a_mn, b_mn, sym;
  uint32_t idesc;
  float* part;
  unsigned int* arrivals;

  // Symmetric: tiles of row tile tm, those that reach n <= m.
  __host__ __device__ int sym_tiles(int tm) const {
    const int c = ceil_div((tm + 1) * BM, bn);
    return c < tiles_n ? c : tiles_n;
  }
};

// Deals out the units of every product of every step, in that order.
template <int PLANES>
struct ChainWalk {
  static constexpr bool kScaled = true, kChained = true;
  static constexpr int kEpiWarps = PLANES == 2 ? 12 : 8;
  static constexpr size_t kTableBytes = 0;

  struct Params {
    Product prod[3];
    int batch, steps;
    int scout;                    // a warp runs ahead of the producer (product_kernel)
    void *X[2], *S, *B, *O;
    long long xplane, splane, ldx, lds, ldo, stride_o;
    int out_type, vec_o;
    const float* scales;          // [matrix][step][2]: factors of the first and the last product
    float diag_s[OZ_MAX_NS_STEPS], alpha_b[OZ_MAX_NS_STEPS], diag_b[OZ_MAX_NS_STEPS];
    unsigned int square;          // bit i: step i has the middle product (c != 0)
    unsigned int* finished;       // [matrix]: CTAs that have finished a tile, over all products
    unsigned int* stopped;        // a pair of this launch gave up
    int* status;
    unsigned long long epi_wait_ns;
  };

  const Params& a;
  int idx, base, step, kind, group;
  unsigned int need;  // a matrix's count when the products before this one are finished

  __device__ static void setup(const Params& a, int*) {
    if (threadIdx.x < 12) {
      const Product& p = a.prod[threadIdx.x >> 2];
      tma_prefetch_desc((threadIdx.x & 2) ? &p.mapB[threadIdx.x & 1] : &p.mapA[threadIdx.x & 1]);
    }
    wait_for_previous();
  }

  __device__ ChainWalk(const Params& p, const int*)
      : a(p), idx(static_cast<int>(blockIdx.x >> 1) - static_cast<int>(gridDim.x >> 1)), base(0), step(0), kind(kGram),
        group(0), need(0) {}

  __device__ int units() const { return kind == kSquare && !(a.square >> step & 1) ? 0 : a.prod[kind].units; }

  __device__ bool next(Unit& u) {
    idx += static_cast<int>(gridDim.x >> 1);
    for (int n = units(); idx - base >= n; n = units()) {  // on to the unit's product
      base += n;
      if (n) need += a.prod[kind].tiles * 2;  // both CTAs report a tile
      if (kind == kApply) {
        kind = kGram;
        if (++step == a.steps) return false;
      } else {
        ++kind;
      }
    }
    describe(u);
    return true;
  }

  __device__ void describe(Unit& u) {
    const Product& p = a.prod[kind];
    int tile = idx - base;
    u.split = 0;
    u.nsplit = 1;
    u.part = p.part;
    u.part_cols = p.bn;
    u.arrivals = p.arrivals;
    if (tile >= p.full && p.nsplit > 1) {
      const int q = tile - p.full, r = q / p.nsplit;
      tile = p.full + r;
      u.split = q - r * p.nsplit;
      u.nsplit = p.nsplit;
      u.part = p.part + 2ll * r * p.nsplit * p.bn * HALF_M;
      u.arrivals = p.arrivals + 2 * r;
    }
    group = tile / p.tiles;
    int r = tile - group * p.tiles, tm, tn;
    if (p.sym) {  // row tile tm has the column tiles that reach n <= m
      tm = 0;
      for (int c = p.sym_tiles(0); r >= c; c = p.sym_tiles(tm)) {
        r -= c;
        ++tm;
      }
      tn = r;
    } else {  // groups of 8 row tiles swept along the column tiles (L2 reuse of both operands)
      const int g = r / (8 * p.tiles_n), gm = min(8, p.tiles_m - 8 * g);
      r -= g * 8 * p.tiles_n;
      tn = r / gm;
      tm = 8 * g + r - tn * gm;
    }
    u.m0 = tm * BM;
    u.n0 = u.orow = tn * p.bn;
    u.nn = min(p.bn, p.N - u.n0);
    const int nkb = ceil_div(p.K, BK);
    u.k0 = 0;
    u.chunk = p.chunk;
    u.kb0 = nkb * u.split / u.nsplit;
    u.kb1 = nkb * (u.split + 1) / u.nsplit;
    u.a_mn = p.a_mn;
    u.b_mn = p.b_mn;
    u.a_4d = true;
    u.b_4d = p.bn % 128 == 0;  // (MN-major) the CTA's half is whole blocks of 64
    u.nmma = p.b_mn ? p.bn : ceil_div(u.nn, 32) * 32;
    u.mapA = &p.mapA[step & 1];
    u.mapB = &p.mapB[step & 1];
    u.boxes = p.b_mn && !u.b_4d ? ceil_div(p.bn / 2, 64) : 1;
    u.box_b = p.bn / 2;
    u.b_plane = !p.b_mn ? p.bn / 2 * BK * 2 : p.bn / 128 * MN_BLOCK;
    u.box_bytes = !p.b_mn || u.b_4d ? PLANES * u.b_plane : MN_BLOCK;
    u.zA = u.zB = group * PLANES;
    u.idesc = p.idesc;
    u.m_extent = p.M;
    u.sym = p.sym;
    u.planes_out = PLANES;
    u.out_type = kOutSlices;
    u.vec = true;
    u.diag = 0.0f;
    const long long sc = 2ll * (group * a.steps + step);
    if (kind == kApply) {  // X_{i+1} 2^t' = 2^(t' - t - sb) (B 2^sb)(X_i 2^t)
      u.f = a.scales[sc + 1];
      if (step + 1 == a.steps) {
        u.out = static_cast<uint8_t*>(a.O) + group * a.stride_o * (a.out_type == kOutF32 ? 4 : 2);
        u.ld = a.ldo;
        u.plane = 0;
        u.planes_out = 1;
        u.out_type = a.out_type;
        u.vec = a.vec_o;
      } else {
        u.out = static_cast<uint16_t*>(a.X[(step & 1) ^ 1]) + group * PLANES * a.xplane;
        u.ld = a.ldx;
        u.plane = a.xplane;
      }
    } else {
      const bool to_s = kind == kGram && (a.square >> step & 1);
      u.f = kind == kGram ? a.scales[sc] : a.alpha_b[step];
      u.diag = to_s ? a.diag_s[step] : a.diag_b[step];
      u.out = static_cast<uint16_t*>(to_s ? a.S : a.B) + group * PLANES * a.splane;
      u.ld = a.lds;
      u.plane = a.splane;
    }
  }

  // Waits until the products before the unit's are finished for its matrix.  They were dealt out
  // earlier to pairs that are all running (cooperative launch).  What those pairs stored is then
  // ordered before this thread's TMA loads (generic to async proxy).
  __device__ bool ready(const volatile int* abort_flag) const {
    if (need == 0) return true;
    const unsigned int* count = a.finished + group;
    auto reached = [&]() {
      unsigned int v;
      asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
      return static_cast<int>(v - need) >= 0;
    };
    if (!reached()) {
      const uint64_t t0 = globaltimer_ns();
      for (int i = 1; !reached(); ++i) {
        if (*abort_flag) return false;
        if ((i & 63) == 0 && (*reinterpret_cast<const volatile unsigned int*>(a.stopped) || globaltimer_ns() - t0 > kWaitLimitNs)) {
          atomicExch(a.stopped, 1u);
          return false;
        }
      }
    }
    asm volatile("fence.acq_rel.gpu;\n\tfence.proxy.async;" ::: "memory");
    return true;
  }

  // A CTA has stored its half of a finished tile.
  __device__ void done() const {
    asm volatile("red.relaxed.gpu.global.add.u32 [%0], %1;" ::"l"(a.finished + group), "r"(1u) : "memory");
  }

  // This pair has given up: the others' waits end.
  __device__ static void gave_up(const Params& a) { atomicExch(a.stopped, 1u); }
};

__device__ __forceinline__ float load_value(const void* p, long long i, int dtype) {
  if (dtype == OZ_F32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == OZ_BF16 ? __bfloat162float(__ushort_as_bfloat16(h)) : __half2float(__ushort_as_half(h));
}

// partial[matrix][block]: the three sums of SumSquares.
__global__ void __launch_bounds__(256) norm_kernel(const void* __restrict__ G, int dtype, int cols, long long rows,
                                                   long long ld, long long stride, double* __restrict__ partial,
                                                   unsigned* __restrict__ counters, int ncounters) {
  let_next_start();
  wait_for_previous();
  if (blockIdx.y == 0)
    for (int i = blockIdx.x * 256 + threadIdx.x; i < ncounters; i += gridDim.x * 256) counters[i] = 0;
  const long long base = blockIdx.y * stride;
  SumSquares sq;
  auto add = [&](float x) { sq.add(x); };
  const bool dense = ld == cols && (reinterpret_cast<uintptr_t>(G) & 15) == 0 && stride % 8 == 0;
  if (dense) {  // 16-byte loads over the whole matrix
    const long long n = rows * cols;
    const int per = dtype == OZ_F32 ? 4 : 8;
    const long long nv = n / per;
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(G) + base * (dtype == OZ_F32 ? 4 : 2));
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < nv; i += gridDim.x * 256ll) {
      const uint4 w = __ldg(v + i);
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
      const float before = sq.mid;  // the vector's squares are summed by themselves first
      sq.mid = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (dtype == OZ_F32) {
          add(__uint_as_float(q[e]));
        } else if (dtype == OZ_BF16) {
          add(__uint_as_float(q[e] << 16));
          add(__uint_as_float(q[e] & 0xFFFF0000u));
        } else {
          add(__half2float(__ushort_as_half(static_cast<uint16_t>(q[e]))));
          add(__half2float(__ushort_as_half(static_cast<uint16_t>(q[e] >> 16))));
        }
      }
      sq.mid += before;
    }
    for (long long i = nv * per + blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll)
      add(load_value(G, base + i, dtype));
  } else {
    for (long long r = blockIdx.x; r < rows; r += gridDim.x)
      for (int c = threadIdx.x; c < cols; c += 256) add(load_value(G, base + r * ld + c, dtype));
  }
  __shared__ double sums[3][8];
  double s[3] = {sq.big, sq.mid, sq.small};
#pragma unroll
  for (int j = 0; j < 3; ++j) {
#pragma unroll
    for (int d = 16; d; d >>= 1) s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], d);
    if ((threadIdx.x & 31) == 0) sums[j][threadIdx.x >> 5] = s[j];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    double t = 0.0;
    for (int w = 0; w < 8; ++w) t += sums[threadIdx.x][w];
    partial[(static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * 3 + threadIdx.x] = t;
  }
}

// X_0 as FP16 slices, and the factors of the products (newton_scales).
__global__ void __launch_bounds__(256) convert_kernel(const void* __restrict__ G, int dtype, int cols, long long rows,
                                                      long long ld, long long stride, const double* __restrict__ partial,
                                                      int nblocks, float eps, const __grid_constant__ NewtonPlan plan,
                                                      uint16_t* __restrict__ X, int ldx, long long plane, int planes,
                                                      float* __restrict__ scales) {
  __shared__ float s_mul[2];
  let_next_start();
  wait_for_previous();
  if (threadIdx.x < 32) {
    double s[3] = {0.0, 0.0, 0.0};
    const double* p = partial + static_cast<long long>(blockIdx.y) * nblocks * 3;
    for (int b = threadIdx.x; b < nblocks; b += 32)
      for (int j = 0; j < 3; ++j) s[j] += p[b * 3 + j];
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
      for (int d = 16; d; d >>= 1) s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], d);
    newton_scales(static_cast<float>(s[0]), static_cast<float>(s[1]), static_cast<float>(s[2]), eps, plan, s_mul,
                  blockIdx.x == 0 ? scales + static_cast<long long>(blockIdx.y) * 2 * plan.steps : nullptr);
  }
  __syncthreads();
  const float f0 = s_mul[0], f1 = s_mul[1];
  const long long base = blockIdx.y * stride;
  X += static_cast<long long>(blockIdx.y) * planes * plane;
  const int per = ldx / 8;  // 8 elements of a row for each thread (ldx is a multiple of 8)
  const long long total = rows * per;
  const int size = dtype == OZ_F32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(G) & 15) == 0 && ld * size % 16 == 0 && stride * size % 16 == 0;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const long long row = i / per;
    const int c = static_cast<int>(i - row * per) * 8;
    const long long at = base + row * ld + c;
    float v[8];
    if (vec && c + 8 <= cols) {
      if (dtype == OZ_F32) {
        const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(G) + at);
        const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(G) + at + 4);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
      } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(G) + at);
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint16_t h = static_cast<uint16_t>(q[e >> 1] >> (16 * (e & 1)));
          v[e] = dtype == OZ_BF16 ? __bfloat162float(__ushort_as_bfloat16(h)) : __half2float(__ushort_as_half(h));
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = c + e < cols ? load_value(G, at + e, dtype) : 0.0f;
    }
    for (int p = 0; p < planes; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = p ? v[e] : v[e] * f0 * f1;
        const __half h = __float2half_rn(x);
        v[e] = x - __half2float(h);
        const uint32_t bits = __half_as_ushort(h);
        w[e >> 1] = (e & 1) ? w[e >> 1] | (bits << 16) : bits;
      }
      *reinterpret_cast<uint4*>(X + p * plane + row * ldx + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

int room(double bound) { return static_cast<int>(std::floor(std::log2(60000.0 / bound))); }

// OZ_ERANGE if the singular values may leave the range in which the scales keep 11 (22) bits
// useful: a bound above 16 on X, or a square whose completion cancels more than 4 bits.
int make_plan(int steps, const float* coeffs, NewtonPlan* out) {
  NewtonPlan p{};
  p.steps = steps;
  double bound = 1.0, worst = 1.0, gain = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double a = coeffs[3 * i], b = coeffs[3 * i + 1], c = coeffs[3 * i + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return OZ_EINVAL;
    const bool square = c != 0.0;
    if (square) p.square |= 1u << i;
    const double beta = square ? b / (2 * c) : 0.0;
    const double top = bound * 1.02, l_top = top * top;  // 2 %: rounding of the stored matrices
    // Maxima over [0, top] at the ends and where the derivative vanishes: of p(l) at l = -b/2c,
    // of s p(s^2) where a + 3 b l + 5 c l^2 = 0.
    auto p_at = [&](double l) { return std::fabs(a + b * l + c * l * l); };
    double p_max = std::fmax(p_at(0.0), p_at(l_top));
    double x_max = top * p_at(l_top);
    double s_max = std::fmax(std::fabs(beta), std::fabs(l_top + beta));
    auto stationary = [&](double l) {
      if (l > 0.0 && l < l_top) x_max = std::fmax(x_max, std::sqrt(l) * p_at(l));
    };
    if (square) {
      if (-beta > 0.0 && -beta < l_top) p_max = std::fmax(p_max, p_at(-beta));
      const double d = 9 * b * b - 20 * a * c;
      if (d >= 0.0) {
        stationary((-3 * b + std::sqrt(d)) / (10 * c));
        stationary((-3 * b - std::sqrt(d)) / (10 * c));
      }
    } else if (b != 0.0) {
      stationary(-a / (3 * b));
    }
    p_max *= 1.01;
    x_max *= 1.01;
    s_max *= 1.01;
    if (!(x_max <= 16.0) || !(p_max <= 1024.0) || p_max == 0.0) return OZ_ERANGE;
    p.sb[i] = room(p_max);
    if (square) {
      if (std::fabs(c) * s_max * s_max > 16.0 * p_max) return OZ_ERANGE;
      const int sa = room(s_max);
      p.gram[i] = static_cast<float>(std::ldexp(1.0, sa));
      p.diag_s[i] = static_cast<float>(std::ldexp(beta, sa));
      p.alpha_b[i] = static_cast<float>(std::ldexp(c, p.sb[i] - 2 * sa));
      p.diag_b[i] = static_cast<float>(std::ldexp(a - b * beta / 2, p.sb[i]));
    } else {
      p.gram[i] = static_cast<float>(std::ldexp(b, p.sb[i]));
      p.diag_b[i] = static_cast<float>(std::ldexp(a, p.sb[i]));
    }
    bound = std::fmax(x_max, 1e-3);
    worst = std::fmax(worst, x_max);
    gain = std::fmax(gain, p_max);
  }
  p.sx = room(worst) < 14 ? room(worst) : 14;
  p.drop = static_cast<int>(std::ceil(std::log2(gain)));
  *out = p;
  return OZ_OK;
}

struct Shape {
  int cols, rows, batch, planes, side;  // contiguous extent, rows; side: the smaller
  int ldx, lds;
  bool wide;                            // rows <= cols
  size_t x_bytes, s_bytes;
  int norm_blocks;
  Shape(int m, int n, int b, int slices) : cols(m), rows(n), batch(b), planes(slices) {
    wide = rows <= cols;
    side = wide ? rows : cols;
    ldx = static_cast<int>(roundup(cols, 64));
    lds = static_cast<int>(roundup(side, 64));
    x_bytes = align256(2 * static_cast<size_t>(batch) * planes * rows * ldx);
    s_bytes = align256(2 * static_cast<size_t>(batch) * planes * side * lds);
    const long long per = (static_cast<long long>(rows) * cols + 8191) / 8192;
    norm_blocks = static_cast<int>(per < kNormBlocks ? per : kNormBlocks);
  }
  size_t part_bytes() const { return align256(sizeof(float) * 2 * HALF_M * BN * kMaxParts); }  // of one product
  int words() const { return 3 * 2 * kMaxParts + 1 + batch; }  // arrivals, stopped, finished
  size_t total() const {
    if (newton_is_small(rows, cols, planes)) return 0;
    return 2 * x_bytes + 2 * s_bytes + 3 * part_bytes() + align256(sizeof(unsigned) * words()) +
           align256(sizeof(double) * 3 * norm_blocks * batch) + align256(sizeof(float) * 2 * OZ_MAX_NS_STEPS * batch);
  }
};

// Tile width and parts of split tiles for one product, by a model of its time in SM cycles.  Cycles
// of a k-block as measured at 8192^2: one slice is bound by what the SM can load (59 bytes a cycle:
// 558 at 256 columns, 413 at 128, 371 at 64), two slices by the MMAs and their issue; single-step
// chunks by the epilogue.
//   One or two matrices, or a single wave: the waves, the last one's drain, and the joining of parts.
//   More: the matrices do not wait for one another, so a wave that one product leaves open is filled by
//     the next one.  A product then costs the larger of its work and its latency (what one matrix
//     waits), and some of the other; splitting gains nothing.  (Counted in waves as for one matrix / so:
//     64 x 256 x 1024 bf16 246 / 187 us, 16 x 2048 x 1024 635 / 575, FP32 1940 / 1841.)
void plan_product(Product& p, int batch, int planes, int pairs) {
  const int nkb = ceil_div(p.K, BK);
  double best = 1e30;
  Product q = p;
  for (int bn = planes == 2 ? BN2 : BN; bn >= 64; bn -= 32) {
    if (planes == 2 && p.b_mn && bn != 128) continue;  // both slices in one box: whole blocks of 64
    if (p.b_mn && bn < 128) break;
    q.bn = bn;
    q.tiles_m = ceil_div(p.M, BM);
    q.tiles_n = ceil_div(p.N, bn);
    q.tiles = q.tiles_m * q.tiles_n;
    if (p.sym) {
      q.tiles = 0;
      for (int i = 0; i < q.tiles_m; ++i) q.tiles += q.sym_tiles(i);
    }
    const long long all = static_cast<long long>(q.tiles) * batch;
    double block = planes == 1 ? 310 + bn : 200 + 5.2 * bn;
    if (planes == 2 && p.chunk == 1) block = KSTEPS * (300.0 + 2 * bn);
    // The epilogue of a tile runs under the next tile's MMAs; that of the last one shows.
    const double drain = bn / 64.0 * (planes == 2 ? 800 : p.sym ? 1900 : 1150);
    const int rest = static_cast<int>(all % pairs);
    const bool shared = batch > 2 && all > pairs;  // products share their waves
    for (int s = 1; s <= 16 && s <= nkb; ++s) {
      if (s > 1 && (rest == 0 || rest * s > kMaxParts || shared)) break;
      const double unit = ceil_div(nkb, s) * block, join = 2500.0 * (bn / 256.0) * (1 + s);
      double t;
      if (!shared) {
        t = static_cast<double>(all / pairs) * std::fmax(nkb * block, drain) + drain + 2500;
        if (rest) t += ceil_div(rest * s, pairs) * unit;
        // parts: each wave's are written out, and the last reads them all (1024 x 4096 FP32: one wave of
        // three parts 379 us, two waves of five 430)
        if (s > 1) t += 3000 + join + ceil_div(rest * s, pairs) * (2500 + 16.0 * bn);
      } else {
        const double step = planes == 2 ? unit + drain + 3000 : std::fmax(unit, drain + 3000);
        const double work = static_cast<double>(all) / pairs * step;
        const double latency = ceil_div(q.tiles, pairs) * unit + drain + 3000;
        t = std::fmax(work, latency) + 0.3 * std::fmin(work, latency);
      }
      if (t < best) {
        best = t;
        q.nsplit = s;
        q.full = s > 1 ? static_cast<int>(all - rest) : static_cast<int>(all);
        q.units = q.full + (s > 1 ? rest * s : 0);
        p = q;
      }
    }
  }
}

int check(int m, int n, int batch, int dtype, int ldg, long long stride_g, int ldo, long long stride_o,
          int steps, const float* coeffs, float eps, int slices) {
  if (m < 0 || n < 0 || batch < 0 || m > kMaxExtent || n > kMaxExtent) return OZ_EINVAL;
  if (dtype != OZ_BF16 && dtype != OZ_F16 && dtype != OZ_F32) return OZ_EINVAL;
  if (ldg < (m > 1 ? m : 1) || ldo < (m > 1 ? m : 1)) return OZ_EINVAL;
  if (batch > 1 && (stride_g < static_cast<long long>(ldg) * n || stride_o < static_cast<long long>(ldo) * n))
    return OZ_EINVAL;
  if (steps < 1 || steps > OZ_MAX_NS_STEPS || !coeffs || slices < 1 || slices > 2) return OZ_EINVAL;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return OZ_EINVAL;
  if (batch > 65535) return OZ_EINVAL;
  return OZ_OK;
}

template <int PLANES>
int run_chain(const Shape& sh, const NewtonPlan& plan, uint16_t* const (&X)[2], uint16_t* S, uint16_t* B, float* part,
              unsigned* words, const float* scales, void* O, int dtype, int ldo, long long stride_o, const Device& dev,
              cudaStream_t stream) {
  typedef ChainWalk<PLANES> Walk;
  typename Walk::Params a{};
  const int side = sh.side, long_side = sh.wide ? sh.cols : sh.rows;
  a.batch = sh.batch;
  a.steps = plan.steps;
  a.X[0] = X[0];
  a.X[1] = X[1];
  a.S = S;
  a.B = B;
  a.O = O;
  a.xplane = static_cast<long long>(sh.rows) * sh.ldx;
  a.splane = static_cast<long long>(side) * sh.lds;
  a.ldx = sh.ldx;
  a.lds = sh.lds;
  a.ldo = ldo;
  a.stride_o = stride_o;
  a.out_type = dtype == OZ_F32 ? kOutF32 : dtype == OZ_BF16 ? kOutBf16 : kOutF16;
  a.vec_o = (reinterpret_cast<uintptr_t>(O) & 15) == 0 && ldo % 8 == 0 && (sh.batch == 1 || stride_o % 8 == 0);
  a.scales = scales;
  a.square = plan.square;
  for (int i = 0; i < a.steps; ++i) {
    a.diag_s[i] = plan.diag_s[i];
    a.alpha_b[i] = plan.alpha_b[i];
    a.diag_b[i] = plan.diag_b[i];
  }
  a.stopped = words + 3 * 2 * kMaxParts;
  a.finished = a.stopped + 1;

  //                 m side, n side, sum
  Product &g = a.prod[kGram], &q = a.prod[kSquare], &x = a.prod[kApply];
  g.M = g.N = q.M = q.N = q.K = x.K = side;
  g.K = long_side;
  x.M = sh.cols;
  x.N = sh.rows;
  g.sym = q.sym = 1;
  g.a_mn = g.b_mn = !sh.wide;  // wide: X X^T, both along its rows; tall: X^T X, both across them
  x.a_mn = sh.wide;            // wide: D[col, row] = sum_j X[j, col] B[row, j]; tall: sum_j B[col, j] X[row, j]
  long long units = 0;
  for (int i = 0; i < 3; ++i) {
    Product& p = a.prod[i];
    p.chunk = i == kSquare && side <= 128 ? 1 : KSTEPS;
    plan_product(p, sh.batch, PLANES, dev.pairs);
    p.idesc = idesc_base(false, p.a_mn, p.b_mn);
    p.part = part + i * (sh.part_bytes() / sizeof(float));
    p.arrivals = words + i * 2 * kMaxParts;
    units += static_cast<long long>(p.units) * a.steps;
    if (static_cast<long long>(p.tiles) * sh.batch > INT32_MAX / 64 || units > INT32_MAX / 2) return OZ_EINVAL;
  }

  const uint64_t mats = static_cast<uint64_t>(sh.batch) * PLANES, xl = 2ull * sh.ldx, sl = 2ull * sh.lds;
  auto s_map = [&](CUtensorMap* t, const void* base, int box) {
    return make_map(t, base, false, side, side, mats, sl, 2ull * a.splane, box, PLANES);
  };
  auto x_map = [&](CUtensorMap* t, int i, int box) {
    return make_map(t, X[i], false, sh.cols, sh.rows, mats, xl, 2ull * a.xplane, box, PLANES);
  };
  // Rows of ldx, a multiple of 64 (so the map is 4-D): the padding past the last column is the
  // workspace's own, and what is read there only reaches output elements that are never stored.
  auto mn_map = [&](CUtensorMap* t, int i, int blocks) {
    int is_4d = 0;
    return make_mn_map(t, &is_4d, blocks, X[i], false, sh.ldx, sh.rows, mats, xl, 2ull * a.xplane, PLANES) && is_4d;
  };
  bool ok = true;
  for (int i = 0; i < 2 && ok; ++i) {
    ok = s_map(&q.mapA[i], S, HALF_M) && s_map(&q.mapB[i], S, q.bn / 2);
    if (sh.wide)
      ok = ok && x_map(&g.mapA[i], i, HALF_M) && x_map(&g.mapB[i], i, g.bn / 2) && mn_map(&x.mapA[i], i, 2) &&
           s_map(&x.mapB[i], B, x.bn / 2);
    else
      ok = ok && mn_map(&g.mapA[i], i, 2) &&
           (g.bn % 128 ? x_map(&g.mapB[i], i, BK) : mn_map(&g.mapB[i], i, g.bn / 128)) && s_map(&x.mapA[i], B, HALF_M) &&
           x_map(&x.mapB[i], i, x.bn / 2);
  }
  if (!ok) return OZ_ECUDA;
  int most = g.units > x.units ? g.units : x.units;
  if (a.square && q.units > most) most = q.units;
  a.scout = most > dev.pairs;
  return launch<Walk, PLANES>(a, dev, most < dev.pairs ? most : dev.pairs, kCooperative, stream);
}

int run(int m, int n, int batch, int dtype, const void* G, int ldg, long long stride_g, void* O, int ldo,
        long long stride_o, const NewtonPlan& plan, float eps, int slices, void* workspace, size_t ws_bytes,
        cudaStream_t stream) {
  if (newton_is_small(n, m, slices))
    return launch_newton_small(n, m, batch, dtype, G, ldg, stride_g, O, ldo, stride_o, plan, eps, slices, stream);
  const Shape sh(m, n, batch, slices);
  if (!workspace || ws_bytes < sh.total() || (reinterpret_cast<uintptr_t>(workspace) & 255)) return OZ_ENOMEM;
  Device dev;
  int rc;
  if ((rc = current_device(&dev))) return rc;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  auto take = [&](size_t bytes) {
    uint8_t* p = at;
    at += align256(bytes);
    return p;
  };
  uint16_t* X[2] = {reinterpret_cast<uint16_t*>(take(sh.x_bytes)), reinterpret_cast<uint16_t*>(take(sh.x_bytes))};
  uint16_t* S = reinterpret_cast<uint16_t*>(take(sh.s_bytes));
  uint16_t* B = reinterpret_cast<uint16_t*>(take(sh.s_bytes));
  float* part = reinterpret_cast<float*>(take(3 * sh.part_bytes()));
  unsigned* words = reinterpret_cast<unsigned*>(take(sizeof(unsigned) * sh.words()));
  double* partial = reinterpret_cast<double*>(take(sizeof(double) * 3 * sh.norm_blocks * batch));
  float* scales = reinterpret_cast<float*>(take(sizeof(float) * 2 * OZ_MAX_NS_STEPS * batch));
  const long long xplane = static_cast<long long>(sh.rows) * sh.ldx;

  const long long work = (static_cast<long long>(sh.rows) * (sh.ldx / 8) + 255) / 256;
  if (launch_overlapping(norm_kernel, dim3(sh.norm_blocks, batch), 256, 0, stream, G, dtype, m, n, ldg, stride_g, partial, words,
                         sh.words()) != cudaSuccess ||
      launch_overlapping(convert_kernel, dim3(static_cast<unsigned>(work < 1024 ? work : 1024), batch), 256, 0, stream, G, dtype, m,
                         n, ldg, stride_g, partial, sh.norm_blocks, eps, plan, X[0], sh.ldx, xplane, slices, scales) != cudaSuccess)
    return OZ_ECUDA;
  return slices == 2 ? run_chain<2>(sh, plan, X, S, B, part, words, scales, O, dtype, ldo, stride_o, dev, stream)
                     : run_chain<1>(sh, plan, X, S, B, part, words, scales, O, dtype, ldo, stride_o, dev, stream);
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

size_t ozaki_newton_schulz_workspace_bytes(int m, int n, int batch, int num_slices) {
  if (m <= 0 || n <= 0 || m > kMaxExtent || n > kMaxExtent || batch <= 0 || batch > 65535 || num_slices < 1 || num_slices > 2) return 0;
  return Shape(m, n, batch, num_slices).total();
}

int ozaki_newton_schulz_ws(int m, int n, int batch, int dtype, const void* G, int ldg, long long strideG, void* O, int ldo,
                           long long strideO, int steps, const float* coeffs, float eps, int num_slices, void* workspace,
                           size_t ws_bytes, cudaStream_t stream) {
  int rc = check(m, n, batch, dtype, ldg, strideG, ldo, strideO, steps, coeffs, eps, num_slices);
  if (rc) return rc;
  NewtonPlan plan;
  if ((rc = make_plan(steps, coeffs, &plan))) return rc;
  if (m == 0 || n == 0 || batch == 0) return OZ_OK;
  if (!G || !O) return OZ_EINVAL;
  return run(m, n, batch, dtype, G, ldg, strideG, O, ldo, strideO, plan, eps, num_slices, workspace, ws_bytes, stream);
}

int ozaki_newton_schulz(int m, int n, int batch, int dtype, const void* G, int ldg, long long strideG, void* O, int ldo,
                        long long strideO, int steps, const float* coeffs, float eps, int num_slices,
                        cudaStream_t stream) {
  int rc = check(m, n, batch, dtype, ldg, strideG, ldo, strideO, steps, coeffs, eps, num_slices);
  if (rc) return rc;
  NewtonPlan plan;
  if ((rc = make_plan(steps, coeffs, &plan))) return rc;
  if (m == 0 || n == 0 || batch == 0) return OZ_OK;
  if (!G || !O) return OZ_EINVAL;
  const size_t bytes = ozaki_newton_schulz_workspace_bytes(m, n, batch, num_slices);
  void* ws = nullptr;
  if (bytes) {
    keep_default_pool_cached();
    if (cudaMallocAsync(&ws, bytes, stream) != cudaSuccess) {
      cudaGetLastError();
      return OZ_ENOMEM;
    }
  }
  rc = run(m, n, batch, dtype, G, ldg, strideG, O, ldo, strideO, plan, eps, num_slices, ws, bytes, stream);
  if (ws && cudaFreeAsync(ws, stream) != cudaSuccess && rc == OZ_OK) rc = OZ_ECUDA;
  return rc;
}

}  // extern "C"
