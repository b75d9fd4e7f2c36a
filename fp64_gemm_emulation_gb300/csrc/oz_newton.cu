// oz_newton.cu -- Newton-Schulz orthogonalisation of matrices on the tensor cores.
//
//   X_0 = G / (|G|_F + eps),   X_{i+1} = a X_i + (b A + c A^2) X_i,   A = X_i X_i^T
// (X_i^T X_i on the right when G has more rows than columns).  Completing the square,
//   S = A + (b / 2c) I,   B = c S^2 + (a - b^2 / 4c) I,   X_{i+1} = B X_i,
// makes a step three plain products whose epilogues only scale and add to the diagonal, so no
// epilogue reads a matrix back.  (c = 0: B = b A + a I comes out of the first product.)
// S and B are symmetric: only tiles that reach the lower triangle are computed, and mirrored.
//
// Numerics.  The products run on the FP16 tensor-core path: FP16 holds 11 bits where bf16
// holds 8, at the same rate, and every range is known beforehand: |X_0| <= 1, and a host-side
// bound on the polynomial bounds the singular values of every X_i, S and B, so each is stored
// times a power of two that fills FP16's range.  |G|_F is divided out as a power of two (exact
// on bf16 inputs); the remaining factor in [1, 2) joins the first step's scalings.  With two
// slices each matrix is h + l in FP16 (22 bits), and a product is h h' + h l' + l h'.  All sums
// are FP32; the norm's partial sums are joined in FP64.
#include <cmath>

#include "oz_products.cuh"

namespace oz {
namespace {

using namespace prod;

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

constexpr int kNormBlocks = 304;       // partial sums of a matrix's norm, at most
constexpr int kMaxSplitUnits = 608;    // (tile, part) pairs the split workspace holds
// Two slices: MMA steps (16 k) summed on the tensor core before the sum moves to FP32 registers.
// The tensor core truncates each addition, which biases long sums; the relative error of the
// result (five steps, against 64 bits) is proportional to it:
//   128 x 128:    1.6e-6 (1 step)  2.3e-6 (2)  3.5e-6 (4)  6.1e-6 (8)   plain FP32: 1.3e-6
//   8192 x 2048:  1.5e-6 (1)       1.9e-6 (2)  2.9e-6 (4)  5.0e-6 (8)   plain FP32: 4.7e-6
// and so is the epilogue's work: 4.1, 3.0, 2.6 and 2.4 ms at 8192 x 2048.  One k-block (4 steps) keeps
// the error below plain FP32's where sums are long; sides up to 256 are bound by launches, so
// they take single steps.
constexpr int kChunk = 4;

// What the small kernels need of the plan.
struct StepScales {
  int steps;
  int sx;                           // |X_i| 2^sx fits FP16
  int drop;                         // 2^drop >= max |p|: bits a tiny X may gain in a step
  float gram[OZ_MAX_NS_STEPS];      // the first product's factor
  int sb[OZ_MAX_NS_STEPS];          // B is stored times 2^sb
};

__device__ __forceinline__ float load_value(const void* p, long long i, int dtype) {
  if (dtype == OZ_F32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == OZ_BF16 ? __bfloat162float(__ushort_as_bfloat16(h)) : __half2float(__ushort_as_half(h));
}

// Sums of squares in three ranges (Blue's method), so that no square over- or underflows:
// partial[matrix][block] = {sum (x 2^-70)^2 of the large, sum x^2, sum (x 2^90)^2 of the small}.
__global__ void __launch_bounds__(256) norm_kernel(const void* __restrict__ G, int dtype, int cols, long long rows,
                                                   long long ld, long long stride, double* __restrict__ partial,
                                                   unsigned* __restrict__ counters, int ncounters) {
  if (blockIdx.y == 0)
    for (int i = blockIdx.x * 256 + threadIdx.x; i < ncounters; i += gridDim.x * 256) counters[i] = 0;
  const long long base = blockIdx.y * stride;
  float big = 0.0f, mid = 0.0f, small = 0.0f;
  auto add = [&](float x) {
    const float m = fabsf(x);
    if (m > 0x1p50f) {
      const float y = x * 0x1p-70f;
      big = fmaf(y, y, big);
    } else if (m < 0x1p-50f) {
      const float y = x * 0x1p90f;
      small = fmaf(y, y, small);
    } else {
      mid = fmaf(x, x, mid);  // and NaN
    }
  };
  const bool dense = ld == cols && (reinterpret_cast<uintptr_t>(G) & 15) == 0 && stride % 8 == 0;
  if (dense) {  // 16-byte loads over the whole matrix
    const long long n = rows * cols;
    const int per = dtype == OZ_F32 ? 4 : 8;
    const long long nv = n / per;
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(G) + base * (dtype == OZ_F32 ? 4 : 2));
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < nv; i += gridDim.x * 256ll) {
      const uint4 w = __ldg(v + i);
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
      const float before = mid;  // the vector's squares are summed by themselves first
      mid = 0.0f;
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
      mid += before;
    }
    for (long long i = nv * per + blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll)
      add(load_value(G, base + i, dtype));
  } else {
    for (long long r = blockIdx.x; r < rows; r += gridDim.x)
      for (int c = threadIdx.x; c < cols; c += 256) add(load_value(G, base + r * ld + c, dtype));
  }
  __shared__ double sums[3][8];
  double s[3] = {big, mid, small};
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

// X_0 = G / (|G|_F + eps) as FP16 slices times 2^t, t = sx + t0: G 2^-e 2^sx with
// 2^e >= |G|_F > 2^(e-1), and what remains, 2^e / (|G|_F + eps) = r 2^-t0 with r in [1, 2),
// goes into the factors of the products (t0 > 0 only when eps dominates the norm; it shrinks
// by `drop` a step, the most a tiny X can grow).
__global__ void __launch_bounds__(256) convert_kernel(const void* __restrict__ G, int dtype, int cols, long long rows,
                                                      long long ld, long long stride, const double* __restrict__ partial,
                                                      int nblocks, float eps, const __grid_constant__ StepScales sc,
                                                      uint16_t* __restrict__ X, int ldx, long long plane, int planes,
                                                      float* __restrict__ scales) {
  __shared__ float s_mul[2];
  if (threadIdx.x < 32) {
    double s[3] = {0.0, 0.0, 0.0};
    const double* p = partial + static_cast<long long>(blockIdx.y) * nblocks * 3;
    for (int b = threadIdx.x; b < nblocks; b += 32)
      for (int j = 0; j < 3; ++j) s[j] += p[b * 3 + j];
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
      for (int d = 16; d; d >>= 1) s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], d);
    if (threadIdx.x == 0) {
      const double norm = sqrt(scalbn(s[0], 140) + s[1] + scalbn(s[2], -180));
      const double whole = norm + static_cast<double>(eps);
      int e = 0, t0 = 0;
      double r = 0.0;
      if (isfinite(norm) && norm > 0.0) {
        e = ilogb(norm);
        if (scalbn(1.0, e) < norm) ++e;
        const double q = scalbn(1.0, e) / whole;
        t0 = -ilogb(q);
        r = scalbn(q, t0);
      } else if (norm != 0.0) {
        r = NAN;  // a matrix that holds Inf or NaN gives NaN everywhere
      }
      const int h = (sc.sx - e) / 2;
      s_mul[0] = static_cast<float>(scalbn(1.0, h));
      s_mul[1] = static_cast<float>(scalbn(1.0, sc.sx - e - h));
      if (blockIdx.x == 0) {
        // factors of the steps: gram_i = gram 2^(-2 t_i), apply_i = 2^(t_{i+1} - t_i - sb), the last to t = 0
        float* f = scales + static_cast<long long>(blockIdx.y) * 2 * sc.steps;
        int t = sc.sx + t0;
        for (int i = 0; i < sc.steps; ++i) {
          int next = t - sc.drop < sc.sx ? sc.sx : t - sc.drop;
          if (i + 1 == sc.steps) next = 0;
          const double q = i == 0 ? r : 1.0;
          f[2 * i] = static_cast<float>(scalbn(sc.gram[i] * q * q, -2 * t));
          f[2 * i + 1] = static_cast<float>(scalbn(q, next - t - sc.sb[i]));
          t = next;
        }
      }
    }
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

// The iteration's plan: power-of-two scales from bounds on the singular values.
struct Plan {
  StepScales sc;
  float diag_s[OZ_MAX_NS_STEPS], alpha_b[OZ_MAX_NS_STEPS], diag_b[OZ_MAX_NS_STEPS];
  bool square[OZ_MAX_NS_STEPS];
};

int room(double bound) { return static_cast<int>(std::floor(std::log2(60000.0 / bound))); }

// OZ_ERANGE if the singular values may leave the range in which the scales keep 11 (22) bits
// useful: a bound above 16 on X, or a square whose completion cancels more than 4 bits.
int make_plan(int steps, const float* coeffs, Plan* out) {
  Plan p{};
  p.sc.steps = steps;
  double bound = 1.0, worst = 1.0, gain = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double a = coeffs[3 * i], b = coeffs[3 * i + 1], c = coeffs[3 * i + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return OZ_EINVAL;
    p.square[i] = c != 0.0;
    const double beta = p.square[i] ? b / (2 * c) : 0.0;
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
    if (p.square[i]) {
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
    p.sc.sb[i] = room(p_max);
    if (p.square[i]) {
      if (std::fabs(c) * s_max * s_max > 16.0 * p_max) return OZ_ERANGE;
      const int sa = room(s_max);
      p.sc.gram[i] = static_cast<float>(std::ldexp(1.0, sa));
      p.diag_s[i] = static_cast<float>(std::ldexp(beta, sa));
      p.alpha_b[i] = static_cast<float>(std::ldexp(c, p.sc.sb[i] - 2 * sa));
      p.diag_b[i] = static_cast<float>(std::ldexp(a - b * beta / 2, p.sc.sb[i]));
    } else {
      p.sc.gram[i] = static_cast<float>(std::ldexp(b, p.sc.sb[i]));
      p.diag_b[i] = static_cast<float>(std::ldexp(a, p.sc.sb[i]));
    }
    bound = std::fmax(x_max, 1e-3);
    worst = std::fmax(worst, x_max);
    gain = std::fmax(gain, p_max);
  }
  p.sc.sx = room(worst) < 14 ? room(worst) : 14;
  p.sc.drop = static_cast<int>(std::ceil(std::log2(gain)));
  *out = p;
  return OZ_OK;
}

struct Shape {
  int cols, rows, batch, planes, side;  // contiguous extent, rows; side: the smaller
  int ldx, lds;
  bool wide;                            // rows <= cols
  size_t x_bytes, s_bytes, part_bytes;
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
  // Split workspace: enough for every product's choice (plan_tiles), at full tile width.
  size_t split_bytes() const { return align256(sizeof(float) * 2 * HALF_M * BN * static_cast<size_t>(split_units())); }
  int split_units() const {
    const long long tiles = static_cast<long long>(batch) * ceil_div(side, BM);
    return tiles >= kMaxSplitUnits ? 0 : kMaxSplitUnits / 4;
  }
  size_t total() const {
    return 2 * x_bytes + 2 * s_bytes + split_bytes() + align256(sizeof(unsigned) * 2 * kMaxSplitUnits) +
           align256(sizeof(double) * 3 * norm_blocks * batch) + align256(sizeof(float) * 2 * OZ_MAX_NS_STEPS * batch);
  }
};

// Tile width and parts of the k range of one product, by a model of its time in SM cycles
// (units per pair x k-blocks x cycles of a block, plus a unit's start and drain and the
// joining of parts).
void plan_tiles(int M, int N, int K, int batch, int sym, int planes, bool b_mn, int pairs, int max_units, int* bn_out,
                int* split_out) {
  const int nkb = ceil_div(K, BK);
  double best = 1e30;
  for (int bn = planes == 2 ? BN2 : BN; bn >= (b_mn ? 128 : 64); bn /= 2) {
    const long long tiles = static_cast<long long>(batch) * dense_tiles(M, N, bn, sym);
    const double block = planes == 2 ? (bn == 128 ? 850 : 640) : (bn == 256 ? 560 : bn == 128 ? 380 : 320);
    for (int s = 1; s <= 16 && s <= nkb; ++s) {
      if (s > 1 && (tiles >= pairs || tiles * s > max_units)) break;
      const double waves = static_cast<double>((tiles * s + pairs - 1) / pairs);
      double t = waves * (ceil_div(nkb, s) * block + 600) + 3000;
      if (s > 1) t += 1500 + 2200.0 * (bn / 256.0) * (1 + s);
      if (t < best) {
        best = t;
        *bn_out = bn;
        *split_out = s;
      }
    }
  }
}

int check(int m, int n, int batch, int dtype, const void* G, int ldg, long long stride_g, int ldo, long long stride_o,
          int steps, const float* coeffs, float eps, int slices) {
  if (m < 0 || n < 0 || batch < 0) return OZ_EINVAL;
  if (dtype != OZ_BF16 && dtype != OZ_F16 && dtype != OZ_F32) return OZ_EINVAL;
  if (ldg < (m > 1 ? m : 1) || ldo < (m > 1 ? m : 1)) return OZ_EINVAL;
  if (batch > 1 && (stride_g < static_cast<long long>(ldg) * n || stride_o < static_cast<long long>(ldo) * n))
    return OZ_EINVAL;
  if (steps < 1 || steps > OZ_MAX_NS_STEPS || !coeffs || slices < 1 || slices > 2) return OZ_EINVAL;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return OZ_EINVAL;
  if (batch > 65535) return OZ_EINVAL;
  (void)G;
  return OZ_OK;
}

int run(int m, int n, int batch, int dtype, const void* G, int ldg, long long stride_g, void* O, int ldo,
        long long stride_o, const Plan& plan, float eps, int slices, void* workspace, size_t ws_bytes,
        cudaStream_t stream) {
  const Shape sh(m, n, batch, slices);
  if (!workspace || ws_bytes < sh.total() || (reinterpret_cast<uintptr_t>(workspace) & 255)) return OZ_ENOMEM;
  Device dev;
  int rc;
  if ((rc = current_device(&dev))) return rc;
  const int pairs = dev.pairs;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  auto take = [&](size_t bytes) {
    uint8_t* p = at;
    at += align256(bytes);
    return p;
  };
  uint16_t* X[2] = {reinterpret_cast<uint16_t*>(take(sh.x_bytes)), reinterpret_cast<uint16_t*>(take(sh.x_bytes))};
  uint16_t* S = reinterpret_cast<uint16_t*>(take(sh.s_bytes));
  uint16_t* B = reinterpret_cast<uint16_t*>(take(sh.s_bytes));
  float* part = reinterpret_cast<float*>(take(sh.split_bytes()));
  unsigned* counters = reinterpret_cast<unsigned*>(take(sizeof(unsigned) * 2 * kMaxSplitUnits));
  double* partial = reinterpret_cast<double*>(take(sizeof(double) * 3 * sh.norm_blocks * batch));
  float* scales = reinterpret_cast<float*>(take(sizeof(float) * 2 * OZ_MAX_NS_STEPS * batch));
  const long long xplane = static_cast<long long>(sh.rows) * sh.ldx, splane = static_cast<long long>(sh.side) * sh.lds;

  norm_kernel<<<dim3(sh.norm_blocks, batch), 256, 0, stream>>>(G, dtype, m, n, ldg, stride_g, partial, counters,
                                                               2 * kMaxSplitUnits);
  const long long work = (static_cast<long long>(sh.rows) * (sh.ldx / 8) + 255) / 256;
  convert_kernel<<<dim3(static_cast<unsigned>(work < 1024 ? work : 1024), batch), 256, 0, stream>>>(
      G, dtype, m, n, ldg, stride_g, partial, sh.norm_blocks, eps, plan.sc, X[0], sh.ldx, xplane, slices, scales);
  if (cudaGetLastError() != cudaSuccess) return OZ_ECUDA;

  const int side = sh.side, P = slices;
  int bn_gram = 0, bn_sq = 0, bn_app = 0, s_gram = 1, s_sq = 1, s_app = 1;
  const int long_side = sh.wide ? sh.cols : sh.rows;
  plan_tiles(side, side, long_side, batch, 1, P, !sh.wide, pairs, sh.split_units(), &bn_gram, &s_gram);
  plan_tiles(side, side, side, batch, 1, P, false, pairs, sh.split_units(), &bn_sq, &s_sq);
  plan_tiles(sh.cols, sh.rows, side, batch, 0, P, false, pairs, sh.split_units(), &bn_app, &s_app);

  // Maps by role: m side (A) and n side (B) of each product.
  CUtensorMap gA[2], gB[2], sA, sB, pA[2], pB[2], bOp;
  const uint64_t mats = static_cast<uint64_t>(batch) * P, xl = 2ull * sh.ldx, sl = 2ull * sh.lds;
  bool ok = make_map(&sA, S, false, side, side, mats, sl, 2ull * splane, HALF_M) &&
            make_map(&sB, S, false, side, side, mats, sl, 2ull * splane, bn_sq / 2) &&
            make_map(&bOp, B, false, side, side, mats, sl, 2ull * splane, sh.wide ? bn_app / 2 : HALF_M);
  for (int i = 0; i < 2 && ok; ++i) {
    auto x_map = [&](CUtensorMap* t, int box) {
      return make_map(t, X[i], false, sh.cols, sh.rows, mats, xl, 2ull * xplane, box);
    };
    // rows of ldx: the padding past the last column is the workspace's own (a multiple of 64), and
    // what is read there only reaches output elements that are never stored
    auto mn_map = [&](CUtensorMap* t, int blocks) {
      int is_4d = 0;  // 1: ldx is a multiple of 64
      return make_mn_map(t, &is_4d, blocks, X[i], false, sh.ldx, sh.rows, mats, xl, 2ull * xplane);
    };
    if (sh.wide)
      ok = x_map(&gA[i], HALF_M) && x_map(&gB[i], bn_gram / 2) && mn_map(&pA[i], 2);
    else
      ok = mn_map(&gA[i], 2) && mn_map(&gB[i], bn_gram / 128) && x_map(&pB[i], bn_app / 2);
  }
  if (!ok) return OZ_ECUDA;

  Args base{};
  base.groups = batch;
  base.chunk = P == 2 ? (side <= 256 ? 1 : kChunk) : 1 << 28;
  base.part = part;
  base.counters = counters;
  base.max_split_units = sh.split_units();
  base.vec = 1;
  base.a_4d = base.b_4d = 1;
  base.planes_out = P;
  auto grid = [&](const Args& a) { return a.tiles * a.nsplit < pairs ? a.tiles * a.nsplit : pairs; };
  const int steps = plan.sc.steps;
  for (int i = 0; i < steps; ++i) {
    const int cur = i & 1;
    const bool last = i + 1 == steps;
    Args g = base;  // S 2^sa = 2^sa A + 2^sa b/(2c) I   (or B itself when c = 0)
    g.M = g.N = side;
    g.K = long_side;
    g.bn = bn_gram;
    g.part_cols = bn_gram;
    g.nsplit = s_gram;
    g.sym = 1;
    g.tiles = batch * dense_tiles(side, side, bn_gram, 1);
    g.out_type = kOutSlices;
    g.box_rows = bn_gram / 2;
    g.out = plan.square[i] ? S : B;
    g.ld = sh.lds;
    g.plane = splane;
    g.stride = splane * P;
    g.alpha = 1.0f;
    g.scale = scales + 2 * i;
    g.scale_stride = 2 * steps;
    g.diag = plan.square[i] ? plan.diag_s[i] : plan.diag_b[i];
    if (sh.wide) {
      g.idesc = idesc_base(false, false, false);
      rc = P == 2 ? launch<kDense, false, false, 2>(gA[cur], gB[cur], gB[cur], g, dev, grid(g), i > 0, stream)
                  : launch<kDense, false, false, 1>(gA[cur], gB[cur], gB[cur], g, dev, grid(g), i > 0, stream);
    } else {
      g.idesc = idesc_base(false, true, true);
      rc = P == 2 ? launch<kDense, true, true, 2>(gA[cur], gB[cur], gB[cur], g, dev, grid(g), i > 0, stream)
                  : launch<kDense, true, true, 1>(gA[cur], gB[cur], gB[cur], g, dev, grid(g), i > 0, stream);
    }
    if (rc) return rc;
    if (plan.square[i]) {  // B 2^sb = c 2^(sb - 2 sa) (S 2^sa)^2 + 2^sb (a - b^2 / 4c) I
      Args q = g;
      q.K = side;
      q.bn = q.part_cols = bn_sq;
      q.nsplit = s_sq;
      q.tiles = batch * dense_tiles(side, side, bn_sq, 1);
      q.box_rows = bn_sq / 2;
      q.out = B;
      q.alpha = plan.alpha_b[i];
      q.scale = nullptr;
      q.diag = plan.diag_b[i];
      q.idesc = idesc_base(false, false, false);
      rc = P == 2 ? launch<kDense, false, false, 2>(sA, sB, sB, q, dev, grid(q), true, stream)
                  : launch<kDense, false, false, 1>(sA, sB, sB, q, dev, grid(q), true, stream);
      if (rc) return rc;
    }
    Args x = base;  // X_{i+1} 2^t' = 2^(t' - t - sb) (B 2^sb)(X_i 2^t)
    x.M = sh.cols;
    x.N = sh.rows;
    x.K = side;
    x.bn = x.part_cols = bn_app;
    x.nsplit = s_app;
    x.tiles = batch * dense_tiles(sh.cols, sh.rows, bn_app, 0);
    x.box_rows = bn_app / 2;
    x.alpha = 1.0f;
    x.scale = scales + 2 * i + 1;
    x.scale_stride = 2 * steps;
    if (last) {
      x.out = O;
      x.ld = ldo;
      x.stride = stride_o;
      x.planes_out = 1;
      x.out_type = dtype == OZ_F32 ? kOutF32 : dtype == OZ_BF16 ? kOutBf16 : kOutF16;
      x.vec = (reinterpret_cast<uintptr_t>(O) & 15) == 0 && ldo % 8 == 0 && (batch == 1 || stride_o % 8 == 0);
    } else {
      x.out = X[cur ^ 1];
      x.ld = sh.ldx;
      x.plane = xplane;
      x.stride = xplane * P;
      x.out_type = kOutSlices;
    }
    if (sh.wide) {  // D[col, row] = sum_j X[j, col] B[row, j]
      x.idesc = idesc_base(false, true, false);
      rc = P == 2 ? launch<kDense, true, false, 2>(pA[cur], bOp, bOp, x, dev, grid(x), true, stream)
                  : launch<kDense, true, false, 1>(pA[cur], bOp, bOp, x, dev, grid(x), true, stream);
    } else {  // D[col, row] = sum_j B[col, j] X[row, j]
      x.idesc = idesc_base(false, false, false);
      rc = P == 2 ? launch<kDense, false, false, 2>(bOp, pB[cur], pB[cur], x, dev, grid(x), true, stream)
                  : launch<kDense, false, false, 1>(bOp, pB[cur], pB[cur], x, dev, grid(x), true, stream);
    }
    if (rc) return rc;
  }
  return OZ_OK;
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

size_t ozaki_newton_schulz_workspace_bytes(int m, int n, int batch, int num_slices) {
  if (m <= 0 || n <= 0 || batch <= 0 || batch > 65535 || num_slices < 1 || num_slices > 2) return 0;
  return Shape(m, n, batch, num_slices).total();
}

int ozaki_newton_schulz_ws(int m, int n, int batch, int dtype, const void* G, int ldg, long long strideG, void* O, int ldo,
                           long long strideO, int steps, const float* coeffs, float eps, int num_slices, void* workspace,
                           size_t ws_bytes, cudaStream_t stream) {
  int rc = check(m, n, batch, dtype, G, ldg, strideG, ldo, strideO, steps, coeffs, eps, num_slices);
  if (rc) return rc;
  Plan plan;
  if ((rc = make_plan(steps, coeffs, &plan))) return rc;
  if (m == 0 || n == 0 || batch == 0) return OZ_OK;
  if (!G || !O) return OZ_EINVAL;
  return run(m, n, batch, dtype, G, ldg, strideG, O, ldo, strideO, plan, eps, num_slices, workspace, ws_bytes, stream);
}

int ozaki_newton_schulz(int m, int n, int batch, int dtype, const void* G, int ldg, long long strideG, void* O, int ldo,
                        long long strideO, int steps, const float* coeffs, float eps, int num_slices,
                        cudaStream_t stream) {
  int rc = check(m, n, batch, dtype, G, ldg, strideG, ldo, strideO, steps, coeffs, eps, num_slices);
  if (rc) return rc;
  Plan plan;
  if ((rc = make_plan(steps, coeffs, &plan))) return rc;
  if (m == 0 || n == 0 || batch == 0) return OZ_OK;
  if (!G || !O) return OZ_EINVAL;
  const size_t bytes = ozaki_newton_schulz_workspace_bytes(m, n, batch, num_slices);
  keep_default_pool_cached();
  void* ws = nullptr;
  if (cudaMallocAsync(&ws, bytes, stream) != cudaSuccess) {
    cudaGetLastError();
    return OZ_ENOMEM;
  }
  rc = run(m, n, batch, dtype, G, ldg, strideG, O, ldo, strideO, plan, eps, num_slices, ws, bytes, stream);
  if (cudaFreeAsync(ws, stream) != cudaSuccess && rc == OZ_OK) rc = OZ_ECUDA;
  return rc;
}

}  // extern "C"
