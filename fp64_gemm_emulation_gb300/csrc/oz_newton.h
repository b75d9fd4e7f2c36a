// oz_newton.h -- what the two Newton-Schulz kernels share: the plan of the iteration, the norm and
// the scales.
#pragma once

#include "oz_internal.h"

namespace oz {

// Power-of-two scales from bounds on the singular values (make_plan), for every step.
struct NewtonPlan {
  int steps;
  int sx;                        // |X_i| 2^sx fits FP16
  int drop;                      // 2^drop >= max |p|: bits a tiny X may gain in a step
  unsigned int square;           // bit i: step i has the middle product (c != 0)
  float gram[OZ_MAX_NS_STEPS];   // the first product's factor
  int sb[OZ_MAX_NS_STEPS];       // B is stored times 2^sb
  float diag_s[OZ_MAX_NS_STEPS], alpha_b[OZ_MAX_NS_STEPS], diag_b[OZ_MAX_NS_STEPS];
};

// A sum of squares in three ranges (Blue's method), so that no square over- or underflows.
struct SumSquares {
  float big = 0.0f, mid = 0.0f, small = 0.0f;  // (x 2^-70)^2, x^2, (x 2^90)^2
  __device__ __forceinline__ void add(float x) {
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
  }
};

// From the three sums: X_0 = G / (|G|_F + eps) is stored as G f0 f1 = G 2^(sx - e) with
// 2^e >= |G|_F > 2^(e-1); what remains, 2^e / (|G|_F + eps) = r 2^-t0 with r in [1, 2), goes into
// the factors of the products (t0 > 0 only when eps dominates the norm; it shrinks by `drop` a step,
// the most a tiny X can grow): factors[2 i] = gram_i 2^(-2 t_i) and factors[2 i + 1] = 2^(t_{i+1} - t_i - sb),
// the last to t = 0.  factors may be null.
__device__ inline void newton_scales(const double (&s)[3], float eps, const NewtonPlan& plan, float* f01, float* factors) {
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
  const int h = (plan.sx - e) / 2;
  f01[0] = static_cast<float>(scalbn(1.0, h));
  f01[1] = static_cast<float>(scalbn(1.0, plan.sx - e - h));
  if (!factors) return;
  int t = plan.sx + t0;
  for (int i = 0; i < plan.steps; ++i) {
    int next = t - plan.drop < plan.sx ? plan.sx : t - plan.drop;
    if (i + 1 == plan.steps) next = 0;
    const double q = i == 0 ? r : 1.0;
    factors[2 * i] = static_cast<float>(scalbn(plan.gram[i] * q * q, -2 * t));
    factors[2 * i + 1] = static_cast<float>(scalbn(q, next - t - plan.sb[i]));
    t = next;
  }
}

// Matrices that one CTA's shared memory holds (oz_newton_small.cu).
inline bool newton_is_small(int rows, int cols, int slices) {
  const int side = rows < cols ? rows : cols, lng = rows < cols ? cols : rows;
  return side <= 128 && lng <= (slices == 2 ? 256 : 512);
}

int launch_newton_small(int rows, int cols, int batch, int dtype, const void* G, long long ldg, long long stride_g, void* O,
                        long long ldo, long long stride_o, const NewtonPlan& plan, float eps, int slices,
                        cudaStream_t stream);

}  // namespace oz
