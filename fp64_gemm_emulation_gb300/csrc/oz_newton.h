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

// A sum of squares in three ranges (Blue's method), so that no square over- or underflows, and no sum of
// fewer than 2^37 of them: the squares stay below 2^76, 2^90 and 2^80 (with values up to 2^50 in the middle
// range, 2^28 of them added up to more than FP32 holds).
struct SumSquares {
  float big = 0.0f, mid = 0.0f, small = 0.0f;  // (x 2^-90)^2, x^2, (x 2^90)^2
  __device__ __forceinline__ void add(float x) {
    const float m = fabsf(x);
    if (m > 0x1p45f) {
      const float y = x * 0x1p-90f;
      big = fmaf(y, y, big);
    } else if (m < 0x1p-50f) {
      const float y = x * 0x1p90f;
      small = fmaf(y, y, small);
    } else {
      mid = fmaf(x, x, mid);  // and NaN
    }
  }
};

// From the three sums, by a warp: X_0 = G / (|G|_F + eps) is stored as G f0 f1 = G 2^(sx - e) with
// 2^e >= |G|_F > 2^(e-1); what remains, 2^e / (|G|_F + eps) = r 2^-t0 with r in [1, 2), goes into
// the factors of the products, a step a lane.  X_i is stored times 2^t_i, t_i = sx + max(0, t0 - drop i)
// (t0 > 0 only when eps dominates the norm; a tiny X gains at most `drop` bits a step) and t = 0 at the end:
// factors[2 i] = gram_i 2^(-2 t_i) and factors[2 i + 1] = 2^(t_{i+1} - t_i - sb_i), the first step's times
// r^2 and r.  factors may be null.
__device__ inline void newton_scales(float big, float mid, float small, float eps, const NewtonPlan& plan, float* f01,
                                     float* factors) {
  const int lane = threadIdx.x & 31;
  // |G|_F = root 2^k, by the largest range that holds anything (with the next one, which may reach into it)
  const int k = big != 0.0f ? 90 : mid != 0.0f ? 0 : -90;
  const float root = sqrtf(k > 0 ? big + ldexpf(mid, -180) : k == 0 ? mid + ldexpf(small, -180) : small);
  int e = 0, t0 = 0;
  float r = 0.0f;
  if (isfinite(root) && root > 0.0f) {
    e = ilogbf(root);
    if (ldexpf(1.0f, e) < root) ++e;
    const float q = ldexpf(1.0f, e) / (root + ldexpf(eps, -k));
    if (q > 0.0f) {
      t0 = -ilogbf(q);
      r = ldexpf(q, t0);
    }
    e += k;
  } else if (root != 0.0f) {
    r = NAN;  // a matrix that holds Inf or NaN gives NaN everywhere
  }
  const int h = (plan.sx - e) / 2;
  if (lane == 0) {
    f01[0] = ldexpf(1.0f, h);
    f01[1] = ldexpf(1.0f, plan.sx - e - h);
  }
  if (!factors || lane >= plan.steps) return;
  static_assert(OZ_MAX_NS_STEPS <= 32, "a lane for each step");
  auto stored = [&](int i) { return plan.sx + max(0, t0 - plan.drop * i); };
  const int t = stored(lane), next = lane + 1 == plan.steps ? 0 : stored(lane + 1);
  const float q = lane == 0 ? r : 1.0f;
  factors[2 * lane] = ldexpf(plan.gram[lane] * q * q, -2 * t);
  factors[2 * lane + 1] = ldexpf(q, next - t - plan.sb[lane]);
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
