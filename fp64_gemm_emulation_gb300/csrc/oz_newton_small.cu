// oz_newton_small.cu -- the Newton-Schulz iteration of a small matrix inside one CTA.
//
// The same iteration, scales and slices as oz_newton.cu (S = A + b/2c I, B = c S^2 + .., X <- B X), for
// matrices whose X and S fit shared memory: the smaller side at most 128, the larger at most 256 (two
// slices) or 512.  Between products of a chain that spans CTAs there is a fence, a flag and a reload
// (128 x 128 FP32: 9 us a product); here a product is handed on by an mbarrier (3.3 us), and the whole
// operator, norm included, is one launch.  One CTA a matrix.
//
// X is kept with its smaller side as rows, in 128-byte-swizzled blocks of 64 columns.  That one
// layout is the K-major operand of the Gram product (K = columns) and the MN-major operand of
// B X (N = columns, K = rows), so nothing is rearranged.  S and B share one buffer, and X_{i+1}
// replaces X_i: a product's sums are all in tensor memory before its operands are overwritten.
// An accumulator lane is a matrix row, so a thread writes 32 consecutive columns as 16-byte stores.
//   epilogue warps (lanes 32 (warp % 4) .., every second or fourth block of 32 columns), then one for the MMAs
// Two slices: sums leave the tensor core, which truncates, and are added up in FP32 registers, h l' + l h'
// before h h'.  S^2 decides the error, so there each MMA step (16 k) is a sum of its own and l l' is kept
// too; the other products take four steps at a time (100 x 100, five steps, against 64 bits; plain FP32 1.3e-6):
//   all by single steps, no l l'    1.8e-6  55 us (128 x 256: 87)   (times when this was chosen)
//   four steps but S^2              2.0e-6  49    (72)
//   and with l l' in S^2            1.6e-6  49    (72)   in all products: 1.6e-6  52 (77)
// Bound by the latency of a product (MMA, tensor-memory read, stores, two hand-overs): with five steps
// 128 x 128 bf16 27.7 us, FP32 50, 300 of them 56 and 102.
#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "oz_device.cuh"
#include "oz_newton.h"

namespace oz {
namespace {

constexpr int kRows = 128;
constexpr uint32_t kBlock = kRows * 128;  // 64 columns of 128 rows
// One slice: 16 epilogue warps (128 x 512 bf16 56 us, 128 x 128 27.7; with 8: 69 and 29.8).  Two: 8, whose running
// sums and hand-overs cost more with 16 (128 x 128 FP32, when this was chosen: 58 us; with 16: 69).
template <int SLICES>
constexpr int kEpiWarpsOf = SLICES == 2 ? 8 : 16;
template <int SLICES>
constexpr int kThreadsOf = (kEpiWarpsOf<SLICES> + 1) * 32;
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride, version, 128-byte swizzle

struct SmallArgs {
  const void* G;
  void* O;
  long long ldg, stride_g, ldo, stride_o;
  int side, lng, wide, dtype;
  float eps;
  NewtonPlan plan;
  int* status;
  unsigned long long epi_wait_ns;
};

__device__ __forceinline__ float load_value(const void* p, long long i, int dtype) {
  if (dtype == OZ_F32) return static_cast<const float*>(p)[i];
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == OZ_BF16 ? __bfloat162float(__ushort_as_bfloat16(h)) : __half2float(__ushort_as_half(h));
}

// Eight values from element `at` on, `count` of which exist (zeros for the others).
__device__ __forceinline__ void load8(float (&v)[8], const void* p, long long at, int count, int dtype, bool vec) {
  if (vec && count == 8) {
    if (dtype == OZ_F32) {
      const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t h = static_cast<uint16_t>(q[e >> 1] >> (16 * (e & 1)));
        v[e] = dtype == OZ_BF16 ? __bfloat162float(__ushort_as_bfloat16(h)) : __half2float(__ushort_as_half(h));
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < count ? load_value(p, at + e, dtype) : 0.0f;
  }
}

// 16 bytes of row r: columns 8 chunk .. of block blk.
__device__ __forceinline__ uint32_t tile_at(int r, int blk, int chunk) {
  return blk * kBlock + r * 128 + ((chunk ^ (r & 7)) << 4);
}

__device__ __forceinline__ void mma(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}

// The values pass through, so that no use of them moves above the wait before this.
__device__ __forceinline__ void tie(uint32_t (&r)[32]) {
#pragma unroll
  for (int e = 0; e < 32; e += 8)
    asm volatile("" : "+r"(r[e]), "+r"(r[e + 1]), "+r"(r[e + 2]), "+r"(r[e + 3]), "+r"(r[e + 4]), "+r"(r[e + 5]), "+r"(r[e + 6]),
                      "+r"(r[e + 7]));
}

template <int SLICES>
__global__ void __launch_bounds__(kThreadsOf<SLICES>, 1) newton_small_kernel(const __grid_constant__ SmallArgs a) {
  constexpr int kEpiWarps = kEpiWarpsOf<SLICES>;
  constexpr int kCols = kEpiWarps / 4;  // warps that share the blocks of 32 columns of a quadrant
  static_assert(SLICES == 1 || kCols == 2, "two slices: two blocks a warp are the 128 columns of a sum");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t accfull[4], accempty[4], ready, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ float sums[3][kEpiWarps];
  __shared__ float f01[2], factors[2 * OZ_MAX_NS_STEPS];
  volatile int* abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int side = a.side, lng = a.lng, steps = a.plan.steps;
  const int xblocks = (lng + 63) / 64, sblocks = (side + 63) / 64;
  const uint32_t xplane = xblocks * kBlock, splane = sblocks * kBlock;
  uint8_t* X = smem;
  uint8_t* S = smem + SLICES * xplane;
  const int dtype = a.dtype;
  const int size = dtype == OZ_F32 ? 4 : 2;
  const uint8_t* G = static_cast<const uint8_t*>(a.G) + blockIdx.x * a.stride_g * size;
  uint8_t* O = static_cast<uint8_t*>(a.O) + blockIdx.x * a.stride_o * size;
  const bool vec_in = ((reinterpret_cast<uintptr_t>(G) | (a.ldg * size)) & 15) == 0;
  const bool vec_out = a.wide && ((reinterpret_cast<uintptr_t>(O) | (a.ldo * size)) & 15) == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], kEpiWarps);
    }
    mbar_init(&ready, kEpiWarps);
    mbar_init(&drain, 1);
    abort_word = 0;
    mbar_fence_init();
  }
  if (warp == kEpiWarps) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }

  // The next launch may start once every CTA of this one holds its tensor memory: one of that launch's that
  // got an SM's columns first would wait for this launch, and this one for the columns.
  __syncthreads();
  let_next_start();
  wait_for_previous();

  // The norm, and X_0.
  if (warp < kEpiWarps) {
    SumSquares s;
    const int cols = a.wide ? lng : side, rows = a.wide ? side : lng;
    const int chunks = (cols + 7) / 8;
#pragma unroll 4
    for (int q = threadIdx.x; q < rows * chunks; q += kEpiWarps * 32) {
      const int r = q / chunks, c = 8 * (q - r * chunks);
      float v[8];
      load8(v, G, r * a.ldg + c, min(8, cols - c), dtype, vec_in);
      float own = s.mid;  // eight squares are summed by themselves first
      s.mid = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s.add(v[e]);
      s.mid += own;
    }
    float d[3] = {s.big, s.mid, s.small};
#pragma unroll
    for (int j = 0; j < 3; ++j) {
#pragma unroll
      for (int o = 16; o; o >>= 1) d[j] += __shfl_xor_sync(0xFFFFFFFFu, d[j], o);
      if (lane == 0) sums[j][warp] = d[j];
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    float d[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      d[j] = lane < kEpiWarps ? sums[j][lane] : 0.0f;
#pragma unroll
      for (int o = kEpiWarps / 2; o; o >>= 1) d[j] += __shfl_xor_sync(0xFFFFFFFFu, d[j], o);
      d[j] = __shfl_sync(0xFFFFFFFFu, d[j], 0);
    }
    newton_scales(d[0], d[1], d[2], a.eps, a.plan, f01, factors);
  }
  __syncthreads();
  const uint32_t tmem = tmem_slot;

  if (warp < kEpiWarps) {
    const float f0 = f01[0], f1 = f01[1];
    const int chunks = xblocks * 8;
#pragma unroll 4
    for (int q = threadIdx.x; q < kRows * chunks; q += kEpiWarps * 32) {
      const int i = a.wide ? q / chunks : q % kRows, c = a.wide ? q % chunks : q / kRows;
      float v[8];
      if (a.wide) {
        load8(v, G, i * a.ldg + 8 * c, i < side ? min(8, lng - 8 * c) : 0, dtype, vec_in);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = i < side && 8 * c + e < lng ? load_value(G, (8 * c + e) * a.ldg + i, dtype) : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * f0 * f1;
#pragma unroll
      for (int p = 0; p < SLICES; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 h = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
          v[2 * e] -= __low2float(h);
          v[2 * e + 1] -= __high2float(h);
          w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(X + p * xplane + tile_at(i, c >> 3, c & 7)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }

  // One product after another: the Gram product, the square (unless c = 0) and B X of each step.
  // With two slices a product is summed 128 columns at a time, so that a thread's running sums stay in
  // registers: the columns of B X do not depend on one another, and those that are done replace X's
  // while the next are still being summed.  Each sum (one k step or four) has an accumulator of its own;
  // two are handed over together (four of 128 columns).
  const int side_n = (side + 31) / 32 * 32, lng_n = (lng + 31) / 32 * 32;
  auto columns = [&](int kind) { return kind == 2 ? lng_n : side_n; };
  auto k_steps = [&](int kind) { return ((kind == 0 ? lng : side) + 15) / 16; };

  if (warp == kEpiWarps) {
    if (elect_one()) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t x_lo = smem_u32(X) >> 4, s_lo = smem_u32(S) >> 4;
      uint32_t ready_phase = 0, empty_bits = 0xFu;  // parities to wait for
      bool ok = true;
      auto next_acc = [&](int b) {  // waits until the epilogue has emptied buffer b
        if (!mbar_wait_or_abort(&accempty[b], empty_bits >> b & 1, kWaitLimitNs, abort_flag)) return false;
        empty_bits ^= 1u << b;
        tc_fence_after();
        return true;
      };
      for (int i = 0; i < steps && ok; ++i) {
        for (int kind = 0; kind < 3 && ok; ++kind) {
          if (kind == 1 && !(a.plan.square >> i & 1)) continue;
          const int n = columns(kind), ks = k_steps(kind);
          if (!mbar_wait_or_abort(&ready, ready_phase, kWaitLimitNs, abort_flag)) {
            ok = false;
            break;
          }
          ready_phase ^= 1;
          tc_fence_after();
          // D[i, j] = sum A[i, k] B[j, k]: Gram X X^T, S S, and B X with X as its MN-major operand
          const bool b_mn = kind == 2;
          const uint32_t a_base = (kind == 0 ? x_lo : s_lo) | (1u << 16);
          const uint32_t b_base = (kind == 1 ? s_lo : x_lo) | (b_mn ? (kBlock >> 4) << 16 : 1u << 16);
          const uint32_t a_plane = (kind == 0 ? xplane : splane) >> 4, b_plane = (kind == 1 ? splane : xplane) >> 4;
          const uint32_t idesc = (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(kRows >> 4) << 24);
          const uint32_t b_step = b_mn ? 16 * 128 >> 4 : 2, b_skip = b_mn ? 0 : (kBlock >> 4) - 8;
          if (SLICES == 1) {
            ok = next_acc(0);
            if (!ok) break;
            // an MMA's N is 256 at most: the columns past it (B X only) are a second product
            const uint32_t id = idesc | static_cast<uint32_t>(min(256, n) >> 3) << 17;
            const uint32_t id2 = idesc | static_cast<uint32_t>((n - 256) >> 3) << 17, b2 = 4 * (kBlock >> 4);
            uint32_t ak = a_base, bk = b_base;
            for (int k = 0; k < ks; k += 4) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (k + q < ks) {
                  mma(tmem, ak, bk, id, (k | q) > 0);
                  if (n > 256) mma(tmem + 256, ak, bk + b2, id2, (k | q) > 0);
                }
                ak += 2;
                bk += b_step;
              }
              ak += (kBlock >> 4) - 8;
              bk += b_skip;
            }
            umma_commit(&accfull[0]);
          } else {
            for (int n0 = 0; n0 < n && ok; n0 += 128) {
              const uint32_t id = idesc | static_cast<uint32_t>(min(128, n - n0) >> 3) << 17;
              uint32_t ak = a_base, bk = b_base + (n0 >> 6) * (kBlock >> 4);
              int buffer = 0;
              // the Gram product and B X: a sum for four steps, the small products first
              for (int k = 0; k < ks && kind != 1; k += 4) {
                if ((k & 4) == 0 && !(ok = next_acc(buffer))) break;
                const uint32_t d = tmem + 256 * buffer + 32 * (k & 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if (k + q < ks) {
                    mma(d, ak + 2 * q, bk + b_plane + b_step * q, id, q > 0);
                    mma(d, ak + a_plane + 2 * q, bk + b_step * q, id, 1u);
                  }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  if (k + q < ks) mma(d, ak + 2 * q, bk + b_step * q, id, 1u);
                if ((k & 4) != 0 || k + 4 >= ks) {
                  umma_commit(&accfull[buffer]);
                  buffer ^= 1;
                }
                ak += kBlock >> 4;
                bk += 4 * b_step + b_skip;
              }
              for (int k = 0; k < ks && kind == 1 && ok; k += 4) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if (k + q < ks) {
                    if ((q & 1) == 0 && !(ok = next_acc(buffer))) break;
                    const uint32_t d = tmem + 256 * buffer + 128 * (q & 1);
                    mma(d, ak + a_plane, bk + b_plane, id, 0u);
                    mma(d, ak, bk + b_plane, id, 1u);
                    mma(d, ak + a_plane, bk, id, 1u);
                    mma(d, ak, bk, id, 1u);
                    if ((q & 1) == 1 || k + q + 1 == ks) {
                      umma_commit(&accfull[buffer]);
                      buffer ^= 1;
                    }
                  }
                  ak += 2;
                  bk += b_step;
                }
                ak += (kBlock >> 4) - 8;
                bk += b_skip;
              }
            }
          }
        }
      }
      if (!ok && !*abort_flag) {
        *abort_flag = 1;
        atomicExch(a.status, OZ_ETIMEOUT);
      }
      umma_commit(&drain);  // arrives when every MMA above is done
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, part = warp >> 2;
    const int row = quad * 32 + lane;
    uint32_t full_bits = 0;
    bool ok = true;
    auto hand_on = [&]() {  // what this warp stored is an operand of the next product
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready);
    };
    hand_on();
    for (int i = 0; i < steps && ok; ++i) {
      for (int kind = 0; kind < 3 && ok; ++kind) {
        if (kind == 1 && !(a.plan.square >> i & 1)) continue;
        const int nblocks = columns(kind) / 32;
        const int sums = kind == 1 ? k_steps(kind) : (k_steps(kind) + 3) / 4;  // two slices
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const bool to_s = kind == 0 && (a.plan.square >> i & 1);
        const float f = kind == 1 ? a.plan.alpha_b[i] : factors[2 * i + (kind == 2 ? 1 : 0)];
        const float diag = kind == 2 ? 0.0f : to_s ? a.plan.diag_s[i] : a.plan.diag_b[i];
        const bool last = kind == 2 && i + 1 == steps;
        uint8_t* dst = kind == 2 ? X : S;
        const uint32_t plane = kind == 2 ? xplane : splane;

        auto wait_full = [&](int acc) {
          const bool got = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&accfull[acc], full_bits >> acc & 1, a.epi_wait_ns, abort_flag));
          full_bits ^= 1u << acc;
          if (!got && lane == 0 && !*abort_flag) {
            *abort_flag = 1;
            atomicExch(a.status, OZ_ETIMEOUT);
          }
          tc_fence_after();
          return got;
        };
        auto release = [&](int acc) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&accempty[acc]);
        };
        // 32 finished columns of this thread's row
        auto finish = [&](float (&v)[32], int cb) {
          const int n = 32 * cb;
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= f;
          if (diag != 0.0f && row >= n && row < n + 32 && row < side) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (row == n + e) v[e] += diag;
          }
          if (!last) {
#pragma unroll
            for (int p = 0; p < SLICES; ++p) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const __half2 h = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
                if (p + 1 < SLICES) {
                  add_two(v[2 * e], v[2 * e + 1], -__low2float(h), -__high2float(h));
                }
                w[e] = *reinterpret_cast<const uint32_t*>(&h);
              }
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(dst + p * plane + tile_at(row, cb >> 1, (cb & 1) * 4 + q)) =
                    make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            }
            return;
          }
          if (row >= side) return;
          if (vec_out && n + 32 <= lng) {
            uint4* to = reinterpret_cast<uint4*>(O + (row * a.ldo + n) * size);
            if (dtype == OZ_F32) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                to[q] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                                   __float_as_uint(v[4 * q + 3]));
            } else {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const __half2 h = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                w[e] = dtype == OZ_BF16 ? *reinterpret_cast<const uint32_t*>(&b) : *reinterpret_cast<const uint32_t*>(&h);
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) to[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            }
            return;
          }
          const long long base = a.wide ? row * a.ldo + n : n * a.ldo + row, step = a.wide ? 1 : a.ldo;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (n + e < lng) {
              const long long at = base + e * step;
              if (dtype == OZ_F32)
                reinterpret_cast<float*>(O)[at] = v[e];
              else if (dtype == OZ_BF16)
                reinterpret_cast<__nv_bfloat16*>(O)[at] = __float2bfloat16_rn(v[e]);
              else
                reinterpret_cast<__half*>(O)[at] = __float2half_rn(v[e]);
            }
          }
        };

        if (SLICES == 1) {
          if (!wait_full(0)) {
            ok = false;
            break;
          }
          for (int cb = part; cb < nblocks; cb += kCols) {
            uint32_t r[32];
            tmem_ld32(lanes + 32 * cb, r);
            tmem_ld_wait();
            tie(r);
            float v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
            finish(v, cb);
          }
          release(0);
        } else {
          for (int b0 = 0; b0 < nblocks && ok; b0 += 4) {  // 128 columns
            float run[2][32];
#pragma unroll
            for (int e = 0; e < 64; ++e) run[e >> 5][e & 31] = 0.0f;
            int buffer = 0;
            for (int k = 0; k < sums; k += 2, buffer ^= 1) {
              if (!wait_full(buffer)) {
                ok = false;
                break;
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int cb = kCols * j + part;
                if (b0 + cb < nblocks) {
                  uint32_t r0[32], r1[32];
                  const uint32_t at = lanes + 256 * buffer + 32 * cb;
                  tmem_ld32(at, r0);
                  if (k + 1 < sums) tmem_ld32(at + 128, r1);
                  tmem_ld_wait();
                  tie(r0);
#pragma unroll
                  for (int e = 0; e < 32; e += 2) add_two(run[j][e], run[j][e + 1], __uint_as_float(r0[e]), __uint_as_float(r0[e + 1]));
                  if (k + 1 < sums) {
                    tie(r1);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) add_two(run[j][e], run[j][e + 1], __uint_as_float(r1[e]), __uint_as_float(r1[e + 1]));
                  }
                }
              }
              release(buffer);
            }
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (b0 + kCols * j + part < nblocks) finish(run[j], b0 + kCols * j + part);
          }
          if (!ok) break;
        }
        hand_on();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && !mbar_wait(&drain, 0)) atomicExch(a.status, OZ_ETIMEOUT);
  __syncthreads();
  tc_fence_after();
  if (warp == kEpiWarps) tmem_dealloc(tmem, 512);
}

}  // namespace

int launch_newton_small(int rows, int cols, int batch, int dtype, const void* G, long long ldg, long long stride_g, void* O,
                        long long ldo, long long stride_o, const NewtonPlan& plan, float eps, int slices,
                        cudaStream_t stream) {
  SmallArgs a{};
  a.G = G;
  a.O = O;
  a.ldg = ldg;
  a.stride_g = stride_g;
  a.ldo = ldo;
  a.stride_o = stride_o;
  a.wide = rows <= cols;
  a.side = a.wide ? rows : cols;
  a.lng = a.wide ? cols : rows;
  a.dtype = dtype;
  a.eps = eps;
  a.plan = plan;
  a.status = device_status_ptr();
  a.epi_wait_ns = epilogue_wait_ns();
  int dev = 0;
  if (!a.status || cudaGetDevice(&dev) != cudaSuccess) return OZ_ECUDA;
  const int blocks = (a.lng + 63) / 64 + (a.side + 63) / 64;
  const size_t smem = 1024 + static_cast<size_t>(slices) * blocks * kBlock;
  auto kernel = slices == 2 ? newton_small_kernel<2> : newton_small_kernel<1>;
  constexpr int most = 1024 + 12 * static_cast<int>(kBlock);  // two slices of 256 + 128 columns, or one of 512 + 128
  static_assert(most + 2048 <= 232448, "shared memory budget");
  static std::atomic<bool> set[64][2] = {};
  for (int attempt = 0; attempt < 2; ++attempt) {  // the limit is set again in a new context (see launch)
    if (dev >= 64 || attempt || !set[dev][slices - 1].load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return OZ_ECUDA;
      if (dev < 64) set[dev][slices - 1].store(true, std::memory_order_release);
    }
    const cudaError_t e = launch_overlapping(kernel, dim3(batch), slices == 2 ? kThreadsOf<2> : kThreadsOf<1>, smem, stream, a);
    if (e == cudaSuccess) return OZ_OK;
    if (e != cudaErrorInvalidValue) break;
  }
  return OZ_ECUDA;
}

}  // namespace oz
