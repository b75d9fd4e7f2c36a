// oz_block8.cu -- products of 8-bit floating-point matrices with a 32-bit scale for each block of 128,
// grouped by expert as oz_grouped.cu's, and their gradients.
//
//   forward  Y_e = W_e^T X_e     D[n, row] = sum_b sw[e, n/128, b] sx[row, b] sum_{k in b} W_e[k, n] X[k, row]
//   dgrad    dX_e = W_e dY_e     D[k, row] = sum_b sw[e, b, k/128] sy[row, b] sum_{n in b} W_e[k, n] dY[n, row]
//   wgrad    dW_e = X_e dY_e^T   D[k, n]   = sum_b sx[b, k] sy[b, n] sum_{row in b} X[k, row] dY[n, row]
// (column-major; b runs over the blocks of 128 of the sum's index).  A block's products are summed by the
// tensor cores (kind::f8f6f4, FP32 sums of 128 products) and its sum is scaled and added to FP32 sums in
// registers, rounding to nearest: any FP32 scales are taken, and no sum is longer than 128 on the tensor cores.
//
// Kernel shape: clusters of two CTAs (cta_group::2), persistent over tiles of 256 m x up to 256 n, m along
// the output's contiguous dimension, so that a CTA's 128 m share one row of the weights' scales.
//   warp 0: TMA producer   warp 1: TMEM owner + MMA issuer (leader)   warp 2: scales   warps 4-11: epilogue
// 6 stages of 32 KB: 128 (or 64 ...) rows of 128 bytes of A and of B, K-major or MN-major as they lie in memory.
#include "oz_products.cuh"
#include "oz_ragged.cuh"

namespace oz {
namespace {

using namespace prod;

constexpr int BK8 = kScaleBlock;
constexpr int STEP8 = 32;                       // k of one MMA
constexpr int STAGES8 = 6;
constexpr uint32_t TILE8 = 128 * BK8;           // bytes of a stage's A (and of its B) in one CTA
constexpr int EPI8_FIRST = 4, EPI8_WARPS = 8, THREADS8 = (EPI8_FIRST + EPI8_WARPS) * 32;
constexpr int BLOCKS8 = 4;                      // blocks of 32 columns whose sums a warp holds
constexpr uint32_t STASH8 = 32 * 64;
// Registers: the four warps of the first warpgroup give theirs to the epilogue, whose threads hold 128 sums.
// 128 x 72 + 256 x 216 = 384 x 168, what the launch has.
constexpr int REGS_FEW = 72, REGS_MANY = 216;

enum Op8 { kForward8, kDgrad8, kWgrad8 };

template <Op8 OP>
struct Scales8 {
  static constexpr int SLOTS = OP == kWgrad8 ? 4 : 8;
  static constexpr int BATCH = SLOTS / 2;       // k-blocks whose scales are fetched at once
  static constexpr int FLOATS = OP == kWgrad8 ? 256 + 128 : 256;
  static constexpr uint32_t BYTES = SLOTS * FLOATS * 4;
};

struct Params8 {
  CUtensorMap tmA, tmB, tmB128;
  int M, N, K;    // contiguous extent of the output; wgrad: its rows; otherwise the sum's length
  int groups, rows, bn;
  int vec, out_type;
  uint32_t idesc;
  const int32_t* offsets;
  void* out;
  long long ld, stride;
  const float *sa, *sb;     // scales of A and B
  long long sa_group, sb_ld;
  int sa_m, sa_k;           // forward, dgrad: strides of a block along m and along the sum
  int* status;
  unsigned long long epi_wait_ns;
};

// Deals out the tiles, as GroupedWalk does: a group's rows in equal tiles (a multiple of 32 rows, at most bn) by
// the output's m, the group's tiles by row tile; wgrad: the output's tiles of every group.
template <Op8 OP>
struct Walk8 {
  static constexpr bool A_MN = OP != kForward8, B_MN = OP == kWgrad8, RAGGED_SUM = OP == kWgrad8;
  static constexpr int BOX = 32;  // ragged rows: the small box of B (the large one has 128 rows)
  static constexpr size_t kTableBytes = (2 * (OZ_MAX_GROUPS + 1) + 1) * 4;

  const Params8& a;
  const int *off, *prefix;
  int total, idx, tiles_m, tiles_n;

  __device__ static void setup(const Params8& a, int* table) {
    int* off = table;
    int* prefix = table + OZ_MAX_GROUPS + 1;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
      tma_prefetch_desc(&a.tmA);
      tma_prefetch_desc(&a.tmB);
      if (!B_MN) tma_prefetch_desc(&a.tmB128);
    }
    let_next_start();
    wait_for_previous();
    if (threadIdx.x >= 32) return;
    if (clamp_offsets(a.offsets, a.groups, a.rows, off) && lane == 0 && blockIdx.x == 0) atomicExch(a.status, OZ_EINVAL);
    __syncwarp();
    if (RAGGED_SUM) return;
    const int tiles_m = ceil_div(a.M, BM);
    int sum = 0;
    for (int b = 0; b <= a.groups; b += 32) {
      const int i = b + lane;
      int t = i >= 1 && i <= a.groups ? ceil_div(off[i] - off[i - 1], a.bn) * tiles_m : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, t, d);
        if (lane >= d) t += o;
      }
      if (i <= a.groups) prefix[i] = sum + t;
      sum += __shfl_sync(0xFFFFFFFFu, t, 31);
    }
  }

  __device__ Walk8(const Params8& p, const int* table) : a(p), off(table), prefix(table + OZ_MAX_GROUPS + 1) {
    tiles_m = ceil_div(a.M, BM);
    tiles_n = RAGGED_SUM ? ceil_div(a.N, a.bn) : 0;
    total = RAGGED_SUM ? a.groups * tiles_m * tiles_n : prefix[a.groups];
    idx = static_cast<int>(blockIdx.x >> 1) - static_cast<int>(gridDim.x >> 1);
  }

  __device__ bool next(Unit& u) {
    idx += static_cast<int>(gridDim.x >> 1);
    if (idx >= total) return false;
    int group;
    if (RAGGED_SUM) {
      const int per = tiles_m * tiles_n;
      group = idx / per;
      const int r = idx - group * per, tn = r / tiles_m;
      u.m0 = (r - tn * tiles_m) * BM;
      u.n0 = u.orow = tn * a.bn;
      u.nn = min(a.bn, a.N - u.n0);
      u.kb1 = ceil_div(off[group + 1] - off[group], BK8);
      u.k0 = a.offsets ? first_column_block(off[group], group) : 0;  // in blocks
      u.zA = u.zB = 0;
      u.nmma = BN;
    } else {
      group = group_of(prefix, a.groups, idx);
      const int r = idx - prefix[group], tn = r / tiles_m;
      const int len = off[group + 1] - off[group];
      const int w = ceil_div(ceil_div(len, ceil_div(len, a.bn)), 32) * 32;
      u.m0 = (r - tn * tiles_m) * BM;
      u.n0 = u.orow = off[group] + tn * w;
      u.nn = min(w, len - tn * w);
      u.kb1 = ceil_div(a.K, BK8);
      u.k0 = 0;
      u.zA = group;
      u.zB = 0;
      u.nmma = ceil_div(u.nn, 32) * 32;
    }
    u.kb0 = 0;
    u.a_mn = A_MN;
    u.b_mn = B_MN;
    const bool wide = u.nmma > 128;
    u.mapA = &a.tmA;
    u.mapB = !B_MN && wide ? &a.tmB128 : &a.tmB;
    u.box_b = B_MN || wide ? 128 : BOX;
    u.boxes = B_MN || wide ? 1 : ceil_div(u.nmma / 2, BOX);
    u.box_bytes = u.box_b * BK8;
    u.idesc = a.idesc | (static_cast<uint32_t>(u.nmma >> 3) << 17);
    u.m_extent = a.M;
    u.out = static_cast<uint16_t*>(a.out) + (RAGGED_SUM ? group * a.stride : 0);
    u.ld = a.ld;
    u.out_type = a.out_type;
    u.vec = a.vec;
    u.sym = false;
    return true;
  }

  // Rows that belong to no group are zero.
  __device__ void outside(int warp) const {
    if (RAGGED_SUM || !a.offsets) return;
    const int lo = off[0], hi = off[a.groups], loose = lo + a.rows - hi;
    for (int i = static_cast<int>(blockIdx.x) * EPI8_WARPS + warp; i < loose; i += gridDim.x * EPI8_WARPS) {
      uint16_t* row = static_cast<uint16_t*>(a.out) + static_cast<long long>(i < lo ? i : hi + i - lo) * a.ld;
      for (int c = threadIdx.x & 31; c < a.M; c += 32) row[c] = 0;
    }
  }
};

__device__ __forceinline__ void umma8_pair(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(DESC_HIGH)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4 with FP32 sums, without its N field (formats: 0 e4m3, 1 e5m2).
constexpr uint32_t idesc8_base(int fa, int fb, bool a_mn, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(fa) << 7) | (static_cast<uint32_t>(fb) << 10) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(BM >> 4) << 24);
}

// Two neighbouring sums in one instruction: a += b s.
__device__ __forceinline__ void fma_two(float& a0, float& a1, float b0, float b1, float2 s) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmov.b64 z, {%4, %5};\n\t"
      "fma.rn.f32x2 x, y, z, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1), "f"(s.x), "f"(s.y));
}
__device__ __forceinline__ float2 mul_two(float2 a, float b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b));
  return r;
}

// A block's sums v, scaled, added to the running ones.  s: this block's 32 column scales in shared memory.
// sm: wgrad's scales of this lane's four m (the others have theirs in s).
template <Op8 OP>
__device__ __forceinline__ void add_scaled(float (&run)[32], const float (&v)[32], const float* s, const float (&sm)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 sn = *reinterpret_cast<const float2*>(s + 8 * q + 2 * (lane & 3));
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // m = lane / 4 + 8 h
      const int i = 16 * (h >> 1) + 4 * q + 2 * (h & 1);
      fma_two(run[i], run[i + 1], v[i], v[i + 1], OP == kWgrad8 ? mul_two(sn, sm[h]) : sn);
    }
  }
}

template <Op8 OP>
__global__ void __launch_bounds__(THREADS8, 1) block8_kernel(const __grid_constant__ Params8 a) {
  typedef Walk8<OP> Walk;
  typedef Scales8<OP> Sc;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES8 * TILE8;
  float* scales = reinterpret_cast<float*>(smem + 2 * STAGES8 * TILE8);
  uint8_t* stash = smem + 2 * STAGES8 * TILE8 + Sc::BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stash + EPI8_WARPS * STASH8);
  uint64_t* full = bars;                     // [STAGES8] TMA (both CTAs) -> MMA  (used in the leader)
  uint64_t* empty = full + STAGES8;          // [STAGES8] MMA -> TMA              (both CTAs)
  uint64_t* accfull = empty + STAGES8;       // [4]       MMA -> epilogue         (both CTAs)
  uint64_t* accempty = accfull + 4;          // [4]       epilogues (both) -> MMA (used in the leader)
  uint64_t* sfull = accempty + 4;            // [SLOTS]   scales -> epilogue      (per CTA)
  uint64_t* sempty = sfull + Sc::SLOTS;      // [SLOTS]   epilogue -> scales      (per CTA)
  uint64_t* drain = sempty + Sc::SLOTS;      // [1]       all MMAs of the pair done (both CTAs)
  uint64_t* exitbar = drain + 1;             // [1]       the peer has finished (per CTA)
  uint64_t* proddone = exitbar + 1;          // [1]       both producers have stopped (used in the leader)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(proddone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued_by = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);  // [2] (leader)
  int* table = reinterpret_cast<int*>(stash + EPI8_WARPS * STASH8 + 512);               // the walker's

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t acc_cols = a.bn > 128 ? 256 : 128, nacc = TMEM_COLS / acc_cols;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES8; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], 2 * EPI8_WARPS);
    }
    for (int i = 0; i < Sc::SLOTS; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], EPI8_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(exitbar, 1);
    mbar_init(proddone, 2);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  Walk::setup(a, table);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp < EPI8_FIRST) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_FEW));
    if (warp == 0) {
      if (elect_one()) {
        // ------------------------------------------------------------ TMA producer (both CTAs)
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
        Walk walk(a, table);
        Unit u{};
        bool ok = true;
        while (ok && !*abort_flag && walk.next(u)) {
          const int rowA = u.m0 + static_cast<int>(rank) * HALF_M;
          const int rowB = u.n0 + static_cast<int>(rank) * (u.nmma >> 1);
          const uint32_t bytes = TILE8 + u.boxes * u.box_bytes;
          int k = u.k0 * BK8;
          for (int kb = 0; kb < u.kb1; ++kb, k += BK8) {
            if (!mbar_wait_or_abort(&empty[stage], phase ^ 1, kWaitLimitNs, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t bar = full_leader + stage * 8;
            mbar_arrive_expect_tx_cluster(bar, bytes);
            uint8_t* dA = sA + stage * TILE8;
            uint8_t* dB = sB + stage * TILE8;
            if (Walk::A_MN)
              tma_load_3d_pair(dA, u.mapA, bar, rowA, k, u.zA);
            else
              tma_load_3d_pair(dA, u.mapA, bar, k, rowA, u.zA);
            if (Walk::B_MN) {
              tma_load_3d_pair(dB, u.mapB, bar, rowB, k, u.zB);
            } else {
              for (int b = 0; b < u.boxes; ++b) tma_load_3d_pair(dB + b * u.box_bytes, u.mapB, bar, k, rowB + u.box_b * b, u.zB);
            }
            ++issued;
            if (++stage == STAGES8) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        if (!ok && !*abort_flag) stop_pair(abort_flag, a.status);
        // Every issued copy must have landed before the pair may exit (see the residue GEMM).
        st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(&issued_by[rank])), 0), issued);
        mbar_arrive_release_cluster(mapa_shared(smem_u32(proddone), 0));
        if (!*abort_flag) {
          for (uint32_t i = 0; i < STAGES8 && i < issued; ++i) {
            if (--stage < 0) {
              stage = STAGES8 - 1;
              phase ^= 1;
            }
            if (!mbar_wait_or_abort(&empty[stage], phase, kWaitLimitNs, abort_flag)) {
              if (!*abort_flag) stop_pair(abort_flag, a.status);
              break;
            }
          }
        }
      }
    } else if (warp == 1) {
      if (rank == 0 && elect_one()) {
        // ------------------------------------------------------------ MMA issuer (leader only)
        int stage = 0;
        uint32_t phase = 0, acc = 0, acc_phase = 1, consumed = 0;
        bool ok = true;
        const uint32_t a_desc = desc_low(smem_u32(sA), Walk::A_MN), b_desc = desc_low(smem_u32(sB), Walk::B_MN);
        constexpr uint32_t a_step = (Walk::A_MN ? STEP8 * 128 : STEP8) >> 4, b_step = (Walk::B_MN ? STEP8 * 128 : STEP8) >> 4;
        Walk walk(a, table);
        Unit u{};
        while (ok && !*abort_flag && walk.next(u)) {
          for (int left = u.kb1; left > 0; --left) {
            if (!mbar_wait_or_abort(&accempty[acc], acc_phase, kWaitLimitNs, abort_flag) ||
                !mbar_wait_or_abort(&full[stage], phase, kWaitLimitNs, abort_flag)) {
              ok = false;
              break;
            }
            ++consumed;
            tc_fence_after();
            const uint32_t ad = a_desc + stage * (TILE8 >> 4), bd = b_desc + stage * (TILE8 >> 4);
            const uint32_t d_tmem = tmem_base + acc * acc_cols;
#pragma unroll
            for (int kk = 0; kk < BK8 / STEP8; ++kk) umma8_pair(d_tmem, ad + kk * a_step, bd + kk * b_step, u.idesc, kk > 0 ? 1u : 0u);
            umma_commit_pair(&empty[stage], 0x3);
            umma_commit_pair(&accfull[acc], 0x3);
            if (++acc == nacc) {
              acc = 0;
              acc_phase ^= 1;
            }
            if (++stage == STAGES8) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        if (!ok && !*abort_flag) stop_pair(abort_flag, a.status);
        // Account for every copy before the pair may exit (see the residue GEMM).
        if (mbar_wait_acquire_cluster(proddone, 0)) {
          const uint32_t n0 = issued_by[0], n1 = issued_by[1];
          const uint32_t top = n0 > n1 ? n0 : n1;
          for (uint32_t q = consumed; q < top && q < consumed + STAGES8; ++q) {
            const int st = static_cast<int>(q % STAGES8);
            if (q >= n0) mbar_arrive(&full[st]);
            if (q >= n1) mbar_arrive(&full[st]);
            if (!mbar_wait(&full[st], (q / STAGES8) & 1)) {
              stop_pair(abort_flag, a.status);
              break;
            }
          }
        } else {
          stop_pair(abort_flag, a.status);
        }
        umma_commit_pair(drain, 0x3);
      }
    } else if (warp == 2) {
      // -------------------------------------------------------------- scales (both CTAs)
      // A slot holds a k-block's scales: for each of the tile's n, times the one of the CTA's 128 m (forward,
      // dgrad); those of n and of m (wgrad).  BATCH blocks are fetched at once, while the epilogue uses the
      // ones before.
      int slot = 0;
      uint32_t sphase = 1;
      bool ok = true;
      Walk walk(a, table);
      Unit u{};
      while (ok && !*abort_flag && walk.next(u)) {
        const int mblock = u.m0 / 128 + static_cast<int>(rank);
        const bool inside = mblock * 128 < a.M;
        const float* sa = OP == kWgrad8 ? a.sa + static_cast<long long>(u.k0) * a.sa_group + mblock * 128
                                        : a.sa + u.zA * a.sa_group + static_cast<long long>(mblock) * a.sa_m;
        const float* sb = a.sb + u.k0 * a.sb_ld + u.orow;
        for (int kb = 0; ok && kb < u.kb1; kb += Sc::BATCH) {
          float n[Sc::BATCH][8], m[Sc::BATCH][4];
#pragma unroll
          for (int j = 0; j < Sc::BATCH; ++j) {
            const bool have = kb + j < u.kb1;
            const float* row = sb + (kb + j) * a.sb_ld;
#pragma unroll
            for (int i = 0; i < 8; ++i) n[j][i] = have && lane + 32 * i < u.nn ? row[lane + 32 * i] : 0.0f;
            if (OP == kWgrad8) {
              const float* col = sa + (kb + j) * a.sa_group;
#pragma unroll
              for (int i = 0; i < 4; ++i) m[j][i] = have && mblock * 128 + lane + 32 * i < a.M ? col[lane + 32 * i] : 0.0f;
            } else {
              m[j][0] = have && inside ? sa[static_cast<long long>(kb + j) * a.sa_k] : 0.0f;
            }
          }
#pragma unroll
          for (int j = 0; j < Sc::BATCH; ++j) {
            if (kb + j < u.kb1 && ok) {
              ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&sempty[slot], sphase, kWaitLimitNs, abort_flag));
              if (ok) {
                float* to = scales + slot * Sc::FLOATS;
#pragma unroll
                for (int i = 0; i < 8; ++i) to[lane + 32 * i] = OP == kWgrad8 ? n[j][i] : n[j][i] * m[j][0];
                if (OP == kWgrad8) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) to[256 + lane + 32 * i] = m[j][i];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfull[slot]);
                if (++slot == Sc::SLOTS) {
                  slot = 0;
                  sphase ^= 1;
                }
              }
            }
          }
        }
      }
      if (!ok && lane == 0 && !*abort_flag) stop_pair(abort_flag, a.status);
    }
  } else {
    // -------------------------------------------------------------- epilogue (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_MANY));
    // A warp scales and sums its 32 lanes of every second block of 32 columns.
    const int quad = warp & 3, first = (warp - EPI8_FIRST) >> 2;
    uint8_t* my_stash = stash + (warp - EPI8_FIRST) * STASH8;
    const uint32_t accempty_leader = mapa_shared(smem_u32(accempty), 0);
    uint32_t acc = 0, acc_phase = 0, slot = 0, sphase = 0;
    bool ok = true;
    Walk walk(a, table);
    walk.outside(warp - EPI8_FIRST);
    Unit u{};
    while (ok && walk.next(u)) {
      const int nblocks = ceil_div(u.nn, 32);
      float run[BLOCKS8][32];
#pragma unroll
      for (int i = 0; i < BLOCKS8 * 32; ++i) run[i >> 5][i & 31] = 0.0f;
      for (int kb = 0; kb < u.kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&sfull[slot], sphase, kWaitLimitNs, abort_flag) &&
                                         mbar_wait_or_abort(&accfull[acc], acc_phase, a.epi_wait_ns, abort_flag))) {
          ok = false;
          if (lane == 0 && !*abort_flag) stop_pair(abort_flag, a.status);
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * acc_cols;
        const float* s = scales + slot * Sc::FLOATS;
        float sm[4] = {};
        if (OP == kWgrad8) {
#pragma unroll
          for (int h = 0; h < 4; ++h) sm[h] = s[256 + quad * 32 + (lane >> 2) + 8 * h];
        }
#pragma unroll
        for (int j = 0; j < BLOCKS8; ++j) {
          const int cb = 2 * j + first;
          if (cb < nblocks) {
            float v[32];
            tmem_ld_block(taddr + cb * 32, v);
            tmem_wait_block(v);
            add_scaled<OP>(run[j], v, s + 32 * cb, sm);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_cluster(accempty_leader + acc * 8);
          mbar_arrive(&sempty[slot]);
        }
        if (++acc == nacc) {
          acc = 0;
          acc_phase ^= 1;
        }
        if (++slot == Sc::SLOTS) {
          slot = 0;
          sphase ^= 1;
        }
      }
      if (!ok) break;
      const Target target = target_of(u, static_cast<int>(rank) * HALF_M + quad * 32, my_stash);
#pragma unroll
      for (int j = 0; j < BLOCKS8; ++j) {
        const int cb = 2 * j + first;
        if (cb < nblocks) emit<false, true>(u, target, run[j], cb, my_stash);
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (!mbar_wait(drain, 0)) {
      *abort_flag = 1;
      atomicExch(a.status, OZ_ETIMEOUT);
    }
    mbar_arrive_cluster(mapa_shared(smem_u32(exitbar), rank ^ 1u));
    if (!mbar_wait(exitbar, 0)) {
      *abort_flag = 1;
      atomicExch(a.status, OZ_ETIMEOUT);
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// ------------------------------------------------------------------ host side
// [mats][rows][cols] of bytes; box {128, box_rows, 1}.
bool make_map8(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t mats, uint64_t ld, uint64_t stride, int box_rows) {
  const EncodeTiled fn = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
  const cuuint64_t dims[3] = {cols, rows, mats}, strides[2] = {ld, stride};
  const cuuint32_t box[3] = {BK8, static_cast<cuuint32_t>(box_rows), 1}, estr[3] = {1, 1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operand8 {
  const void* p;
  int type;                    // OZ_E4M3, OZ_E5M2
  long long cols, rows, mats;  // contiguous extent, rows, matrices
  long long ld, stride;
  const float* scales;
  bool valid() const {
    if ((type != OZ_E4M3 && type != OZ_E5M2) || ld < (cols > 1 ? cols : 1) || (mats > 1 && stride < ld * rows)) return false;
    return cols == 0 || rows == 0 || mats == 0 ||
           ((rows == 1 || ld % 16 == 0) && (mats == 1 || stride % 16 == 0) && (reinterpret_cast<uintptr_t>(p) & 15) == 0 &&
            (reinterpret_cast<uintptr_t>(scales) & 3) == 0);
  }
  bool map(CUtensorMap* m, int box_rows) const {
    const uint64_t pitch = rows > 1 ? ld : roundup(cols, 16);  // one row has no stride to speak of
    return make_map8(m, p, cols, rows, mats, pitch, mats > 1 ? stride : pitch * rows, box_rows);
  }
};

struct Problem8 {
  Op8 op;
  int n, k, rows, groups;
  Operand8 a, b;  // A: W, or X (wgrad); B: X, or dY
  long long lds_a, lds_b;  // row scales: distance of blocks; column scales: likewise
  const int32_t* offsets;
  int out_type;
  void* out;
  int ldo;
  long long strideo;

  int m_out() const { return op == kForward8 ? n : k; }
  int sum() const { return op == kForward8 ? k : op == kDgrad8 ? n : rows; }
  bool empty() const { return m_out() == 0 || (op == kWgrad8 ? n : rows) == 0; }
};

int check8(const Problem8& p) {
  if (p.n < 0 || p.k < 0 || p.rows < 0 || p.n > kMaxExtent || p.k > kMaxExtent || p.rows > kMaxExtent - 128 * (OZ_MAX_GROUPS + 1)) return OZ_EINVAL;
  if (p.groups < 1 || p.groups > OZ_MAX_GROUPS || (!p.offsets && p.groups != 1)) return OZ_EINVAL;
  if (p.out_type != OZ_BF16 && p.out_type != OZ_F16) return OZ_EINVAL;
  if (!p.a.valid() || !p.b.valid()) return OZ_EINVAL;
  if (p.op == kWgrad8 ? p.lds_a < (p.k > 1 ? p.k : 1) || p.lds_b < (p.n > 1 ? p.n : 1) : p.lds_b < (p.rows > 1 ? p.rows : 1)) return OZ_EINVAL;
  const int m = p.m_out();
  if (p.ldo < (m > 1 ? m : 1)) return OZ_EINVAL;
  if (p.op == kWgrad8 && p.groups > 1 && p.strideo < static_cast<long long>(p.ldo) * p.n) return OZ_EINVAL;
  if (p.empty()) return OZ_OK;
  if (!p.out || (reinterpret_cast<uintptr_t>(p.out) & 1)) return OZ_EINVAL;
  if (p.sum() > 0 && (!p.a.p || !p.b.p || !p.a.scales || !p.b.scales)) return OZ_EINVAL;
  return OZ_OK;
}

template <Op8 OP>
int launch8(const Problem8& p, const Device& d, cudaStream_t stream) {
  typedef Walk8<OP> Walk;
  Params8 a{};
  a.M = p.m_out();
  a.N = p.n;
  a.K = OP == kForward8 ? p.k : p.n;
  a.groups = p.groups;
  a.rows = p.rows;
  a.bn = BN;
  a.vec = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.ldo % 8 == 0 && (OP != kWgrad8 || p.groups == 1 || p.strideo % 8 == 0);
  a.out_type = p.out_type == OZ_BF16 ? kOutBf16 : kOutF16;
  a.idesc = idesc8_base(p.a.type == OZ_E5M2, p.b.type == OZ_E5M2, Walk::A_MN, Walk::B_MN);
  a.offsets = p.offsets;
  a.out = p.out;
  a.ld = p.ldo;
  a.stride = p.strideo;
  a.sa = p.a.scales;
  a.sb = p.b.scales;
  a.sb_ld = p.lds_b;
  const int kb = ceil_div(p.k, 128);
  if (OP == kWgrad8) {
    a.sa_group = p.lds_a;
  } else {
    a.sa_group = static_cast<long long>(ceil_div(p.n, 128)) * kb;
    a.sa_m = OP == kForward8 ? kb : 1;
    a.sa_k = OP == kForward8 ? 1 : kb;
  }
  bool ok = p.a.map(&a.tmA, 128) && p.b.map(&a.tmB, OP == kWgrad8 ? 128 : Walk::BOX);
  if (OP != kWgrad8) ok = ok && p.b.map(&a.tmB128, 128);
  if (!ok) return OZ_ECUDA;
  a.status = d.status;
  a.epi_wait_ns = epilogue_wait_ns();
  auto kernel = block8_kernel<OP>;
  constexpr size_t smem = 1024 /*alignment*/ + 2 * STAGES8 * TILE8 + Scales8<OP>::BYTES + EPI8_WARPS * STASH8 + 512 /*barriers*/ + Walk::kTableBytes;
  static_assert(smem <= 232448, "shared memory budget");
  static_assert(smem + 2 * 16384 > 232448, "alone on its SM, as the other holders of tensor memory");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * d.pairs, 1, 1);
  cfg.blockDim = dim3(THREADS8);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  static std::atomic<bool> ready[64] = {};  // as prod::launch
  for (int attempt = 0; attempt < 2; ++attempt) {
    if (d.id >= 64 || attempt || !ready[d.id].load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return OZ_ECUDA;
      if (d.id < 64) ready[d.id].store(true, std::memory_order_release);
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) return OZ_OK;
    cudaGetLastError();
    if (e != cudaErrorInvalidValue) break;
  }
  return OZ_ECUDA;
}

// The matrices outside every sum: zeros of the output.
int zero_output8(const Problem8& p, cudaStream_t stream) {
  const size_t width = 2 * static_cast<size_t>(p.m_out()), pitch = 2 * static_cast<size_t>(p.ldo);
  const int mats = p.op == kWgrad8 ? p.groups : 1, rows = p.op == kWgrad8 ? p.n : p.rows;
  for (int e = 0; e < mats; ++e)
    if (cudaMemset2DAsync(static_cast<uint8_t*>(p.out) + 2 * e * p.strideo, pitch, 0, width, rows, stream) != cudaSuccess)
      return OZ_ECUDA;
  return OZ_OK;
}

int run8(const Problem8& p, cudaStream_t stream) {
  int rc = check8(p);
  if (rc || p.empty()) return rc;
  if (p.sum() == 0) return zero_output8(p, stream);
  Device dev;
  if ((rc = current_device(&dev))) return rc;
  switch (p.op) {
    case kForward8: return launch8<kForward8>(p, dev, stream);
    case kDgrad8: return launch8<kDgrad8>(p, dev, stream);
    default: return launch8<kWgrad8>(p, dev, stream);
  }
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

int ozaki_grouped_gemm_f8(int n, int k, int rows, int groups, int type_w, const void* W, int ldw, long long strideW, const float* SW,
                          int type_x, const void* X, int ldx, const float* SX, int ldsx, const int32_t* offsets, int dtype, void* Y,
                          int ldy, cudaStream_t stream) {
  return run8(Problem8{kForward8, n, k, rows, groups, {W, type_w, k, n, groups, ldw, strideW, SW}, {X, type_x, k, rows, 1, ldx, 0, SX},
                       0, ldsx, offsets, dtype, Y, ldy, 0}, stream);
}
int ozaki_grouped_gemm_f8_dgrad(int n, int k, int rows, int groups, int type_w, const void* W, int ldw, long long strideW, const float* SW,
                                int type_dy, const void* dY, int lddy, const float* SdY, int ldsdy, const int32_t* offsets, int dtype,
                                void* dX, int lddx, cudaStream_t stream) {
  return run8(Problem8{kDgrad8, n, k, rows, groups, {W, type_w, k, n, groups, ldw, strideW, SW}, {dY, type_dy, n, rows, 1, lddy, 0, SdY},
                       0, ldsdy, offsets, dtype, dX, lddx, 0}, stream);
}
int ozaki_grouped_gemm_f8_wgrad(int n, int k, int rows, int groups, int type_dy, const void* dY, int lddy, const float* SdY, int ldsdy,
                                int type_x, const void* X, int ldx, const float* SX, int ldsx, const int32_t* offsets, int dtype,
                                void* dW, int ldw, long long strideW, cudaStream_t stream) {
  if (rows < 0 || rows > kMaxExtent - 128 * (OZ_MAX_GROUPS + 1) || groups < 1 || groups > OZ_MAX_GROUPS) return OZ_EINVAL;
  const long long laid = offsets ? static_cast<long long>(kScaleBlock) * column_blocks(rows, groups, true) : rows;
  return run8(Problem8{kWgrad8, n, k, rows, groups, {X, type_x, k, laid, 1, ldx, 0, SX}, {dY, type_dy, n, laid, 1, lddy, 0, SdY},
                       ldsx, ldsdy, offsets, dtype, dW, ldw, strideW}, stream);
}

}  // extern "C"
