// oz_block8.cu -- products of 8-bit floating-point matrices with a 32-bit scale for each block of 128,
// grouped by expert as oz_grouped.cu's, and their gradients.
//
//   forward  Y_e = W_e^T X_e     D[row, n] = sum_b sx[row, b] sw[e, n/128, b] sum_{k in b} X[k, row] W_e[k, n]
//   dgrad    dX_e = W_e dY_e     D[row, k] = sum_b sy[row, b] sw[e, b, k/128] sum_{n in b} dY[n, row] W_e[k, n]
//   wgrad    dW_e = X_e dY_e^T   D[k, n]   = sum_b sx[b, k] sy[b, n] sum_{row in b} X[k, row] dY[n, row]
// (column-major; b runs over the blocks of 128 of the sum's index).  A block's products are summed by the
// tensor cores (kind::f8f6f4, FP32 sums of 128 products) and its sum is scaled and added to FP32 sums in
// registers, rounding to nearest: no sum is longer than 128 on the tensor cores.  The two scales of a sum are multiplied first: a
// product below 2^-126 is off by up to 2^-150, one of 2^128 and more is Inf.  (To add such blocks in FP64 instead cost the
// others: 8192 x 4096 x 8192 234 us instead of 227, 64 rows 17.9 instead of 15.9, weight gradient 410 instead of 385.)
//
// Kernel shape: clusters of two CTAs (cta_group::2), persistent over tiles of 256 m (the first index of D above) x
// 256 n, 128 m in each CTA.
//   warp 0: TMA producer   warps 1 and 3: MMA issuers of the two halves (leader; 1: TMEM owner)   warp 2: scales (wgrad)
//   warps 4-11: epilogue
// 4 stages (wgrad: 6) of 32 KB: 128 x 128 bytes of A and two tiles of 64 n of B, K-major or MN-major as they lie in memory.
// What bounds it: every 128 k each of a CTA's 128 x 256 sums is read from tensor memory, scaled and added, while the
// MMAs take 512 cycles.  So:
//  - rows of tokens are m, one a lane (tcgen05.ld.32x32b): a lane needs one factor for its 128 columns, its row's
//    scale times the one of the 128 features.  With features as m a lane needs every column's scale in
//    a register: 128 KB a k-block through the 128 bytes a cycle of shared memory's way back, 1024 cycles.
//  - wgrad has a scale for each row and column of a block.  It reads fragments (16x256b), where a lane's 32 sums are
//    of 4 m x 8 n, although their way out of tensor memory is slower (560 cycles for 128 x 256, 32x32b: below 300).
//  - the tile's halves of 128 columns are accumulators of their own, two each, and belong to 4 warps each: the way
//    from the MMAs to the epilogue and back (about 1000 cycles with both CTAs' barriers) overlaps more.
//  - a k-block costs one thread about 100 cycles for each wait and each copy, and 50 for a commit: the halves' MMAs are
//    issued by a thread each, and an operand is one copy where its tile is whole blocks of 128.
#include "oz_products.cuh"
#include "oz_ragged.cuh"

namespace oz {
namespace {

using namespace prod;

constexpr int BK8 = kScaleBlock;
constexpr int STEP8 = 32;                       // k of one MMA
constexpr uint32_t TILE8 = 128 * BK8;           // bytes of a stage's A (and of its B) in one CTA
constexpr uint32_t HALF8 = 64 * BK8;            // of the 64 n that a CTA holds of one accumulator
constexpr int ACC8 = 128;                       // columns of an accumulator; two for each half of the tile
constexpr int EPI8_FIRST = 4, EPI8_WARPS = 8, THREADS8 = (EPI8_FIRST + EPI8_WARPS) * 32;
constexpr int BLOCKS8 = ACC8 / 32;              // blocks of 32 columns whose sums a warp holds
constexpr int EARLY8 = 3;                       // reads of 16 columns before the next accumulator's first
// Registers: the four warps of the first warpgroup give theirs to the epilogue, whose threads hold 128 sums.
// 128 x 72 + 256 x 216 = 384 x 168, what the launch has.
constexpr int REGS_FEW = 72, REGS_MANY = 216;

enum Op8 { kForward8, kDgrad8, kWgrad8 };

// wgrad: scales of a k-block in shared memory, 256 of n and 128 of the CTA's m.
constexpr int SLOTS8 = 4, BATCH8 = 2, SLOT_FLOATS8 = 256 + 128;  // BATCH8: k-blocks whose scales are fetched at once
// The ring of stages, the scales, and the epilogue warps' stashes: wgrad's a block of 32 x 32, otherwise 32 rows of 128
// finished columns, which leave while the next tile is summed (16 bytes more a row: no bank conflicts, and room for a note).
template <Op8 OP>
struct Smem8 {
  static constexpr int STAGES = OP == kWgrad8 ? 6 : 4;
  static constexpr uint32_t SCALES = OP == kWgrad8 ? SLOTS8 * SLOT_FLOATS8 * 4 : 0;
  static constexpr uint32_t ROW = ACC8 * 2 + 16, STASH = OP == kWgrad8 ? 32 * 64 : 32 * ROW;
};

struct Params8 {
  CUtensorMap tmA, tmA128, tmB;
  int N, K;       // forward, dgrad: the output's contiguous extent, the sum's length
  int M;          // wgrad: the output's contiguous extent (N: its rows)
  int groups, rows, bn;
  int vec, out_type;
  int b_whole;    // tmB's box is the CTA's whole tile of B
  uint32_t idesc;
  const int32_t* offsets;
  void* out;
  long long ld, stride;
  const float *sa, *sb;       // scales of A and of B
  long long sa_ld, sb_ld;     // distance of a row scale's (column scale's) blocks
  long long sb_group;         // forward, dgrad: of the matrices' scales,
  int sb_n, sb_k;             // and strides of a block along n and along the sum
  int* status;
  unsigned long long epi_wait_ns;
};

struct Unit8 {
  int m0, n0;       // the tile's first token (wgrad: first k) and first n
  int mcount, ncount;  // how many of its 256 x bn exist
  int group, kb0, kbs;  // kb0: the sum's first block of 128 (wgrad: of the laid-out rows)
};

// Deals out the tiles: a group's tokens in tiles of 256, each with all tiles of n in turn; wgrad: the output's
// tiles of every group.
template <Op8 OP>
struct Walk8 {
  static constexpr bool A_MN = OP == kWgrad8, B_MN = OP != kForward8, RAGGED_SUM = OP == kWgrad8;
  static constexpr int BOX = 32;  // few tokens: the small box of A (the large one has 128 rows)
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
      if (!A_MN) tma_prefetch_desc(&a.tmA128);
    }
    let_next_start();
    wait_for_previous();
    if (threadIdx.x >= 32) return;
    if (clamp_offsets(a.offsets, a.groups, a.rows, off) && lane == 0 && blockIdx.x == 0) atomicExch(a.status, OZ_EINVAL);
    __syncwarp();
    if (RAGGED_SUM) return;
    const int tiles_n = ceil_div(a.N, a.bn);
    int sum = 0;
    for (int b = 0; b <= a.groups; b += 32) {
      const int i = b + lane;
      int t = i >= 1 && i <= a.groups ? ceil_div(off[i] - off[i - 1], BM) * tiles_n : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, t, d);
        if (lane >= d) t += o;
      }
      if (i <= a.groups) prefix[i] = sum + t;
      sum += __shfl_sync(0xFFFFFFFFu, t, 31);
    }
  }

  // at: the tile before the pair's next one.
  __device__ Walk8(const Params8& p, const int* table, int at) : a(p), off(table), prefix(table + OZ_MAX_GROUPS + 1) {
    tiles_m = RAGGED_SUM ? ceil_div(a.M, BM) : 0;
    tiles_n = ceil_div(a.N, a.bn);
    total = RAGGED_SUM ? a.groups * tiles_m * tiles_n : prefix[a.groups];
    idx = at;
  }
  __device__ Walk8(const Params8& p, const int* table)
      : Walk8(p, table, static_cast<int>(blockIdx.x >> 1) - static_cast<int>(gridDim.x >> 1)) {}

  __device__ bool next(Unit8& u) {
    idx += static_cast<int>(gridDim.x >> 1);
    if (idx >= total) return false;
    if (RAGGED_SUM) {
      const int per = tiles_m * tiles_n;
      u.group = idx / per;
      const int r = idx - u.group * per, tn = r / tiles_m;
      u.m0 = (r - tn * tiles_m) * BM;
      u.mcount = min(BM, a.M - u.m0);
      u.n0 = tn * a.bn;
      u.kbs = ceil_div(off[u.group + 1] - off[u.group], BK8);
      u.kb0 = a.offsets ? first_column_block(off[u.group], u.group) : 0;
    } else {
      u.group = group_of(prefix, a.groups, idx);
      const int r = idx - prefix[u.group], tm = r / tiles_n;
      u.m0 = off[u.group] + tm * BM;
      u.mcount = min(BM, off[u.group + 1] - u.m0);
      u.n0 = (r - tm * tiles_n) * a.bn;
      u.kbs = ceil_div(a.K, BK8);
      u.kb0 = 0;
    }
    u.ncount = min(a.bn, a.N - u.n0);
    return true;
  }

  // Rows that belong to no group are zero.
  __device__ void outside(int warp) const {
    if (RAGGED_SUM || !a.offsets) return;
    const int lo = off[0], hi = off[a.groups], loose = lo + a.rows - hi;
    for (int i = static_cast<int>(blockIdx.x) * EPI8_WARPS + warp; i < loose; i += gridDim.x * EPI8_WARPS) {
      uint16_t* row = static_cast<uint16_t*>(a.out) + static_cast<long long>(i < lo ? i : hi + i - lo) * a.ld;
      for (int c = threadIdx.x & 31; c < a.N; c += 32) row[c] = 0;
    }
  }
};

// High words of the shared-memory descriptors.  MN-major B lies in rows of 64 bytes, so that an accumulator's 64
// columns of a CTA are a tile of their own: 64-byte swizzle, 8 k rows are 512 bytes.
constexpr uint32_t DESC_HIGH_64 = (512u >> 4) | (1u << 14) | (4u << 29);

template <uint32_t B_HIGH>
__device__ __forceinline__ void umma8_pair(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(DESC_HIGH), "r"(B_HIGH)
      : "memory");
}

// Instruction descriptor of kind::f8f6f4 with FP32 sums, without its N field (formats: 0 e4m3, 1 e5m2).
constexpr uint32_t idesc8_base(int fa, int fb, bool a_mn, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(fa) << 7) | (static_cast<uint32_t>(fb) << 10) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(BM >> 4) << 24);
}

// c += a b for an a from tensor memory.  volatile: stays behind the wait for the tensor-memory load.
__device__ __forceinline__ void fma_loaded(float a, float b, float& c) { asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(c) : "f"(a), "f"(b)); }
// Two neighbouring sums: c += v (b s).
__device__ __forceinline__ void fma_loaded(float v0, float v1, float2 b, float s, float& c0, float& c1) {
  asm volatile(
      "{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%4, %5};\n\tmov.b64 y, {%6, %6};\n\tmul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 y, {%2, %3};\n\tmov.b64 z, {%0, %1};\n\tfma.rn.f32x2 z, y, x, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "+f"(c0), "+f"(c1)
      : "f"(v0), "f"(v1), "f"(b.x), "f"(b.y), "f"(s));
}

// 32 finished columns of this lane's row into its row of the stash.
__device__ __forceinline__ void stash_row(uint8_t* row, const float (&v)[32], bool bf16) {
  uint32_t w[16];
  pack_block(v, w, bf16);
#pragma unroll
  for (int p = 0; p < 4; ++p) *reinterpret_cast<uint4*>(row + 16 * p) = make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
}

// The warp's finished rows from its stash (`pitch` bytes a row) to the output.  Each lane sends its own row off as a bulk
// copy, which the next tile's sums do not wait for (8192 x 4096 x 8192: 224 us; 226 with 16-byte stores by the lanes, 202
// with no stores at all).  Elements behind the last whole 16 bytes are stored one by one, and so is everything where
// rows do not start at multiples of 16 bytes.  row0, col: the first; rows, cols: how many exist.
__device__ __forceinline__ void send_rows(const Params8& a, uint8_t* stash, uint32_t pitch, long long row0, int rows, int col, int cols) {
  const int lane = threadIdx.x & 31;
  cols = min(cols, ACC8);
  uint16_t* out = static_cast<uint16_t*>(a.out) + row0 * a.ld + col;
  if (a.vec) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if (lane < rows) {
      const uint8_t* from = stash + lane * pitch;
      uint16_t* to = out + lane * a.ld;
      const int whole = cols & ~7;
      if (whole)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(smem_u32(from)), "r"(2 * whole) : "memory");
      for (int c = whole; c < cols; ++c) to[c] = reinterpret_cast<const uint16_t*>(from)[c];
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  } else {
    __syncwarp();
    for (int r = 0; r < min(rows, 32); ++r)
      for (int c = lane; c < cols; c += 32) out[r * a.ld + c] = reinterpret_cast<const uint16_t*>(stash + r * pitch)[c];
    __syncwarp();
  }
}

// 32 lanes x 16 columns in the fragments of tcgen05.ld.16x256b.x2: element i is
//   m = 16 (i / 8) + lane / 4 + 8 ((i / 2) % 2),   n = 8 ((i / 4) % 2) + 2 (lane % 4) + i % 2
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[8 * h]), "=f"(v[8 * h + 1]), "=f"(v[8 * h + 2]), "=f"(v[8 * h + 3]), "=f"(v[8 * h + 4]), "=f"(v[8 * h + 5]),
                   "=f"(v[8 * h + 6]), "=f"(v[8 * h + 7])
                 : "r"(taddr + (h ? 16u << 16 : 0u)));
}

template <Op8 OP>
__global__ void __launch_bounds__(THREADS8, 1) block8_kernel(const __grid_constant__ Params8 a) {
  typedef Walk8<OP> Walk;
  constexpr int STAGES8 = Smem8<OP>::STAGES;
  constexpr uint32_t STASH8 = Smem8<OP>::STASH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES8 * TILE8;
  float* scales = reinterpret_cast<float*>(smem + 2 * STAGES8 * TILE8);
  uint8_t* stash = smem + 2 * STAGES8 * TILE8 + Smem8<OP>::SCALES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stash + EPI8_WARPS * STASH8);
  uint64_t* full = bars;                     // [STAGES8] TMA (both CTAs) -> MMA  (used in the leader)
  uint64_t* empty = full + STAGES8;          // [STAGES8] MMA issuers -> TMA      (both CTAs)
  uint64_t* accfull = empty + STAGES8;       // [4]       MMA -> epilogue, by buffer and half (both CTAs)
  uint64_t* accempty = accfull + 4;          // [4]       the half's warps (both) -> MMA (used in the leader)
  uint64_t* sfull = accempty + 4;            // [SLOTS8]  scales -> epilogue      (per CTA)
  uint64_t* sempty = sfull + SLOTS8;         // [SLOTS8]  epilogue -> scales      (per CTA)
  uint64_t* drain = sempty + SLOTS8;         // [1]       all MMAs of the pair done, by each issuer (both CTAs)
  uint64_t* exitbar = drain + 1;             // [1]       the peer has finished (per CTA)
  uint64_t* proddone = exitbar + 1;          // [1]       both producers have stopped (used in the leader)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(proddone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued_by = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);  // [2] (leader)
  int* table = reinterpret_cast<int*>(stash + EPI8_WARPS * STASH8 + 512);               // the walker's

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  // Accumulator buf * halves + half: two buffers of two halves, or four of one.
  const uint32_t halves = OP == kWgrad8 ? 2 : a.bn / ACC8, buffers = 4 / halves;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES8; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], halves);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], EPI8_WARPS);  // four warps of either CTA
    }
    for (int i = 0; i < SLOTS8; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], EPI8_WARPS);
    }
    mbar_init(drain, halves);
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
        Unit8 u{};
        bool ok = true;
        while (ok && !*abort_flag && walk.next(u)) {
          const int m = u.m0 + static_cast<int>(rank) * HALF_M;
          // Tokens: only what the tile has, in one box of 128 or in boxes of 32.  What the stage holds in the other rows
          // are sums of rows that are not stored.
          const int have = min(HALF_M, u.mcount - static_cast<int>(rank) * HALF_M);
          const bool whole = Walk::A_MN || have > 64;
          const int boxes = whole ? 1 : max(0, ceil_div(max(have, 0), Walk::BOX));
          const uint32_t bytes = (whole ? TILE8 : boxes * Walk::BOX * BK8) + halves * HALF8;
          for (int kb = u.kb0; kb < u.kb0 + u.kbs; ++kb) {
            if (!mbar_wait_or_abort(&empty[stage], phase ^ 1, kWaitLimitNs, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t bar = full_leader + stage * 8;
            mbar_arrive_expect_tx_cluster(bar, bytes);
            uint8_t* dA = sA + stage * TILE8;
            uint8_t* dB = sB + stage * TILE8;
            const int k = kb * BK8;
            const int z = OP == kWgrad8 ? 0 : u.group;
            if (a.b_whole) {
              if (Walk::B_MN)
                tma_load_5d_pair(dB, &a.tmB, bar, 0, k, static_cast<int>(rank), u.n0 / ACC8, z);
              else
                tma_load_4d_pair(dB, &a.tmB, bar, k, 64 * static_cast<int>(rank), u.n0 / ACC8, z);
            } else {
              for (int h = 0; h < static_cast<int>(halves); ++h) {
                const int n = u.n0 + ACC8 * h + 64 * static_cast<int>(rank);
                if (Walk::B_MN)
                  tma_load_3d_pair(dB + h * HALF8, &a.tmB, bar, n, k, z);
                else
                  tma_load_3d_pair(dB + h * HALF8, &a.tmB, bar, k, n, z);
              }
            }
            if (Walk::A_MN)
              tma_load_3d_pair(dA, &a.tmA, bar, m, k, 0);
            else if (whole)
              tma_load_3d_pair(dA, &a.tmA128, bar, k, m, 0);
            else
              for (int b = 0; b < boxes; ++b) tma_load_3d_pair(dA + b * Walk::BOX * BK8, &a.tmA, bar, k, m + Walk::BOX * b, 0);
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
    } else if (warp & 1) {
      const uint32_t half = warp >> 1;
      if (rank == 0 && half < halves && elect_one()) {
        // ------------------------------------------------------------ MMA issuers (leader only), one for each half
        int stage = 0;
        uint32_t phase = 0, buf = 0, acc_phase = 1, consumed = 0;
        bool ok = true;
        const uint32_t a_desc = desc_low(smem_u32(sA), Walk::A_MN), b_desc = desc_low(smem_u32(sB) + half * HALF8, Walk::B_MN);
        constexpr uint32_t a_step = (Walk::A_MN ? STEP8 * 128 : STEP8) >> 4, b_step = (Walk::B_MN ? STEP8 * 64 : STEP8) >> 4;
        constexpr uint32_t B_HIGH = Walk::B_MN ? DESC_HIGH_64 : DESC_HIGH;
        const uint32_t idesc = a.idesc;
        Walk walk(a, table);
        Unit8 u{};
        while (ok && !*abort_flag && walk.next(u)) {
          for (int left = u.kbs; left > 0; --left) {
            if (!mbar_wait_or_abort(&full[stage], phase, kWaitLimitNs, abort_flag)) {
              ok = false;
              break;
            }
            ++consumed;
            const uint32_t acc = buf * halves + half;
            if (!mbar_wait_or_abort(&accempty[acc], acc_phase, kWaitLimitNs, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t ad = a_desc + stage * (TILE8 >> 4), bd = b_desc + stage * (TILE8 >> 4), d = tmem_base + acc * ACC8;
#pragma unroll
            for (int kk = 0; kk < BK8 / STEP8; ++kk) umma8_pair<B_HIGH>(d, ad + kk * a_step, bd + kk * b_step, idesc, kk > 0 ? 1u : 0u);
            umma_commit_pair(&accfull[acc], 0x3);
            umma_commit_pair(&empty[stage], 0x3);
            if (++buf == buffers) {
              buf = 0;
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
        if (half == 0) {
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
        }
        umma_commit_pair(drain, 0x3);
      }
    } else if (warp == 2 && OP == kWgrad8) {
      // -------------------------------------------------------------- scales (both CTAs)
      // A slot holds a k-block's scales of the tile's n and of the CTA's m.  BATCH8 blocks are fetched at once, while
      // the epilogue uses the ones before.
      int slot = 0;
      uint32_t sphase = 1;
      bool ok = true;
      Walk walk(a, table);
      Unit8 u{};
      while (ok && !*abort_flag && walk.next(u)) {
        const int m0 = u.m0 + static_cast<int>(rank) * HALF_M, mine = u.mcount - static_cast<int>(rank) * HALF_M;
        const float* sm = a.sa + u.kb0 * a.sa_ld + m0;
        const float* sn = a.sb + u.kb0 * a.sb_ld + u.n0;
        for (int kb = 0; ok && kb < u.kbs; kb += BATCH8) {
          float n[BATCH8][8], m[BATCH8][4];
#pragma unroll
          for (int j = 0; j < BATCH8; ++j) {
            const bool have = kb + j < u.kbs;
#pragma unroll
            for (int i = 0; i < 8; ++i) n[j][i] = have && lane + 32 * i < u.ncount ? sn[(kb + j) * a.sb_ld + lane + 32 * i] : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) m[j][i] = have && lane + 32 * i < mine ? sm[(kb + j) * a.sa_ld + lane + 32 * i] : 0.0f;
          }
#pragma unroll
          for (int j = 0; j < BATCH8; ++j) {
            if (kb + j < u.kbs && ok) {
              ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&sempty[slot], sphase, kWaitLimitNs, abort_flag));
              if (ok) {
                float* to = scales + slot * SLOT_FLOATS8;
#pragma unroll
                for (int i = 0; i < 8; ++i) to[lane + 32 * i] = n[j][i];
#pragma unroll
                for (int i = 0; i < 4; ++i) to[256 + lane + 32 * i] = m[j][i];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sfull[slot]);
                if (++slot == SLOTS8) {
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
    // A warp scales and sums 32 lanes of one half's 128 columns.
    const uint32_t half = (warp - EPI8_FIRST) >> 2;
    const int quad = warp & 3;
    uint8_t* my_stash = stash + (warp - EPI8_FIRST) * STASH8;
    const uint32_t accempty_leader = mapa_shared(smem_u32(accempty), 0);
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const int mrow = static_cast<int>(rank) * HALF_M + quad * 32;
    uint32_t acc = half, acc_phase = 0;  // its accumulators: half, half + halves, ...
    bool ok = true;
    Walk(a, table).outside(warp - EPI8_FIRST);
    auto wait = [&](uint64_t* bar, uint32_t phase, uint64_t limit) {
      if (__all_sync(0xFFFFFFFFu, limit ? mbar_try_wait(bar, phase) : mbar_test_wait(bar, phase))) return true;
      ok = limit && __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar, phase, limit, abort_flag));
      if (!ok && lane == 0 && !*abort_flag) stop_pair(abort_flag, a.status);
      return ok;
    };
    auto sums_there = [&]() {
      const bool there = wait(&accfull[acc], acc_phase, a.epi_wait_ns);
      tc_fence_after();
      return there;
    };
    // All of this warp's sums of an accumulator are in registers: it goes back to the MMAs.
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(accempty_leader + acc * 8);
      if ((acc += halves) >= 4) {
        acc = half;
        acc_phase ^= 1;
      }
    };
    // Whether the accumulator after this one is full by now: asked EARLY8 reads before the answer is needed, as a wait that
    // is over at once takes 80 cycles of a k-block's 820 (8192 x 4096 x 8192: 224 us instead of 228; wgrad of 32768 rows
    // and 16 groups, which waits for scales too: 386 instead of 405).
    auto next_there = [&]() {
      const bool turn = acc + halves >= 4;
      return mbar_test_wait(&accfull[turn ? half : acc + halves], acc_phase ^ (turn ? 1u : 0u));
    };
    if constexpr (OP != kWgrad8) {
      // The sums take nearly all registers: the walker is made anew for each tile, and where the tile goes waits in the
      // warp's stash.
      int4* const kept = reinterpret_cast<int4*>(my_stash + ACC8 * 2);  // first row, rows, first column, columns
      int at = static_cast<int>(blockIdx.x >> 1) - static_cast<int>(gridDim.x >> 1);
      int left = 0, blocks = 0;  // k-blocks to come, blocks of 32 columns
      const float *sx, *sw;      // this lane's row's scales (lanes without a row take the last one's), the half's features'
      // Scales are fetched two k-blocks ahead and multiplied only when they are used (a product formed at once would
      // wait for both); a tile's first ones before the tile before it is stored.
      float x[2] = {}, w[2] = {};
      auto begin = [&]() {
        Walk walk(a, table, at);
        at += static_cast<int>(gridDim.x >> 1);
        Unit8 u;
        if (!walk.next(u)) return false;
        const int rows = u.mcount - mrow, col = u.n0 + static_cast<int>(half) * ACC8, cols = u.ncount - static_cast<int>(half) * ACC8;
        blocks = rows > 0 ? min(BLOCKS8, ceil_div(max(0, cols), 32)) : 0;
        left = u.kbs;
        sx = a.sa + u.m0 + mrow + min(lane, rows - 1);
        sw = a.sb + u.group * a.sb_group + static_cast<long long>(col / 128) * a.sb_n;
        __syncwarp();
        if (lane == 0) *kept = make_int4(u.m0 + mrow, rows, col, cols);
        if (blocks && left) {
          x[0] = x[1] = *sx;
          w[0] = w[1] = *sw;
          if (left > 1) {
            x[1] = *(sx += a.sa_ld);
            w[1] = *(sw += a.sb_k);
          }
        }
        return true;
      };
      for (bool more = half < halves && begin(); ok && more;) {
        float run[BLOCKS8][32];
#pragma unroll
        for (int i = 0; i < BLOCKS8 * 32; ++i) run[i >> 5][i & 31] = 0.0f;
        const int tile_blocks = blocks;
        auto factor = [&](float& x, float& w) {
          const float f = x * w;
          if (left > 2) {
            x = *(sx += a.sa_ld);
            w = *(sw += a.sb_k);
          }
          return f;
        };
        if (blocks == BLOCKS8) {
          // Half a block is read while the one before it is scaled and added, across k-blocks too; after the last one
          // the read is of a free accumulator's columns, and dropped.
          uint32_t v[2][16];
          auto step = [&](float& x, float& w) {
            const float f = factor(x, w);
            bool early = false;
#pragma unroll
            for (int j = 0; j < 2 * BLOCKS8; ++j) {
              tmem_ld_wait();
              if (j + EARLY8 == 2 * BLOCKS8) early = next_there();
              if (j + 1 == 2 * BLOCKS8) {
                release();
                if (--left > 0) {
                  if (__all_sync(0xFFFFFFFFu, early)) tc_fence_after();
                  else sums_there();
                }
              }
              tmem_ld16(lanes + acc * ACC8 + 16 * ((j + 1) % (2 * BLOCKS8)), v[(j + 1) & 1]);
#pragma unroll
              for (int i = 0; i < 16; ++i) fma_loaded(__uint_as_float(v[j & 1][i]), f, run[j >> 1][16 * (j & 1) + i]);
            }
          };
          if (left > 0 && sums_there()) {
            tmem_ld16(lanes + acc * ACC8, v[0]);
            // Two k-blocks a turn, so that no scale under way is moved from one register to another.
            while (ok && left > 0) {
              step(x[0], w[0]);
              if (!ok || left == 0) break;
              step(x[1], w[1]);
            }
            tmem_ld_wait();
          }
        } else {
          auto step = [&](float& x, float& w) {
            const float f = blocks ? factor(x, w) : 0.0f;
            const uint32_t from = lanes + acc * ACC8;
            --left;
            if (blocks == 0) release();
#pragma unroll
            for (int j = 0; j < BLOCKS8 - 1; ++j) {
              if (j < blocks) {
                uint32_t v[32];
                tmem_ld32(from + 32 * j, v);
                tmem_ld_wait();
                if (j + 1 == blocks) release();
#pragma unroll
                for (int i = 0; i < 32; ++i) fma_loaded(__uint_as_float(v[i]), f, run[j][i]);
              }
            }
          };
          while (left > 0 && sums_there()) {
            step(x[0], w[0]);
            if (left == 0 || !sums_there()) break;
            step(x[1], w[1]);
          }
        }
        if (!ok) break;
        __syncwarp();
        const int4 to = *kept;
        __syncwarp();
        more = begin();
        if (tile_blocks) {
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the stash's last rows have left it
#pragma unroll
          for (int j = 0; j < BLOCKS8; ++j)
            if (j < tile_blocks) stash_row(my_stash + lane * Smem8<OP>::ROW + 64 * j, run[j], a.out_type == kOutBf16);
          send_rows(a, my_stash, Smem8<OP>::ROW, to.x, to.y, to.z, to.w);
        }
      }
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else {
      uint32_t slot = 0, sphase = 0;
      auto scales_there = [&]() { return wait(&sfull[slot], sphase, kWaitLimitNs); };
      auto scales_done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[slot]);
        if (++slot == SLOTS8) {
          slot = 0;
          sphase ^= 1;
        }
      };
      Unit8* const kept = reinterpret_cast<Unit8*>(my_stash);
      for (int at = static_cast<int>(blockIdx.x >> 1) - static_cast<int>(gridDim.x >> 1); ok; at += static_cast<int>(gridDim.x >> 1)) {
        int left, blocks;
        {
          Walk walk(a, table, at);
          Unit8 u;
          if (!walk.next(u)) break;
          blocks = u.mcount > mrow ? min(BLOCKS8, ceil_div(max(0, u.ncount - static_cast<int>(half) * ACC8), 32)) : 0;
          left = u.kbs;
          __syncwarp();
          if (lane == 0) *kept = u;
        }
        float run[BLOCKS8][32];
#pragma unroll
        for (int i = 0; i < BLOCKS8 * 32; ++i) run[i >> 5][i & 31] = 0.0f;
        if (blocks) {
          // 16 columns are read while the ones before them are scaled and added, across k-blocks too: all 128, whether the
          // tile has them or not, and 16 of a free accumulator after the last k-block.
          float v[2][16], sm[4];
          auto scales_of_m = [&]() {
#pragma unroll
            for (int h = 0; h < 4; ++h) sm[h] = scales[slot * SLOT_FLOATS8 + 256 + quad * 32 + (lane >> 2) + 8 * h];
          };
          if (left > 0 && sums_there() && scales_there()) {
            scales_of_m();
            tmem_ld_frag16(lanes + acc * ACC8, v[0]);
          }
          while (ok && left > 0) {
            bool early = false;
#pragma unroll
            for (int j = 0; j < 2 * BLOCKS8; ++j) {
              if (j + EARLY8 == 2 * BLOCKS8) {
                early = next_there() & mbar_test_wait(&sfull[slot + 1 == SLOTS8 ? 0 : slot + 1], sphase ^ (slot + 1 == SLOTS8 ? 1u : 0u));
              }
              float2 s[2];
#pragma unroll
              for (int q = 0; q < 2; ++q)
                s[q] = *reinterpret_cast<const float2*>(scales + slot * SLOT_FLOATS8 + half * ACC8 + 2 * (lane & 3) + 16 * j + 8 * q);
              tmem_ld_wait();
              if (j + 1 == 2 * BLOCKS8) {
                release();
                scales_done();
                if (--left > 0) {
                  if (__all_sync(0xFFFFFFFFu, early)) tc_fence_after();
                  else if (scales_there()) sums_there();
                }
              }
              tmem_ld_frag16(lanes + acc * ACC8 + 16 * ((j + 1) % (2 * BLOCKS8)), v[(j + 1) & 1]);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {  // m = lane / 4 + 8 h, n = 16 j + 8 q + 2 (lane % 4), + 1
                  const int i = 8 * (h >> 1) + 4 * q + 2 * (h & 1), r = 16 * (h >> 1) + 8 * (j & 1) + 4 * q + 2 * (h & 1);
                  fma_loaded(v[j & 1][i], v[j & 1][i + 1], s[q], sm[h], run[j >> 1][r], run[j >> 1][r + 1]);
                }
              }
            }
            if (ok && left > 0) scales_of_m();
          }
          tmem_ld_wait();
        } else {
          for (; left > 0 && sums_there() && scales_there(); --left) {
            release();
            scales_done();
          }
        }
        if (!ok) break;
        __syncwarp();
        const Unit8 u = *kept;
        __syncwarp();
        Unit t{};  // as the 16-bit products' epilogue takes it
        t.m0 = u.m0;
        t.m_extent = a.M;
        t.nn = u.ncount - static_cast<int>(half) * ACC8;
        t.orow = u.n0 + static_cast<int>(half) * ACC8;
        t.out = static_cast<uint16_t*>(a.out) + u.group * a.stride;
        t.ld = a.ld;
        t.out_type = a.out_type;
        t.vec = a.vec;
        const Target target = target_of(t, mrow, my_stash);
#pragma unroll
        for (int j = 0; j < BLOCKS8; ++j)
          if (j < blocks) emit<false, true>(t, target, run[j], j, my_stash);
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
// A tensor map of bytes, swizzled over its rows of 128 or 64 bytes (box[0]).
bool encode8(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const EncodeTiled fn = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, box[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  uint64_t pitch() const { return rows > 1 ? ld : roundup(cols, 16); }  // one row has no stride to speak of
  uint64_t mat_pitch() const { return mats > 1 ? stride : pitch() * rows; }
  // [mats][rows][cols], box {box_cols, box_rows, 1}.
  bool map(CUtensorMap* m, int box_cols, int box_rows) const {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(mats)};
    const cuuint64_t strides[2] = {pitch(), mat_pitch()};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    return encode8(m, p, 3, dims, strides, box);
  }
  // B, where its n are whole blocks of 128: a box holds 64 n of each of `halves` neighbouring blocks.
  //   K-major:  [mats][n / 128][128][k], box {128, 64, halves, 1}
  //   MN-major: [mats][n / 128][2][k][64], box {64, 128, 1, halves, 1}
  bool map_halves(CUtensorMap* m, bool mn, int halves) const {
    const cuuint32_t h = static_cast<cuuint32_t>(halves);
    if (mn) {
      const cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(rows), 2, static_cast<cuuint64_t>(cols / 128), static_cast<cuuint64_t>(mats)};
      const cuuint64_t strides[4] = {pitch(), 64, 128, mat_pitch()};
      const cuuint32_t box[5] = {64, 128, 1, h, 1};
      return encode8(m, p, 5, dims, strides, box);
    }
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(cols), 128, static_cast<cuuint64_t>(rows / 128), static_cast<cuuint64_t>(mats)};
    const cuuint64_t strides[3] = {pitch(), 128 * pitch(), mat_pitch()};
    const cuuint32_t box[4] = {128, 64, h, 1};
    return encode8(m, p, 4, dims, strides, box);
  }
};

struct Problem8 {
  Op8 op;
  int n, k, rows, groups;
  Operand8 a, b;  // A: X, or dY (dgrad); B: W, or dY (wgrad)
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
  if (p.op == kWgrad8 ? p.lds_a < (p.k > 1 ? p.k : 1) || p.lds_b < (p.n > 1 ? p.n : 1) : p.lds_a < (p.rows > 1 ? p.rows : 1)) return OZ_EINVAL;
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
  a.N = OP == kDgrad8 ? p.k : p.n;
  a.K = OP == kForward8 ? p.k : p.n;
  a.M = p.k;
  a.groups = p.groups;
  a.rows = p.rows;
  a.bn = BN;
  // Tiles of 128 n where that takes fewer turns of all pairs: they take 0.72 of the time of tiles of 256 (8192 x 4096 x
  // 8192: 325 us, and 227; 64 rows x 4096 x 8192, one turn of either: 16.3 us, and 18.9).  (The rows of each
  // group are not known here: at most so many tiles.)
  if (OP != kWgrad8) {
    const int tiles_m = p.groups == 1 ? ceil_div(p.rows, BM) : (p.groups < p.rows ? p.groups : p.rows) + p.rows / BM;
    const long long wide = static_cast<long long>(tiles_m) * ceil_div(a.N, BN), narrow = static_cast<long long>(tiles_m) * ceil_div(a.N, ACC8);
    if ((narrow + d.pairs - 1) / d.pairs * 18 < (wide + d.pairs - 1) / d.pairs * 25) a.bn = ACC8;
  }
  a.vec = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.ldo % 8 == 0 && (OP != kWgrad8 || p.groups == 1 || p.strideo % 8 == 0);
  a.out_type = p.out_type == OZ_BF16 ? kOutBf16 : kOutF16;
  a.idesc = idesc8_base(p.a.type == OZ_E5M2, p.b.type == OZ_E5M2, Walk::A_MN, Walk::B_MN) | (static_cast<uint32_t>(ACC8 >> 3) << 17);
  a.offsets = p.offsets;
  a.out = p.out;
  a.ld = p.ldo;
  a.stride = p.strideo;
  a.sa = p.a.scales;
  a.sb = p.b.scales;
  a.sa_ld = p.lds_a;
  a.sb_ld = p.lds_b;
  const int kb = ceil_div(p.k, 128);
  a.sb_group = static_cast<long long>(ceil_div(p.n, 128)) * kb;
  a.sb_n = OP == kForward8 ? kb : 1;
  a.sb_k = OP == kForward8 ? 1 : kb;
  a.b_whole = a.N % 128 == 0;
  bool ok = (a.b_whole ? p.b.map_halves(&a.tmB, Walk::B_MN, a.bn / ACC8) : p.b.map(&a.tmB, Walk::B_MN ? 64 : 128, Walk::B_MN ? 128 : 64)) &&
            p.a.map(&a.tmA, 128, OP == kWgrad8 ? 128 : Walk::BOX);
  if (OP != kWgrad8) ok = ok && p.a.map(&a.tmA128, 128, 128);
  if (!ok) return OZ_ECUDA;
  a.status = d.status;
  a.epi_wait_ns = epilogue_wait_ns();
  auto kernel = block8_kernel<OP>;
  constexpr size_t smem = 1024 /*alignment*/ + 2 * Smem8<OP>::STAGES * TILE8 + Smem8<OP>::SCALES + EPI8_WARPS * Smem8<OP>::STASH + 512 /*barriers*/ + Walk::kTableBytes;
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
  return run8(Problem8{kForward8, n, k, rows, groups, {X, type_x, k, rows, 1, ldx, 0, SX}, {W, type_w, k, n, groups, ldw, strideW, SW},
                       ldsx, 0, offsets, dtype, Y, ldy, 0}, stream);
}
int ozaki_grouped_gemm_f8_dgrad(int n, int k, int rows, int groups, int type_w, const void* W, int ldw, long long strideW, const float* SW,
                                int type_dy, const void* dY, int lddy, const float* SdY, int ldsdy, const int32_t* offsets, int dtype,
                                void* dX, int lddx, cudaStream_t stream) {
  return run8(Problem8{kDgrad8, n, k, rows, groups, {dY, type_dy, n, rows, 1, lddy, 0, SdY}, {W, type_w, k, n, groups, ldw, strideW, SW},
                       ldsdy, 0, offsets, dtype, dX, lddx, 0}, stream);
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
