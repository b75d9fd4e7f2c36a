// oz_products.cuh -- the tensor-core kernel behind the grouped expert products and the
// Newton-Schulz iteration: many 16-bit matrix products of different extents in one launch.
//
// Every product is D[m, n] = sum_k A[m, k] B[n, k] with FP32 sums, where m runs along the
// output's contiguous dimension and n over its rows.  That orientation is chosen for all
// operators: an accumulator lane is then one contiguous output element, so a warp's 32 lanes
// are 64 contiguous bytes of an output row, and a ragged number of output rows (the tokens of
// an expert) is the MMA's N, which takes any multiple of 32, so a short expert does not pay
// for a full tile.  Either operand may be K-contiguous ("K-major") or m/n-contiguous
// ("MN-major"); the tensor core reads both from the 128-byte-swizzled tiles that TMA writes,
// so nothing is ever transposed in memory.
//
// Ragged sums (the weight gradient sums over an expert's rows): the k-blocks of 64 rows are
// aligned to the END of the expert's rows, and its rows are addressed as (offset within the
// expert, first row): the first block starts at a negative offset, which TMA fills with
// zeros.  No row of a neighbouring expert is ever read into a sum, so its NaNs cannot leak.
//
// Kernel shape: clusters of two CTAs (cta_group::2), persistent over units (tile, split).
//   warp 0: TMA producer   warp 1: TMEM owner + MMA issuer (leader)   warps 2-9: epilogue
//   6 stages of 32 KB (128 x 64 of A and up to 128 x 64 of B in each CTA); two 256-column
//   FP32 accumulators in tensor memory, so a tile's epilogue runs under the next one's MMAs.
// Split k: when there are fewer tiles than CTA pairs, a tile's k range is cut into nsplit
// parts.  Each part's FP32 sums go to the workspace, and the CTA that arrives last (an atomic
// counter per tile and CTA) adds the parts in their order, so results do not depend on timing
// and nobody waits.
// Two slices (PLANES == 2): operands are h + l with h, l in FP16.  h h' has an accumulator of
// its own and h l' + l h' (2^-11 of it) another, tiles being 128 wide at most; the tensor core
// truncates as it accumulates, so the sums are taken out every `chunk` MMA steps and
// continued in FP32 registers (round to nearest).
// Every wait is bounded (as in the residue GEMM): on expiry the pair records OZ_ETIMEOUT,
// drains what it issued and returns.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "oz_device.cuh"
#include "oz_internal.h"

namespace oz {
namespace prod {

constexpr int BM = 256, HALF_M = 128;
constexpr int BN = 256, HALF_N = 128;
constexpr int BK = 64;
constexpr int UMMA_K = 16;
constexpr int KSTEPS = BK / UMMA_K;
constexpr int STAGES = 6;
constexpr uint32_t A_STAGE = HALF_M * BK * 2;
constexpr uint32_t B_STAGE = HALF_N * BK * 2;
constexpr uint32_t STAGE_BYTES = A_STAGE + B_STAGE;
constexpr uint32_t MN_BLOCK = 64 * BK * 2;  // 64 contiguous m (or n) x 64 k
constexpr int EPI_WARPS = 8;
constexpr int EPI_THREADS = EPI_WARPS * 32;
constexpr int THREADS = 64 + EPI_THREADS;
constexpr uint32_t TMEM_COLS = 512;
constexpr int BN2 = 128;                     // tile width with two slices
constexpr int CROSS = 128;                   // its second accumulator: columns past the first
constexpr uint32_t WARP_STASH = 32 * 32 * 2;  // 32 columns x 32 lanes of 16 bits, per epilogue warp
constexpr uint32_t STASH = EPI_WARPS * WARP_STASH;
constexpr int MAX_GROUPS = OZ_MAX_GROUPS;
constexpr uint32_t TABLE = 2 * (MAX_GROUPS + 1) * 4;  // row offsets and tile prefix of the groups
constexpr int BOX_ROWS = 32;                 // ragged rows: the small box of B (the large one has HALF_N rows)
constexpr size_t SMEM_DENSE = 1024 + STAGES * STAGE_BYTES + STASH + 256;
constexpr size_t SMEM_GROUPED = SMEM_DENSE + TABLE;
static_assert(SMEM_GROUPED <= 232448, "shared memory budget");

enum Mode { kDense = 0, kRaggedN = 1, kRaggedK = 2 };
enum OutType { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2, kOutSlices = 3 };

struct Args {
  int M, N, K;          // dense: the product's extents; ragged N: N unused; ragged K: K unused
  int groups;           // dense: matrices of the batch; otherwise the number of groups
  int tiles;            // dense: tiles of all matrices
  int rows;             // grouped: rows of the token matrices
  int bn;               // tile width in n
  int nsplit;           // dense: parts of the k range; grouped: chosen on the device (see split_for)
  int max_split_units;  // grouped: units the split workspace holds
  int sym;              // dense: the product is symmetric; tiles with n <= m only, mirrored
  int chunk;            // MMA steps (16 k) summed in one accumulator
  int out_type, planes_out;
  int vec;              // 16-byte stores are allowed (base and row stride)
  int box_rows;         // rows of one TMA box of a K-major B operand (ragged rows: of the small one)
  int a_4d, b_4d;       // MN-major operands: the map is 4-D and its box holds the CTA's whole tile
                        // (2 blocks of 64 of A, bn / 128 of B); otherwise 3-D, one block a box
  const int32_t* offsets;
  void* out;
  long long ld, stride;  // output row stride, stride between the groups' outputs (elements)
  long long plane;       // kOutSlices: distance of the low slices
  float alpha, diag;     // v = alpha v (* scale[group * scale_stride]), + diag on the diagonal
  const float* scale;    // null: 1
  int scale_stride;
  float* part;           // split workspace: [unit][2 CTAs][part_cols][128]
  unsigned int* counters;
  int part_cols;
  uint32_t idesc;        // instruction descriptor without N
  int* status;
  unsigned long long epi_wait_ns;
};

struct Unit {
  int group;
  int m0, n0;      // first output element of a row, first output row
  int orow;        // output row of n0 (grouped by rows: n0; otherwise n0 within the group)
  int nn, nmma;    // rows of the tile, the MMA's N
  int k0, kstart;  // coordinate of k-block 0, and the group's first row (ragged K)
  int kb0, kb1;    // k-blocks of this part
  int tile, split, nsplit;
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Parts of the k range for `tiles` tiles of nkb k-blocks on `pairs` CTA pairs: the count that
// minimises waves * (blocks of a part + fixed cost), the fixed cost in k-blocks.
__host__ __device__ inline int split_for(int tiles, int nkb, int pairs, int max_units, int fixed) {
  if (tiles <= 0 || tiles >= pairs) return 1;
  int best = 1, best_cost = 1 << 30;
  for (int s = 1; s <= 16 && s <= nkb && (s == 1 || tiles * s <= max_units); ++s) {
    const int cost = ceil_div(tiles * s, pairs) * (ceil_div(nkb, s) + fixed) + (s > 1 ? fixed : 0);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// Tiles of a symmetric product's row block tm: the column tiles that reach n <= m.
__host__ __device__ inline int sym_tiles(int tm, int tiles_n, int bn) {
  const int c = ceil_div((tm + 1) * BM, bn);
  return c < tiles_n ? c : tiles_n;
}

__host__ __device__ inline int dense_tiles(int M, int N, int bn, int sym) {
  const int tm = ceil_div(M, BM), tn = ceil_div(N, bn);
  if (!sym) return tm * tn;
  int t = 0;
  for (int i = 0; i < tm; ++i) t += sym_tiles(i, tn, bn);
  return t;
}

struct Schedule {
  int tiles, total, nsplit, first, step, tiles_m, tiles_n;
  const int* off;
  const int* prefix;
};

template <int MODE, bool B_MN>
__device__ __forceinline__ void unit_at(const Args& a, const Schedule& s, int idx, Unit& u) {
  u.nsplit = s.nsplit;
  u.tile = idx / s.nsplit;
  u.split = idx - u.tile * s.nsplit;
  int nkb;
  if (MODE == kDense) {
    const int per = s.tiles / a.groups;
    u.group = u.tile / per;
    int r = u.tile - u.group * per;
    int tm, tn;
    if (a.sym) {
      tm = 0;
      for (int c = sym_tiles(0, s.tiles_n, a.bn); r >= c; c = sym_tiles(tm, s.tiles_n, a.bn)) {
        r -= c;
        ++tm;
      }
      tn = r;
    } else {  // groups of 8 row blocks swept along the column tiles (L2 reuse of both operands)
      const int g = r / (8 * s.tiles_n);
      const int gm = min(8, s.tiles_m - 8 * g);
      r -= g * 8 * s.tiles_n;
      tm = 8 * g + r % gm;
      tn = r / gm;
    }
    u.m0 = tm * BM;
    u.n0 = u.orow = tn * a.bn;
    u.nn = min(a.bn, a.N - u.n0);
    u.k0 = u.kstart = 0;
    nkb = ceil_div(a.K, BK);
  } else if (MODE == kRaggedN) {
    int lo = 0, hi = a.groups;  // the group with prefix[g] <= tile < prefix[g + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.prefix[mid] <= u.tile) lo = mid; else hi = mid;
    }
    u.group = lo;
    const int r = u.tile - s.prefix[lo];
    const int tn = r / s.tiles_m;
    const int len = s.off[lo + 1] - s.off[lo];
    // equal tiles: the same number of them as with full ones, with the least padding
    const int w = ceil_div(ceil_div(len, ceil_div(len, a.bn)), 32) * 32;
    u.m0 = (r - tn * s.tiles_m) * BM;
    u.n0 = u.orow = s.off[lo] + tn * w;
    u.nn = min(w, len - tn * w);
    u.k0 = u.kstart = 0;
    nkb = ceil_div(a.K, BK);
  } else {
    const int per = s.tiles_m * s.tiles_n;
    u.group = u.tile / per;
    const int r = u.tile - u.group * per;
    const int tn = r / s.tiles_m;
    u.m0 = (r - tn * s.tiles_m) * BM;
    u.n0 = u.orow = tn * a.bn;
    u.nn = min(a.bn, a.N - u.n0);
    const int len = s.off[u.group + 1] - s.off[u.group];
    nkb = ceil_div(len, BK);
    u.k0 = len - nkb * BK;  // negative in the first block: TMA reads zeros there
    u.kstart = s.off[u.group];
  }
  u.nmma = B_MN ? ceil_div(u.nn, 128) * 128 : ceil_div(u.nn, 32) * 32;
  u.kb0 = static_cast<int>(static_cast<long long>(nkb) * u.split / s.nsplit);
  u.kb1 = static_cast<int>(static_cast<long long>(nkb) * (u.split + 1) / s.nsplit);
}

// Shared-memory descriptors, low word: address / 16 and the leading byte offset.  K-major tiles:
// rows of 64 k (128 bytes, 128-byte swizzle), 8 rows are 1024 bytes, no leading offset.
// MN-major tiles: blocks of 64 contiguous m (128 bytes a k row, 128-byte swizzle), 8 k rows are
// 1024 bytes, the next 64 m are MN_BLOCK bytes on.  The high word is the same for both.
template <bool MN>
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr) {
  return ((smem_addr >> 4) & 0x3FFFu) | ((MN ? MN_BLOCK >> 4 : 1u) << 16);
}
constexpr uint32_t DESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride, version, 128-byte swizzle

__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(DESC_HIGH)
      : "memory");
}

// Instruction descriptor of kind::f16 with FP32 accumulation, without its N field.
__host__ __device__ constexpr uint32_t idesc_base(bool bf16, bool a_mn, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(BM >> 4) << 24);
}

// Two values as 16-bit elements, the first in the low half.
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void stop_pair(volatile int* abort_flag, int* status) {
  *abort_flag = 1;
  st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), cluster_ctarank() ^ 1u), 1u);
  atomicExch(status, OZ_ETIMEOUT);
}

__device__ __forceinline__ bool warps_meet(uint64_t* bar, uint32_t& phase, const volatile int* abort) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_abort(bar, phase, kWaitLimitNs, abort));
  phase ^= 1;
  return ok;
}

// The epilogue works on blocks of 32 m x 32 n.  tcgen05.ld.16x256b gives a thread the elements
//   m = 16 (i / 16) + lane / 4 + 8 ((i / 2) % 2),   n = 8 ((i / 4) % 4) + 2 (lane % 4) + i % 2
// in register i: the fragments that stmatrix stores, as they are (rows of m) or transposed (rows
// of n), so a block goes through the warp's 2 KB stash with 4 + 4 shared-memory instructions and
// leaves as 16-byte stores in either orientation.  (One lane per m, 32 two-byte stores a block:
// the epilogue took 7600 cycles of a 256 x 256 tile and bounded the weight gradient.)
__device__ __forceinline__ int frag_m(int i, int lane) { return ((i >> 4) << 4) + (lane >> 2) + ((i >> 1 & 1) << 3); }
__device__ __forceinline__ int frag_n(int i, int lane) { return ((i >> 2 & 3) << 3) + ((lane & 3) << 1) + (i & 1); }

__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}

// 32 lanes (from the address's) x 32 columns; the values are there after tmem_wait_block.
__device__ __forceinline__ void tmem_ld_block(uint32_t taddr, float (&v)[32]) {
  tmem_ld_frag(taddr, v);
  tmem_ld_frag(taddr + (16u << 16), v + 16);
}

// Waits for this thread's tensor-memory loads; v passes through, so that no use of it moves above.
__device__ __forceinline__ void tmem_wait_block(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
  asm volatile(""
               : "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

// A row of the stash is 64 bytes; its 16-byte parts are permuted so that neither the fragments'
// stores (8 rows, one part) nor the 16-byte loads (2 rows, 4 parts) conflict.
__device__ __forceinline__ uint32_t stash_at(int row, int part) {
  return static_cast<uint32_t>(row * 64 + ((part ^ (row >> 1 & 3)) << 4));
}

template <bool TRANS>
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  if (TRANS)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
  else
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r0), "r"(r1), "r"(r2),
                 "r"(r3)
                 : "memory");
}

// Writes a block of 16-bit values, w[i / 2] holding elements i and i + 1.  ROWS_N: rows of n, element
// (m, n) at out[n * ld + m]; otherwise rows of m, at out[m * ld + n].  rows, width: how much of it exists.
template <bool ROWS_N>
__device__ __forceinline__ void store_block(const uint32_t (&w)[16], uint8_t* stash, uint16_t* out, long long ld, int rows,
                                            int width, bool vec) {
  const int lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(stash);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (ROWS_N)  // the four 8-element groups of m, rows n = 8 j ..
      stmatrix4<true>(base + stash_at(8 * j + (lane & 7), lane >> 3), w[2 * j], w[2 * j + 1], w[8 + 2 * j], w[9 + 2 * j]);
    else  // the four 8-element groups of n, rows m = 8 j ..
      stmatrix4<false>(base + stash_at(8 * j + (lane & 7), lane >> 3), w[(j >> 1) * 8 + (j & 1)],
                       w[(j >> 1) * 8 + 2 + (j & 1)], w[(j >> 1) * 8 + 4 + (j & 1)], w[(j >> 1) * 8 + 6 + (j & 1)]);
  }
  __syncwarp();
  if (vec && width == 32) {
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint4*>(stash + stash_at(8 * j + (lane >> 2), lane & 3));
    uint16_t* dst = out + (lane >> 2) * ld + (lane & 3) * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (8 * j + (lane >> 2) < rows) *reinterpret_cast<uint4*>(dst + 8 * j * ld) = x[j];
  } else if (lane < width) {
    for (int r = 0; r < rows; ++r)
      out[r * ld + lane] = *reinterpret_cast<const uint16_t*>(stash + stash_at(r, lane >> 3) + (lane & 7) * 2);
  }
  __syncwarp();
}

// The finished sums of one block, whose first m is mrow within the tile and first n is c0.  f: their factor (dense).
template <int MODE>
__device__ __forceinline__ void emit(const Args& a, const Unit& u, float f, float (&v)[32], int mrow, int c0,
                                     uint8_t* stash) {
  const int lane = threadIdx.x & 31;
  const int m = u.m0 + mrow;
  const int ncount = min(32, u.nn - c0);
  const int mcount = min(32, a.M - m);
  if (ncount <= 0 || mcount <= 0) return;
  const bool bf16 = a.out_type == kOutBf16;
  const int n = u.orow + c0;
  uint32_t w[16];
  if (MODE != kDense) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) w[i >> 1] = pack16(v[i], v[i + 1], bf16);
    uint16_t* out = static_cast<uint16_t*>(a.out) + (MODE == kRaggedN ? 0 : u.group * a.stride) + n * a.ld + m;
    store_block<true>(w, stash, out, a.ld, ncount, mcount, a.vec);
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] *= f;
  if (a.sym && m == n) {  // blocks and tiles start at multiples of 32
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (frag_m(i, lane) == frag_n(i, lane)) v[i] += a.diag;
  }
  if (a.out_type == kOutF32) {
    float* out = static_cast<float*>(a.out) + u.group * a.stride + n * a.ld + m;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int mi = frag_m(i, lane), ni = frag_n(i, lane);
      if (mi < mcount && ni < ncount) out[ni * a.ld + mi] = v[i];
    }
    return;
  }
  uint16_t* out = static_cast<uint16_t*>(a.out) + u.group * a.stride;
  const int np = a.out_type == kOutSlices ? a.planes_out : 1;
  for (int p = 0; p < np; ++p, out += a.plane) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      w[i >> 1] = pack16(v[i], v[i + 1], bf16);
      if (np > 1) {  // what the slice leaves
        const __half2 h = *reinterpret_cast<const __half2*>(&w[i >> 1]);
        v[i] -= __low2float(h);
        v[i + 1] -= __high2float(h);
      }
    }
    if (!a.sym) {
      store_block<true>(w, stash, out + n * a.ld + m, a.ld, ncount, mcount, a.vec);
    } else if (n < m) {  // below the diagonal: both copies
      store_block<true>(w, stash, out + n * a.ld + m, a.ld, ncount, mcount, a.vec);
      store_block<false>(w, stash, out + m * a.ld + n, a.ld, mcount, ncount, a.vec);
    } else if (n == m) {  // on it: the block is its own mirror
      store_block<true>(w, stash, out + n * a.ld + m, a.ld, ncount, mcount, a.vec);
    }
  }
}

// One block of a split sum's part: 16 bytes a thread and instruction.
__device__ __forceinline__ void put_part(float* part, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    __stcg(reinterpret_cast<float4*>(part + i * 32), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
}
__device__ __forceinline__ void add_part(const float* part, float (&v)[32]) {
  float4 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __ldcg(reinterpret_cast<const float4*>(part + i * 128));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[4 * i] += x[i].x;
    v[4 * i + 1] += x[i].y;
    v[4 * i + 2] += x[i].z;
    v[4 * i + 3] += x[i].w;
  }
}

__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int MODE, bool A_MN, bool B_MN, int PLANES>
__global__ void __launch_bounds__(THREADS, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmB128, const __grid_constant__ Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * A_STAGE;
  uint8_t* stash = smem + STAGES * STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stash + STASH);
  uint64_t* full = bars;                   // [STAGES] TMA (both CTAs) -> MMA  (used in the leader)
  uint64_t* empty = bars + STAGES;         // [STAGES] MMA -> TMA              (both CTAs)
  uint64_t* accfull = bars + 2 * STAGES;   // [2]      MMA -> epilogue         (both CTAs)
  uint64_t* accempty = accfull + 2;        // [2]      epilogues (both) -> MMA (used in the leader)
  uint64_t* drain = accempty + 2;          // [1]      all MMAs of the pair done (both CTAs)
  uint64_t* epibar = drain + 1;            // [1]      epilogue warps rendezvous (per CTA)
  uint64_t* exitbar = epibar + 1;          // [1]      the peer has finished (per CTA)
  uint64_t* proddone = exitbar + 1;        // [1]      both producers have stopped (used in the leader)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(proddone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued_by = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);  // [2] (leader)
  volatile uint32_t* arrived = issued_by + 2;
  int* tab_off = reinterpret_cast<int*>(stash + STASH + 256);  // grouped modes only
  int* tab_prefix = tab_off + MAX_GROUPS + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(epibar, EPI_WARPS);
    mbar_init(exitbar, 1);
    mbar_init(proddone, 2);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (MODE == kRaggedN) tma_prefetch_desc(&tmB128);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  // The next launch may set itself up meanwhile.  Dense launches come in chains: what touches the
  // matrices waits for the launch before (the producer's first load, the epilogue's first store).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (MODE != kDense) {
    wait_for_previous();
    for (int i = threadIdx.x; i <= a.groups; i += THREADS) tab_off[i] = a.offsets[i];
    __syncthreads();
    if (warp == 0) {
      // Offsets are clamped to [0, rows] and to their predecessors, so that no access leaves the
      // matrices whatever they hold; offsets that needed it are reported.
      const int tiles_m = ceil_div(a.M, BM);
      int floor_off = 0, sum = 0;
      bool bad = false;
      for (int b = 0; b <= a.groups; b += 32) {
        const int i = b + lane;
        int v = i <= a.groups ? tab_off[i] : 0;
        const int given = v;
        v = max(0, min(v, a.rows));
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
          if (lane >= d) v = max(v, o);
        }
        v = max(v, floor_off);
        bad |= i <= a.groups && v != given;
        int prev = __shfl_up_sync(0xFFFFFFFFu, v, 1);
        if (lane == 0) prev = floor_off;
        floor_off = __shfl_sync(0xFFFFFFFFu, v, 31);
        int t = (i >= 1 && i <= a.groups) ? ceil_div(v - prev, a.bn) * tiles_m : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xFFFFFFFFu, t, d);
          if (lane >= d) t += o;
        }
        if (i <= a.groups) {
          tab_off[i] = v;
          tab_prefix[i] = sum + t;
        }
        sum += __shfl_sync(0xFFFFFFFFu, t, 31);
      }
      if (__any_sync(0xFFFFFFFFu, bad) && lane == 0 && blockIdx.x == 0) atomicExch(a.status, OZ_EINVAL);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  Schedule sched;
  sched.off = tab_off;
  sched.prefix = tab_prefix;
  sched.tiles_m = ceil_div(a.M, BM);
  sched.tiles_n = MODE == kRaggedN ? 0 : ceil_div(a.N, a.bn);
  sched.first = static_cast<int>(blockIdx.x >> 1);
  sched.step = static_cast<int>(gridDim.x >> 1);
  if (MODE == kDense) {
    sched.tiles = a.tiles;
    sched.nsplit = a.nsplit;
  } else if (MODE == kRaggedN) {
    sched.tiles = tab_prefix[a.groups];
    sched.nsplit = split_for(sched.tiles, ceil_div(a.K, BK), sched.step, a.max_split_units, 4);
  } else {
    sched.tiles = a.groups * sched.tiles_m * sched.tiles_n;
    sched.nsplit = split_for(sched.tiles, ceil_div(tab_off[a.groups] - tab_off[0], BK * a.groups), sched.step,
                             a.max_split_units, 4);
  }
  sched.total = sched.tiles * sched.nsplit;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      for (int idx = sched.first; idx < sched.total && !*abort_flag; idx += sched.step) {
        Unit u;
        unit_at<MODE, B_MN>(a, sched, idx, u);
        const int rowA = u.m0 + static_cast<int>(rank) * HALF_M;
        const int half_n = u.nmma >> 1;
        const int rowB = u.n0 + static_cast<int>(rank) * half_n;
        // Few TMA instructions a stage: their issue, not the bytes, is what a stage waits for first.
        const bool wide_b = MODE == kRaggedN && half_n > 64;
        const int box_b = wide_b ? HALF_N : a.box_rows;
        const int boxes = B_MN ? (a.b_4d ? 1 : half_n / 64) : ceil_div(half_n, box_b);
        const CUtensorMap* mapB = wide_b ? &tmB128 : &tmB;
        const uint32_t box_bytes = B_MN ? (a.b_4d ? a.bn / 128 : 1) * MN_BLOCK : box_b * BK * 2;
        const uint32_t bytes = A_STAGE + boxes * box_bytes;
        if (MODE == kDense && idx == sched.first) wait_for_previous();
        for (int kb = u.kb0; kb < u.kb1 && !*abort_flag; ++kb) {
#pragma unroll
          for (int p = 0; p < PLANES; ++p) {
            if (!mbar_wait_or_abort(&empty[stage], phase ^ 1, kWaitLimitNs, abort_flag)) {
              if (!*abort_flag) stop_pair(abort_flag, a.status);
              break;
            }
            const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
            mbar_arrive_expect_tx_cluster(bar, bytes);
            const int k = u.k0 + kb * BK;
            // last coordinate: matrix (slice) of the batch, or the group's first row
            const int zA = MODE == kRaggedK ? u.kstart : u.group * PLANES + p;
            const int zB = MODE == kDense ? u.group * PLANES + p : (MODE == kRaggedK ? u.kstart : 0);
            uint8_t* dA = sA + stage * A_STAGE;
            uint8_t* dB = sB + stage * B_STAGE;
            if (!A_MN) {
              tma_load_3d_pair(dA, &tmA, bar, k, rowA, zA);
            } else if (a.a_4d) {
              tma_load_4d_pair(dA, &tmA, bar, 0, k, rowA / 64, zA);
            } else {
              tma_load_3d_pair(dA, &tmA, bar, rowA, k, zA);
              tma_load_3d_pair(dA + MN_BLOCK, &tmA, bar, rowA + 64, k, zA);
            }
            if (!B_MN) {
              tma_load_3d_pair(dB, mapB, bar, k, rowB, zB);
              for (int b = 1; b < boxes; ++b) tma_load_3d_pair(dB + b * box_bytes, mapB, bar, k, rowB + box_b * b, zB);
            } else if (a.b_4d) {  // a last, narrower tile loads the full box: B_STAGE has room for it
              tma_load_4d_pair(dB, &tmB, bar, 0, k, rowB / 64, zB);
            } else {
              for (int b = 0; b < boxes; ++b) tma_load_3d_pair(dB + b * MN_BLOCK, mapB, bar, rowB + 64 * b, k, zB);
            }
            ++issued;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
      // Every issued copy must have landed before the pair may exit (see the residue GEMM).
      st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(&issued_by[rank])), 0),
                            static_cast<uint32_t>(issued));
      mbar_arrive_release_cluster(mapa_shared(smem_u32(proddone), 0));
      if (!*abort_flag) {
        for (int i = 0; i < STAGES && i < issued; ++i) {
          if (--stage < 0) {
            stage = STAGES - 1;
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
    if (lane == 0 && rank == 0) {
      // ------------------------------------------------------------ MMA issuer (leader only)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t g = 0;
      uint32_t consumed = 0;
      bool ok = true;
      // Low words of stage 0's descriptors; a stage or a k step only adds to the address field.
      constexpr uint32_t A_STEP = (A_MN ? UMMA_K * 128 : UMMA_K * 2) >> 4, B_STEP = (B_MN ? UMMA_K * 128 : UMMA_K * 2) >> 4;
      const uint32_t a_desc = desc_low<A_MN>(smem_u32(sA)), b_desc = desc_low<B_MN>(smem_u32(sB));
      for (int idx = sched.first; idx < sched.total && ok && !*abort_flag; idx += sched.step) {
        Unit u;
        unit_at<MODE, B_MN>(a, sched, idx, u);
        const uint32_t idesc = a.idesc | (static_cast<uint32_t>(u.nmma >> 3) << 17);
        int left = u.kb1 - u.kb0;
        if (left == 0) continue;
        uint32_t in_chunk = 0, d_tmem = 0;
        if (PLANES == 1) {  // the whole part in one accumulator
          if (!mbar_wait_or_abort(&accempty[g & 1], ((g >> 1) & 1) ^ 1, kWaitLimitNs, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          d_tmem = tmem_base + (g & 1) * BN;
        }
        for (; left > 0; --left) {
#pragma unroll
          for (int p = 0; p < PLANES; ++p) {
            if (!mbar_wait_or_abort(&full[stage + p], phase, kWaitLimitNs, abort_flag)) {
              ok = false;
              break;
            }
            ++consumed;
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t ad = a_desc + stage * (A_STAGE >> 4), bd = b_desc + stage * (B_STAGE >> 4);
#pragma unroll
          for (int kk = 0; kk < KSTEPS; ++kk) {
            if (PLANES == 1) {
              umma_pair(d_tmem, ad + kk * A_STEP, bd + kk * B_STEP, idesc, kk > 0 ? 1u : in_chunk);
              in_chunk = 1;
            } else {
              if (in_chunk == 0) {  // a new sum: the next accumulator
                if (!mbar_wait_or_abort(&accempty[g & 1], ((g >> 1) & 1) ^ 1, kWaitLimitNs, abort_flag)) {
                  ok = false;
                  break;
                }
                tc_fence_after();
                d_tmem = tmem_base + (g & 1) * BN;
              }
              umma_pair(d_tmem, ad + kk * A_STEP, bd + kk * B_STEP, idesc, in_chunk);                              // h h'
              umma_pair(d_tmem + CROSS, ad + kk * A_STEP, bd + (B_STAGE >> 4) + kk * B_STEP, idesc, in_chunk);     // h l'
              umma_pair(d_tmem + CROSS, ad + (A_STAGE >> 4) + kk * A_STEP, bd + kk * B_STEP, idesc, 1u);           // l h'
              if (++in_chunk == static_cast<uint32_t>(a.chunk) || (left == 1 && kk + 1 == KSTEPS)) {
                umma_commit_pair(&accfull[g & 1], 0x3);
                in_chunk = 0;
                ++g;
              }
            }
          }
          if (!ok) break;
#pragma unroll
          for (int p = 0; p < PLANES; ++p) umma_commit_pair(&empty[stage + p], 0x3);
          stage += PLANES;
          if (stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (PLANES == 1) {
          umma_commit_pair(&accfull[g & 1], 0x3);
          ++g;
        }
      }
      if (!ok && !*abort_flag) stop_pair(abort_flag, a.status);
      // Account for every copy before the pair may exit (see the residue GEMM).
      if (mbar_wait_acquire_cluster(proddone, 0)) {
        const uint32_t n0 = issued_by[0], n1 = issued_by[1];
        const uint32_t top = n0 > n1 ? n0 : n1;
        for (uint32_t q = consumed; q < top && q < consumed + STAGES; ++q) {
          const int st = static_cast<int>(q % STAGES);
          if (q >= n0) mbar_arrive(&full[st]);
          if (q >= n1) mbar_arrive(&full[st]);
          if (!mbar_wait(&full[st], (q / STAGES) & 1)) {
            stop_pair(abort_flag, a.status);
            break;
          }
        }
      } else {
        stop_pair(abort_flag, a.status);
      }
      umma_commit_pair(drain, 0x3);
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2-9, both CTAs)
    // A warp drains its 32 lanes and every second block of 32 columns.
    const int quad = warp & 3;
    const int half = (warp - 2) >> 2;
    const int etid = threadIdx.x - 64;
    const int mrow = static_cast<int>(rank) * HALF_M + quad * 32;
    uint8_t* my_stash = stash + (warp - 2) * WARP_STASH;
    uint32_t g = 0, eph = 0;
    bool ok = true;
    if (MODE == kRaggedN) {  // rows that belong to no group are zero
      const int lo = tab_off[0], hi = tab_off[a.groups];
      const int loose = lo + a.rows - hi;
      for (int i = static_cast<int>(blockIdx.x) * EPI_WARPS + warp - 2; i < loose; i += gridDim.x * EPI_WARPS) {
        uint16_t* row = static_cast<uint16_t*>(a.out) + static_cast<long long>(i < lo ? i : hi + i - lo) * a.ld;
        for (int c = lane; c < a.M; c += 32) row[c] = 0;
      }
    }
    for (int idx = sched.first; idx < sched.total && ok; idx += sched.step) {
      Unit u;
      unit_at<MODE, B_MN>(a, sched, idx, u);
      const int nblocks = ceil_div(u.nn, 32);  // this warp: blocks half, half + 2, ...
      if (MODE == kDense && idx == sched.first) wait_for_previous();
      const float f = MODE == kDense && a.scale ? a.alpha * a.scale[u.group * a.scale_stride] : a.alpha;
      const bool split = u.nsplit > 1;
      float* part = nullptr;
      const long long part_unit = 2ll * a.part_cols * HALF_M;
      if (split)
        part = a.part + (static_cast<long long>(u.tile) * u.nsplit + u.split) * part_unit +
               static_cast<long long>(rank) * a.part_cols * HALF_M + quad * 1024 + lane * 4;  // block cb: + cb * 4096
      float run[PLANES == 2 ? 2 : 1][32];
      const int nchunks = ceil_div((u.kb1 - u.kb0) * KSTEPS, a.chunk);
      for (int ch = 0; ch < nchunks; ++ch, ++g) {
        const uint32_t acc = g & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&accfull[acc], (g >> 1) & 1, a.epi_wait_ns, abort_flag))) {
          ok = false;
          if (lane == 0 && !*abort_flag) stop_pair(abort_flag, a.status);
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * BN;
        if (PLANES == 2) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int cb = 2 * j + half;
            if (cb < nblocks) {
              float v[32], w[32];
              tmem_ld_block(taddr + cb * 32, v);
              tmem_ld_block(taddr + CROSS + cb * 32, w);
              tmem_wait_block(v);
              tmem_wait_block(w);
#pragma unroll
              for (int i = 0; i < 32; ++i) run[j][i] = ch ? run[j][i] + (v[i] + w[i]) : v[i] + w[i];
            }
          }
        } else {
#pragma unroll 1
          for (int cb = half; cb < nblocks; cb += 2) {
            float v[32];
            tmem_ld_block(taddr + cb * 32, v);
            tmem_wait_block(v);
            if (cb + 2 >= nblocks) {  // the last block is in registers: hand the accumulator back
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&accempty[acc]), 0));
            }
            if (split)
              put_part(part + cb * 4096, v);
            else
              emit<MODE>(a, u, f, v, mrow, cb * 32, my_stash);
          }
        }
        if (PLANES == 2 || half >= nblocks) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&accempty[acc]), 0));
        }
      }
      if (!ok) break;
      if (PLANES == 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int cb = 2 * j + half;
          if (cb < nblocks) {
            if (split)
              put_part(part + cb * 4096, run[j]);
            else
              emit<MODE>(a, u, f, run[j], mrow, cb * 32, my_stash);
          }
        }
      } else if (nchunks == 0) {  // an empty sum (a group without rows, or with few for this many parts)
#pragma unroll 1
        for (int cb = half; cb < nblocks; cb += 2) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
          if (split)
            put_part(part + cb * 4096, v);
          else
            emit<MODE>(a, u, f, v, mrow, cb * 32, my_stash);
        }
      }
      if (split) {
        // This CTA's part is written; the last of the tile's parts to arrive adds them all.
        __threadfence();
        if (!warps_meet(epibar, eph, abort_flag)) ok = false;
        if (ok && etid == 0) *arrived = atomicAdd(&a.counters[u.tile * 2 + rank], 1u);
        if (ok && !warps_meet(epibar, eph, abort_flag)) ok = false;
        if (!ok) {
          if (lane == 0 && !*abort_flag) stop_pair(abort_flag, a.status);
          break;
        }
        const bool last = *arrived == static_cast<uint32_t>(u.nsplit - 1);
        if (!warps_meet(epibar, eph, abort_flag)) {  // everyone has read `arrived`
          ok = false;
          if (lane == 0 && !*abort_flag) stop_pair(abort_flag, a.status);
          break;
        }
        if (last) {
          __threadfence();
          if (etid == 0) a.counters[u.tile * 2 + rank] = 0;  // as it was found: a later launch may use it
          const float* p0 = part - u.split * part_unit;
#pragma unroll 1
          for (int cb = half; cb < nblocks; cb += 2) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            for (int q = 0; q < u.nsplit; ++q) add_part(p0 + q * part_unit + cb * 4096, v);
            emit<MODE>(a, u, f, v, mrow, cb * 32, my_stash);
          }
        }
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
// An operand's tensor map: 16-bit elements, 128-byte swizzle, zeros out of bounds.
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline bool encode(CUtensorMap* map, const void* base, bool bf16, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
  const EncodeTiled fn = reinterpret_cast<EncodeTiled>(tensor_map_encoder());
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn && fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [d2][d1][d0] with strides s1, s2 in bytes (multiples of 16); box {64, box_rows, 1}.
inline bool make_map(CUtensorMap* map, const void* base, bool bf16, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1,
                     uint64_t s2, int box_rows) {
  const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1, s2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  return encode(map, base, bf16, 3, dims, strides, box);
}

// The same matrix for an MN-major operand: when d0 is a multiple of 64, a 4-D map
// [d2][d0 / 64][d1][64] whose box is 64 rows by `blocks` blocks of 64 contiguous elements; otherwise
// (a last partial block in such a map would reach past the end of the last row) make_map's, one
// block a box.  *is_4d says which: a load's rank has to be its map's.
inline bool make_mn_map(CUtensorMap* map, int* is_4d, int blocks, const void* base, bool bf16, uint64_t d0, uint64_t d1,
                        uint64_t d2, uint64_t s1, uint64_t s2) {
  *is_4d = d0 % 64 == 0;
  if (!*is_4d) return make_map(map, base, bf16, d0, d1, d2, s1, s2, BK);
  const cuuint64_t dims[4] = {64, d1, d0 / 64, d2}, strides[3] = {s1, 128, s2};
  const cuuint32_t box[4] = {64, BK, static_cast<cuuint32_t>(blocks), 1};
  return encode(map, base, bf16, 4, dims, strides, box);
}

struct Device {
  int id, pairs;  // CTA pairs that fit at once
  int* status;
};

inline int current_device(Device* d) {
  int sms = 0;
  if (cudaGetDevice(&d->id) != cudaSuccess) return OZ_ECUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d->id) != cudaSuccess) return OZ_ECUDA;
  d->pairs = sms / 2;
  d->status = device_status_ptr();
  return d->status ? OZ_OK : OZ_ECUDA;
}

// Launches the product on `pairs` CTA pairs.  dependent: the launch may begin while the one
// before it on the stream ends (the kernel waits for it before it reads anything).
template <int MODE, bool A_MN, bool B_MN, int PLANES>
int launch(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmB128, Args a, const Device& d, int pairs,
           bool dependent, cudaStream_t stream) {
  const int dev = d.id;
  a.status = d.status;
  auto kernel = product_kernel<MODE, A_MN, B_MN, PLANES>;
  const size_t smem = MODE == kDense ? SMEM_DENSE : SMEM_GROUPED;
  a.epi_wait_ns = epilogue_wait_ns();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
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
  cfg.numAttrs = dependent ? 2 : 1;
  // The shared-memory limit is the function's, in this context: set on the first launch, and again
  // should a launch be refused (a new context after a device reset).
  static std::atomic<bool> ready[64] = {};
  for (int attempt = 0; attempt < 2; ++attempt) {
    if (dev >= 64 || attempt || !ready[dev].load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return OZ_ECUDA;
      if (dev < 64) ready[dev].store(true, std::memory_order_release);
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tmA, tmB, tmB128, a);
    if (e == cudaSuccess) return OZ_OK;
    cudaGetLastError();
    if (e != cudaErrorInvalidValue) break;
  }
  return OZ_ECUDA;
}

}  // namespace prod
}  // namespace oz
