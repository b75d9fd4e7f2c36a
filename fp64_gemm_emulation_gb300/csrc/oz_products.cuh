// oz_products.cuh -- the tensor-core kernel behind the grouped expert products and the
// Newton-Schulz iteration: many 16-bit matrix products of different extents in one launch.
//
// Every product is D[m, n] = sum_k A[m, k] B[n, k] with FP32 sums, where m runs along the
// output's contiguous dimension and n over its rows.  That orientation is chosen for all
// operators: a ragged number of output rows (the tokens of an expert) is then the MMA's N, which
// takes any multiple of 32, so a short expert does not pay for a full tile.  Either operand may
// be K-contiguous ("K-major") or m/n-contiguous ("MN-major"); the tensor core reads both from the
// 128-byte-swizzled tiles that TMA writes, so nothing is ever transposed in memory.
//
// Kernel shape: clusters of two CTAs (cta_group::2), persistent over the units (tile, part of k)
// that a walker deals out (GroupedWalk in oz_grouped.cu, ChainWalk in oz_newton.cu).
//   warp 0: TMA producer   warp 1: TMEM owner + MMA issuer (leader)   then Walk::kEpiWarps: epilogue
//   a last one, where units depend on one another: the scout, which looks whether the next ones may start
//   6 stages of 32 KB (128 x 64 of A and up to 128 x 64 of B in each CTA), with two slices 4 of 52 KB
//   two 256-column FP32 accumulators in tensor memory, so that a tile's epilogue runs under the next one's
//   MMAs (two slices: three of 160 columns; with two of 192, each chunk's hand-over to the epilogue and
//   back, about 840 cycles beside its 930 of work, left the tensor cores idle for a fifth of the time)
// What bounds it: one thread issues every MMA and one every copy, so both loops are kept to a few
// instructions (at 8192^3, descriptors rebuilt for each MMA: 981 TFLOP/s; two descriptor words and
// one add: 1524; one TMA copy for each operand and stage instead of up to six: 1780).
//
// Split k: the tiles that do not fill a last wave of CTA pairs are cut into parts along k
// (split_cost, or plan_product in oz_newton.cu).  Each part's FP32 sums go to the workspace, and the CTA that arrives last (an
// atomic counter for each tile and CTA) adds the parts in their order, so results do not depend
// on timing and nobody waits.
// Two slices (PLANES == 2): operands are h + l with h, l in FP16.  A chunk (a k-block or one MMA
// step) sums h l' + l h' and then h h' into one accumulator; the tensor core truncates as it accumulates,
// so the sums leave it after every chunk and go on in FP32 registers (round to nearest).
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
constexpr int BN2 = 160;                      // widest tile with two slices: three accumulators fit tensor memory
constexpr int BK = 64;
constexpr int UMMA_K = 16;
constexpr int KSTEPS = BK / UMMA_K;
constexpr uint32_t A_PLANE = HALF_M * BK * 2;  // one slice of a stage's A
constexpr uint32_t MN_BLOCK = 64 * BK * 2;    // 64 contiguous m (or n) x 64 k
constexpr int EPI_FIRST = 2;                  // the first epilogue warp
constexpr uint32_t TMEM_COLS = 512;

// The ring of stages: 64 k of A and B, both slices of them with two slices.
template <int PLANES>
struct Ring {
  static constexpr int STAGES = PLANES == 2 ? 4 : 6;
  static constexpr uint32_t A_STAGE = PLANES * A_PLANE;
  static constexpr uint32_t B_STAGE = PLANES == 2 ? 2 * (BN2 / 2) * BK * 2 : HALF_N * BK * 2;
  static constexpr uint32_t BYTES = STAGES * (A_STAGE + B_STAGE);
  // An epilogue warp's stash: a 32 x 32 block of 16 bits (two slices: no room, store_regs; the warp's unit).
  static constexpr uint32_t WARP_STASH = PLANES == 2 ? 256 : 32 * 64;
};

constexpr long long PART_BLOCK = 32 * HALF_M;  // floats of 32 columns of one CTA's part

enum OutType { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2, kOutSlices = 3 };

constexpr int kMaxExtent = INT32_MAX - 1024;  // a dimension rounded up to a tile stays an int

// a >= 0, b > 0; a + b may pass INT32_MAX.
__host__ __device__ inline int ceil_div(int a, int b) {
  return static_cast<int>((static_cast<unsigned>(a) + static_cast<unsigned>(b) - 1) / static_cast<unsigned>(b));
}

// One unit of work.  A role uses the fields it needs; the rest is never computed for it.
struct Unit {
  int m0, n0, nn, nmma;     // the tile: first m, first row of B, its rows, the MMA's N
  int k0, kb0, kb1;         // k coordinate of k-block 0; the part's k-blocks
  int chunk;                // two slices: MMA steps summed on the tensor core (1, or KSTEPS: a k-block)
  const CUtensorMap *mapA, *mapB;
  bool a_mn, b_mn;          // MN-major operands ...
  bool a_4d, b_4d;          // ... with a 4-D map, whose box holds the CTA's whole tile
  int box_b, boxes;         // B copies: rows of a box (K-major), boxes of a stage
  uint32_t box_bytes;       // all slices'
  uint32_t b_plane;         // distance of B's slices in a stage
  int zA, zB;               // last coordinate of A and B (matrix of the batch, or first row)
  uint32_t idesc;
  int m_extent;             // the output's m
  void* out;
  long long ld, plane;      // output row stride; distance of the low slices
  int orow;                 // output row of the tile's first n
  int out_type, planes_out;
  bool vec, sym;            // 16-byte stores are allowed; a symmetric product, mirrored
  float f, diag;            // v = f v, + diag on the diagonal (sym)
  int split, nsplit;
  float* part;              // the tile's parts: [nsplit][2 CTAs][part_cols][128]
  int part_cols;
  unsigned int* arrivals;   // [2 CTAs]
};
static_assert(sizeof(Unit) <= Ring<2>::WARP_STASH, "the stash holds a unit");

// Time, in k-blocks, of a last, partial wave of `tiles` tiles cut into s parts each: the waves of the
// parts and the joining (each CTA writes its part and the last one reads all: about 4 k-blocks
// of time for 256 columns, and 2 for the rendezvous).  kSplitFixed: a unit's start and drain.
constexpr int kSplitFixed = 4, kMaxSplit = 16;
__host__ __device__ inline int split_cost(int tiles, int nkb, int pairs, int max_parts, int cols, int s) {
  if (s > 1 && (s > nkb || tiles * s > max_parts)) return 1 << 30;
  return ceil_div(tiles * s, pairs) * (ceil_div(nkb, s) + kSplitFixed) + (s > 1 ? 2 + 4 * (1 + s) * cols / 256 : 0);
}

// Shared-memory descriptors, low word: address / 16 and the leading byte offset.  K-major tiles:
// rows of 64 k (128 bytes, 128-byte swizzle), 8 rows are 1024 bytes, no leading offset.
// MN-major tiles: blocks of 64 contiguous m (128 bytes a k row, 128-byte swizzle), 8 k rows are
// 1024 bytes, the next 64 m are MN_BLOCK bytes on.  The high word is the same for both.
__device__ __forceinline__ uint32_t desc_low(uint32_t smem_addr, bool mn) {
  return ((smem_addr >> 4) & 0x3FFFu) | ((mn ? MN_BLOCK >> 4 : 1u) << 16);
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

// Neighbouring values as pairs of 16-bit elements, the first in the low half.
__device__ __forceinline__ void pack_block(const float (&v)[32], uint32_t (&w)[16], bool bf16) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
}

__device__ __forceinline__ void stop_pair(volatile int* abort_flag, int* status) {
  *abort_flag = 1;
  st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), cluster_ctarank() ^ 1u), 1u);
  atomicExch(status, OZ_ETIMEOUT);
}

__device__ __forceinline__ uint32_t add_shared_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t old;
  asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(smem_u32(p)), "r"(v) : "memory");
  return old;
}

// Waits until *count >= want.
__device__ __forceinline__ bool wait_for_count(const uint32_t* count, uint32_t want, const volatile int* abort) {
  auto reached = [&]() {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(count)) : "memory");
    return v >= want;
  };
  if (reached()) return true;
  const uint64_t t0 = globaltimer_ns();
  for (int i = 1; !reached(); ++i) {
    if (*abort || ((i & 255) == 0 && globaltimer_ns() - t0 > kWaitLimitNs)) return false;
  }
  return true;
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
// of n), so a block goes through the warp's stash with 4 + 4 shared-memory instructions and
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

// Where a thread's stores of a tile go, set up once for a unit: a block is then little more than its
// conversions and its 12 shared and global accesses.  (With the addresses and the cases of each
// block worked out in place it was 130 instructions at 8 cycles each, and two warps to a
// scheduler cannot hide that: 4260 cycles a tile in the weight gradient.)
struct Target {
  uint32_t put;         // stmatrix's row, and the 16 bytes read back, in the warp's stash
  const uint8_t* get;
  uint16_t* by_n;       // this lane's 16 bytes of row n = lane / 4 of the tile's first block
  long long step;       // 8 rows
  int m, mcount;        // first m of the warp's lanes, how many exist
  bool fast;            // 16-bit output, whole lanes, 16-byte stores
};

__device__ __forceinline__ Target target_of(const Unit& u, int mrow, uint8_t* stash) {
  const int lane = threadIdx.x & 31;
  Target t;
  t.put = smem_u32(stash) + stash_at(lane & 7, lane >> 3);
  t.get = stash + stash_at(lane >> 2, lane & 3);
  t.m = u.m0 + mrow;
  t.mcount = min(32, u.m_extent - t.m);
  t.step = 8 * u.ld;
  t.by_n = static_cast<uint16_t*>(u.out) + (u.orow + (lane >> 2)) * u.ld + t.m + (lane & 3) * 8;
  t.fast = u.vec && t.mcount == 32 && u.out_type != kOutF32;
  return t;
}

// A block of 16-bit values, w[i / 2] holding elements i and i + 1, into the warp's stash (8 rows are
// 512 bytes, which leave the permutation as it is).  ROWS_N: rows of n, otherwise rows of m.
template <bool ROWS_N>
__device__ __forceinline__ void stash_block(const uint32_t (&w)[16], const Target& t) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (ROWS_N)  // the four 8-element groups of m, rows n = 8 j ..
      stmatrix4<true>(t.put + 512 * j, w[2 * j], w[2 * j + 1], w[8 + 2 * j], w[9 + 2 * j]);
    else  // the four 8-element groups of n, rows m = 8 j ..
      stmatrix4<false>(t.put + 512 * j, w[(j >> 1) * 8 + (j & 1)], w[(j >> 1) * 8 + 2 + (j & 1)],
                       w[(j >> 1) * 8 + 4 + (j & 1)], w[(j >> 1) * 8 + 6 + (j & 1)]);
  }
  __syncwarp();
}

// A whole block; dst: this lane's 16 bytes of row lane / 4.
template <bool ROWS_N>
__device__ __forceinline__ void store_whole(const uint32_t (&w)[16], const Target& t, uint16_t* dst) {
  stash_block<ROWS_N>(w, t);
  uint4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(t.get + 512 * i);
#pragma unroll
  for (int i = 0; i < 4; ++i, dst += t.step) *reinterpret_cast<uint4*>(dst) = x[i];
  __syncwarp();
}

// The 4 x 4 words of four neighbouring lanes, transposed: lane q gets word q of each.
__device__ __forceinline__ void transpose4(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
  uint32_t x = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1), y = __shfl_xor_sync(0xFFFFFFFFu, odd ? c : d, 1);
  if (odd) a = x, c = y; else b = x, d = y;
  x = __shfl_xor_sync(0xFFFFFFFFu, high ? a : c, 2);
  y = __shfl_xor_sync(0xFFFFFFFFu, high ? b : d, 2);
  if (high) a = x, b = y; else c = x, d = y;
}

// A block without a stash (two slices have no shared memory left): each 8 x 8 of the fragments
// transposed in registers where rows of n are wanted, and 16 bytes gathered in each lane.  All
// of it comes before the first store, so that the latencies of the 32 exchanges overlap.
// out: the block's first element; rows of `width` elements.  w is used up.
template <bool ROWS_N>
__device__ __forceinline__ void store_regs(uint32_t (&w)[16], uint16_t* out, long long ld, int rows, int width, bool vec) {
  const int lane = threadIdx.x & 31, q = 8 * (lane & 3);
  if (ROWS_N) {
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(w[i]));
  }
  // Rows 8 j + lane / 4: the groups of 8 m, or of 8 n.
#define OZ_GROUP(j, e) w[ROWS_N ? 8 * ((e) >> 1) + 2 * (j) + ((e) & 1) : 8 * ((j) >> 1) + ((j) & 1) + 2 * (e)]
#pragma unroll
  for (int j = 0; j < 4; ++j) transpose4(OZ_GROUP(j, 0), OZ_GROUP(j, 1), OZ_GROUP(j, 2), OZ_GROUP(j, 3));
  uint16_t* dst = out + (lane >> 2) * ld + q;
  if (vec && rows >= 32 && width >= 32) {
#pragma unroll
    for (int j = 0; j < 4; ++j, dst += 8 * ld)
      *reinterpret_cast<uint4*>(dst) = make_uint4(OZ_GROUP(j, 0), OZ_GROUP(j, 1), OZ_GROUP(j, 2), OZ_GROUP(j, 3));
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j, dst += 8 * ld) {
    if (8 * j + (lane >> 2) < rows) {
      if (vec && q + 8 <= width) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(OZ_GROUP(j, 0), OZ_GROUP(j, 1), OZ_GROUP(j, 2), OZ_GROUP(j, 3));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (q + e < width) dst[e] = static_cast<uint16_t>(OZ_GROUP(j, e >> 1) >> (16 * (e & 1)));
      }
    }
  }
#undef OZ_GROUP
}

// A block of which only `rows` rows of `width` elements exist, or whose stores cannot be wide: a row at a
// time, one element a lane.  out: the block's first element.
template <bool ROWS_N>
__device__ __forceinline__ void store_part(const uint32_t (&w)[16], const Target& t, const uint8_t* stash, uint16_t* out,
                                           long long ld, int rows, int width) {
  const int lane = threadIdx.x & 31;
  stash_block<ROWS_N>(w, t);
  if (lane < width) {
    for (int r = 0; r < rows; ++r)
      out[r * ld + lane] = *reinterpret_cast<const uint16_t*>(stash + stash_at(r, lane >> 3) + (lane & 7) * 2);
  }
  __syncwarp();
}

// The finished sums of block cb (32 columns) of a tile.  SCALED: the Newton-Schulz products; STASH: one slice.
template <bool SCALED, bool STASH>
__device__ __forceinline__ void emit(const Unit& u, const Target& t, float (&v)[32], int cb, uint8_t* stash) {
  const int lane = threadIdx.x & 31;
  const int ncount = min(32, u.nn - 32 * cb);
  uint32_t w[16];
  if (!SCALED) {
    pack_block(v, w, u.out_type == kOutBf16);
    if (t.fast && ncount == 32)
      store_whole<true>(w, t, t.by_n + 4 * cb * t.step);
    else if (t.mcount > 0)
      store_part<true>(w, t, stash, static_cast<uint16_t*>(u.out) + (u.orow + 32 * cb) * u.ld + t.m, u.ld, ncount,
                             t.mcount);
  } else {
    const int n = u.orow + 32 * cb;
    if (t.mcount <= 0 || (u.sym && n > t.m)) return;  // above the diagonal: some block's mirror
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= u.f;
    if (u.sym && t.m == n) {  // blocks and tiles start at multiples of 32
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (frag_m(i, lane) == frag_n(i, lane)) v[i] += u.diag;
    }
    if (u.out_type == kOutF32) {
      float* out = static_cast<float*>(u.out) + n * u.ld + t.m;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int mi = frag_m(i, lane), ni = frag_n(i, lane);
        if (mi < t.mcount && ni < ncount) out[ni * u.ld + mi] = v[i];
      }
      return;
    }
    const bool whole = t.fast && ncount == 32;
    const bool mirror = u.sym && n < t.m;  // a block on the diagonal is its own mirror
    auto store = [&](uint32_t (&x)[16], long long plane) {
      uint16_t* out = static_cast<uint16_t*>(u.out) + plane;
      if (!STASH) {
        if (mirror) {
          uint32_t y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = x[i];
          store_regs<false>(y, out + t.m * u.ld + n, u.ld, t.mcount, ncount, u.vec);
        }
        store_regs<true>(x, out + n * u.ld + t.m, u.ld, ncount, t.mcount, u.vec);
      } else if (whole) {
        store_whole<true>(x, t, t.by_n + plane + 4 * cb * t.step);
        if (mirror) store_whole<false>(x, t, out + (t.m + (lane >> 2)) * u.ld + n + (lane & 3) * 8);
      } else {
        store_part<true>(x, t, stash, out + n * u.ld + t.m, u.ld, ncount, t.mcount);
        if (mirror) store_part<false>(x, t, stash, out + t.m * u.ld + n, u.ld, t.mcount, ncount);
      }
    };
    if (!STASH && u.planes_out == 2) {  // FP16 slices: the second is what the first leaves; both take the sums' registers
      uint32_t l[16];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const __half2 h = __floats2half2_rn(v[i], v[i + 1]);
        const __half2 r = __floats2half2_rn(v[i] - __low2float(h), v[i + 1] - __high2float(h));
        w[i >> 1] = *reinterpret_cast<const uint32_t*>(&h);
        l[i >> 1] = *reinterpret_cast<const uint32_t*>(&r);
      }
      store(w, 0);
      store(l, u.plane);
    } else {
      pack_block(v, w, u.out_type == kOutBf16);
      store(w, 0);
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

// The producer's loop over a unit's stages, compiled for each way its operands are copied, so that
// a stage is a wait, an arrival and (mostly) two copies and nothing else: boxes hold both slices.
// KA: K-major, MN-major 4-D, MN-major in two 3-D boxes.  KB: K-major in one box, in several,
// MN-major 4-D, 3-D boxes.  Returns false when a wait ran out or the pair was stopped.
template <int KA, int KB, int PLANES>
__device__ __forceinline__ bool load_unit(const Unit& u, uint8_t* sA, uint8_t* sB, uint64_t* empty, uint32_t full_leader,
                                          uint32_t rank, int& stage, uint32_t& phase, uint32_t& issued,
                                          const volatile int* abort_flag) {
  typedef Ring<PLANES> R;
  const int rowA = u.m0 + static_cast<int>(rank) * HALF_M;
  const int rowB = u.n0 + static_cast<int>(rank) * (u.nmma >> 1);
  const uint32_t bytes = R::A_STAGE + (KB == 0 || KB == 2 ? 1 : u.boxes) * u.box_bytes;
  int k = u.k0 + u.kb0 * BK;
  for (int kb = u.kb0; kb < u.kb1; ++kb, k += BK) {
    if (!mbar_wait_or_abort(&empty[stage], phase ^ 1, kWaitLimitNs, abort_flag)) return false;
    const uint32_t bar = full_leader + stage * 8;
    mbar_arrive_expect_tx_cluster(bar, bytes);
    uint8_t* dA = sA + stage * R::A_STAGE;
    uint8_t* dB = sB + stage * R::B_STAGE;
    if (KA == 0) {
      tma_load_3d_pair(dA, u.mapA, bar, k, rowA, u.zA);
    } else if (KA == 1) {
      tma_load_4d_pair(dA, u.mapA, bar, 0, k, rowA / 64, u.zA);
    } else {
      tma_load_3d_pair(dA, u.mapA, bar, rowA, k, u.zA);
      tma_load_3d_pair(dA + MN_BLOCK, u.mapA, bar, rowA + 64, k, u.zA);
    }
    if (KB == 0) {
      tma_load_3d_pair(dB, u.mapB, bar, k, rowB, u.zB);
    } else if (KB == 1) {
      for (int b = 0; b < u.boxes; ++b) tma_load_3d_pair(dB + b * u.box_bytes, u.mapB, bar, k, rowB + u.box_b * b, u.zB);
    } else if (KB == 2) {  // a last, narrower tile loads the full box: the stage has room for it
      tma_load_4d_pair(dB, u.mapB, bar, 0, k, rowB / 64, u.zB);
    } else {
      for (int b = 0; b < u.boxes; ++b) tma_load_3d_pair(dB + b * MN_BLOCK, u.mapB, bar, rowB + 64 * b, k, u.zB);
    }
    ++issued;
    if (++stage == R::STAGES) {
      stage = 0;
      phase ^= 1;
    }
  }
  return true;
}

// The kernel.  Walk deals out the units: Walk::Params are the launch's, setup() runs once for the
// whole CTA, and a Walk of its own in every role gives the pair's units in order (next).  kChained: units
// depend on one another.  ready()
// waits for what a unit depends on (the producer, or a warp of its own ahead of it), done() reports a tile (one
// thread of each CTA, when all its warps have stored their blocks), and gave_up() tells the other
// pairs that they wait in vain.  Otherwise outside() stores what belongs to no unit.
template <class Walk>
constexpr int kThreadsOf = (EPI_FIRST + Walk::kEpiWarps + (Walk::kChained ? 1 : 0)) * 32;

template <class Walk, int PLANES>
__global__ void __launch_bounds__(kThreadsOf<Walk>, 1)
    product_kernel(const __grid_constant__ typename Walk::Params a) {
  typedef Ring<PLANES> R;
  constexpr int STAGES = R::STAGES;
  constexpr int EPI_WARPS = Walk::kEpiWarps;
  constexpr int COLS = EPI_WARPS / 4;                 // warps that share the blocks of 32 columns of a quadrant
  constexpr int RUNS = PLANES == 2 ? (BN2 / 32 + COLS - 1) / COLS : 1;  // two slices: blocks whose sums a warp holds
  constexpr uint32_t STASH = EPI_WARPS * R::WARP_STASH;
  constexpr uint32_t NACC = PLANES == 2 ? 3 : 2, ACC_COLS = PLANES == 2 ? BN2 : BN;  // accumulators, their columns
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * R::A_STAGE;
  uint8_t* stash = smem + R::BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stash + STASH);
  uint64_t* full = bars;                   // [STAGES] TMA (both CTAs) -> MMA  (used in the leader)
  uint64_t* empty = bars + STAGES;         // [STAGES] MMA -> TMA              (both CTAs)
  uint64_t* accfull = bars + 2 * STAGES;   // [NACC]   MMA -> epilogue         (both CTAs)
  uint64_t* accempty = accfull + NACC;     // [NACC]   epilogues (both) -> MMA (used in the leader)
  uint64_t* drain = accempty + NACC;         // [1]      all MMAs of the pair done (both CTAs)
  uint64_t* epibar = drain + 1;            // [1]      epilogue warps rendezvous (per CTA)
  uint64_t* exitbar = epibar + 1;          // [1]      the peer has finished (per CTA)
  uint64_t* proddone = exitbar + 1;        // [1]      both producers have stopped (used in the leader)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(proddone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued_by = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);  // [2] (leader)
  volatile uint32_t* arrived = issued_by + 2;
  uint32_t* warps_done = const_cast<uint32_t*>(issued_by + 3);  // [4]
  uint32_t* units_ready = warps_done + 4;
  int* table = reinterpret_cast<int*>(stash + STASH + 256);  // the walker's

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 1);
    }
    for (uint32_t i = 0; i < NACC; ++i) {
      mbar_init(&accfull[i], 1);
      mbar_init(&accempty[i], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(epibar, EPI_WARPS);
    mbar_init(exitbar, 1);
    mbar_init(proddone, 2);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) warps_done[i] = 0;
    *units_ready = 0;
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

  if (warp == 0) {
    if (elect_one()) {
      // ------------------------------------------------------------ TMA producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0;
      uint32_t seq = 0;
      const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
      Walk walk(a, table);
      Unit u{};
      while (!*abort_flag && walk.next(u)) {
        if constexpr (Walk::kChained) {
          if (!(a.scout ? wait_for_count(units_ready, ++seq, abort_flag) : walk.ready(abort_flag))) {
            if (!*abort_flag) stop_pair(abort_flag, a.status);
            break;
          }
        }
        const int kind_b = !u.b_mn ? (u.boxes == 1 ? 0 : 1) : (u.b_4d ? 2 : 3);
        bool ok;
#define OZ_LOAD(KA, KB) load_unit<KA, KB, PLANES>(u, sA, sB, empty, full_leader, rank, stage, phase, issued, abort_flag)
        if (!u.a_mn)
          ok = kind_b == 0 ? OZ_LOAD(0, 0) : OZ_LOAD(0, 1);
        else if (u.a_4d)
          ok = kind_b == 0 ? OZ_LOAD(1, 0) : kind_b == 1 ? OZ_LOAD(1, 1) : kind_b == 2 ? OZ_LOAD(1, 2) : OZ_LOAD(1, 3);
        else
          ok = kind_b == 0 ? OZ_LOAD(2, 0) : kind_b == 1 ? OZ_LOAD(2, 1) : kind_b == 2 ? OZ_LOAD(2, 2) : OZ_LOAD(2, 3);
#undef OZ_LOAD
        if (!ok) {
          if (!*abort_flag) stop_pair(abort_flag, a.status);
          break;
        }
      }
      // Every issued copy must have landed before the pair may exit (see the residue GEMM).
      st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(&issued_by[rank])), 0), issued);
      mbar_arrive_release_cluster(mapa_shared(smem_u32(proddone), 0));
      if (!*abort_flag) {
        for (uint32_t i = 0; i < STAGES && i < issued; ++i) {
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
    if (rank == 0 && elect_one()) {
      // ------------------------------------------------------------ MMA issuer (leader only)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t acc = 0, acc_phase = 1;  // the next accumulator, and the parity of its being free
      uint32_t consumed = 0;
      bool ok = true;
      auto sum_done = [&]() {
        umma_commit_pair(&accfull[acc], 0x3);
        if (++acc == NACC) {
          acc = 0;
          acc_phase ^= 1;
        }
      };
      Walk walk(a, table);
      Unit u{};
      while (ok && !*abort_flag && walk.next(u)) {
        // Low words of stage 0's descriptors; a stage or a k step only adds to the address field.
        const uint32_t a_desc = desc_low(smem_u32(sA), u.a_mn), b_desc = desc_low(smem_u32(sB), u.b_mn);
        const uint32_t a_step = (u.a_mn ? UMMA_K * 128 : UMMA_K * 2) >> 4, b_step = (u.b_mn ? UMMA_K * 128 : UMMA_K * 2) >> 4;
        const uint32_t idesc = u.idesc | (static_cast<uint32_t>(u.nmma >> 3) << 17);
        int left = u.kb1 - u.kb0;
        if (left == 0) continue;
        uint32_t in_chunk = 0, d_tmem = 0;
        if (PLANES == 1) {  // the whole part in one accumulator
          if (!mbar_wait_or_abort(&accempty[acc], acc_phase, kWaitLimitNs, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          d_tmem = tmem_base + acc * ACC_COLS;
        }
        for (; left > 0; --left) {
          if (!mbar_wait_or_abort(&full[stage], phase, kWaitLimitNs, abort_flag)) {
            ok = false;
            break;
          }
          ++consumed;
          tc_fence_after();
          const uint32_t ad = a_desc + stage * (R::A_STAGE >> 4), bd = b_desc + stage * (R::B_STAGE >> 4);
          if constexpr (PLANES == 1) {
#pragma unroll
            for (int kk = 0; kk < KSTEPS; ++kk) {
              umma_pair(d_tmem, ad + kk * a_step, bd + kk * b_step, idesc, kk > 0 ? 1u : in_chunk);
              in_chunk = 1;
            }
          } else {
            // A chunk is a whole k-block or a single step; the small products come first, so that the
            // truncation of their additions is small too.
            const uint32_t al = ad + (A_PLANE >> 4), bl = bd + (u.b_plane >> 4);
            auto next_sum = [&]() {
              if (!mbar_wait_or_abort(&accempty[acc], acc_phase, kWaitLimitNs, abort_flag)) return false;
              tc_fence_after();
              d_tmem = tmem_base + acc * ACC_COLS;
              return true;
            };
            if (u.chunk == KSTEPS) {
              if (!next_sum()) {
                ok = false;
                break;
              }
#pragma unroll
              for (int kk = 0; kk < KSTEPS; ++kk) {
                umma_pair(d_tmem, ad + kk * a_step, bl + kk * b_step, idesc, kk > 0 ? 1u : 0u);
                umma_pair(d_tmem, al + kk * a_step, bd + kk * b_step, idesc, 1u);
              }
#pragma unroll
              for (int kk = 0; kk < KSTEPS; ++kk) umma_pair(d_tmem, ad + kk * a_step, bd + kk * b_step, idesc, 1u);
              sum_done();
            } else {
              for (int kk = 0; kk < KSTEPS; ++kk) {
                if (!next_sum()) {
                  ok = false;
                  break;
                }
                umma_pair(d_tmem, ad + kk * a_step, bl + kk * b_step, idesc, 0u);
                umma_pair(d_tmem, al + kk * a_step, bd + kk * b_step, idesc, 1u);
                umma_pair(d_tmem, ad + kk * a_step, bd + kk * b_step, idesc, 1u);
                sum_done();
              }
            }
            if (!ok) break;
          }
          umma_commit_pair(&empty[stage], 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (PLANES == 1) {
          sum_done();
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
  } else if (warp < EPI_FIRST + EPI_WARPS) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // A warp drains its 32 lanes and every COLS-th block of 32 columns.
    const int quad = warp & 3;
    const int first = (warp - EPI_FIRST) >> 2;
    const int mrow = static_cast<int>(rank) * HALF_M + quad * 32;
    uint8_t* my_stash = stash + (warp - EPI_FIRST) * R::WARP_STASH;
    uint32_t acc = 0, acc_phase = 0, eph = 0, seq = 0;
    bool ok = true;
    Walk walk(a, table);
    if constexpr (!Walk::kChained) walk.outside(warp - EPI_FIRST);
    Unit u{};
    for (; ok && walk.next(u); ++seq) {
      const int nblocks = ceil_div(u.nn, 32);  // this warp: blocks first, first + COLS, ...
      // Two slices: the sums take all registers meanwhile, so the unit waits in shared memory (working it
      // out anew took 0.8 us a tile).
      Unit* kept = reinterpret_cast<Unit*>(my_stash);
      if (PLANES == 2) {
        __syncwarp();
        if (lane == 0) *kept = u;
        __syncwarp();
      }
      Target target;
      bool split;
      auto place = [&]() {  // where the tile's blocks go
        if (PLANES == 2) u = *kept;
        target = target_of(u, mrow, my_stash);
        split = u.nsplit > 1;
      };
      auto parts = [&](int q) {  // this thread's values of part q of a split tile
        return u.part + (2ll * q + rank) * u.part_cols * HALF_M + quad * 1024 + lane * 4;
      };
      if (PLANES == 1) place();
      float run[RUNS][32];  // two slices: the sums of this warp's blocks
      if (PLANES == 2) {
#pragma unroll
        for (int i = 0; i < RUNS * 32; ++i) run[i >> 5][i & 31] = 0.0f;
      }
      int nchunks = u.kb1 > u.kb0;
      if (PLANES == 2) nchunks = (u.kb1 - u.kb0) * (u.chunk == 1 ? KSTEPS : 1);
      for (int ch = 0; ch < nchunks; ++ch) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_or_abort(&accfull[acc], acc_phase, a.epi_wait_ns, abort_flag))) {
          ok = false;
          if (lane == 0 && !*abort_flag) stop_pair(abort_flag, a.status);
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * ACC_COLS;
        if (PLANES == 2) {
#pragma unroll
          for (int j = 0; j < RUNS; ++j) {
            const int cb = COLS * j + first;
            if (cb < nblocks) {
              float v[32];
              tmem_ld_block(taddr + cb * 32, v);
              tmem_wait_block(v);
#pragma unroll
              for (int i = 0; i < 32; i += 2) add_two(run[j][i], run[j][i + 1], v[i], v[i + 1]);
            }
          }
        } else {
#pragma unroll 1
          for (int cb = first; cb < nblocks; cb += COLS) {
            float v[32];
            tmem_ld_block(taddr + cb * 32, v);
            tmem_wait_block(v);
            if (cb + COLS >= nblocks) {  // the last block is in registers: hand the accumulator back
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&accempty[acc]), 0));
            }
            if (split)
              put_part(parts(u.split) + cb * PART_BLOCK, v);
            else
              emit<Walk::kScaled, PLANES == 1>(u, target, v, cb, my_stash);
          }
        }
        if (PLANES == 2 || first >= nblocks) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&accempty[acc]), 0));
        }
        if (++acc == NACC) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (!ok) break;
      if (PLANES == 2) {
        place();
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
          const int cb = COLS * j + first;
          if (cb < nblocks) {
            if (split)
              put_part(parts(u.split) + cb * PART_BLOCK, run[j]);
            else
              emit<Walk::kScaled, PLANES == 1>(u, target, run[j], cb, my_stash);
          }
        }
      } else if (nchunks == 0) {  // an empty sum (a group without rows, or with few for this many parts)
#pragma unroll 1
        for (int cb = first; cb < nblocks; cb += COLS) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
          if (split)
            put_part(parts(u.split) + cb * PART_BLOCK, v);
          else
            emit<Walk::kScaled, PLANES == 1>(u, target, v, cb, my_stash);
        }
      }
      bool finished = true;
      if (split) {
        // This CTA's part is written; the last of the tile's parts to arrive adds them all.  One thread's
        // fences order what all warps wrote before they met, and what they read after they meet again.
        ok = warps_meet(epibar, eph, abort_flag);
        if (ok && threadIdx.x == EPI_FIRST * 32) {
          wait_for_previous();  // the arrival counters' zeros may come from a launch that this one overlaps
          __threadfence();
          *arrived = atomicAdd(&u.arrivals[rank], 1u);  // all have read the last one: they met since
          __threadfence();
        }
        ok = ok && warps_meet(epibar, eph, abort_flag);
        finished = ok && *arrived == static_cast<uint32_t>(u.nsplit - 1);
        if (!ok) {
          if (lane == 0 && !*abort_flag) stop_pair(abort_flag, a.status);
          break;
        }
        if (finished) {
          if (threadIdx.x == EPI_FIRST * 32) u.arrivals[rank] = 0;  // as it was found: a later unit may use it
#pragma unroll 1
          for (int cb = first; cb < nblocks; cb += COLS) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            for (int q = 0; q < u.nsplit; ++q) add_part(parts(q) + cb * PART_BLOCK, v);
            emit<Walk::kScaled, PLANES == 1>(u, target, v, cb, my_stash);
          }
        }
      }
      // The CTA's last warp to have stored its blocks reports the tile, so that a tile is one fence and
      // one global atomic a CTA (one a warp: the 1152 of a 2048-wide product held the next one up by 2 us).
      if constexpr (Walk::kChained) {
        if (finished) {
          __syncwarp();
          if (lane == 0) {
            // A warp can be NACC units ahead of another (the next one needs an accumulator that the other
            // has yet to hand back), so units in a row count apart.
            static_assert(NACC + 1 <= 4, "counters of warps_done");
            if (add_shared_acq_rel(&warps_done[seq & 3], 1u) == EPI_WARPS - 1) {
              warps_done[seq & 3] = 0;
              __threadfence();  // of all warps' stores: they were counted before this
              walk.done();
            }
          }
        }
      }
    }
  }

  if constexpr (Walk::kChained) {
    if (warp == EPI_FIRST + EPI_WARPS && a.scout && elect_one()) {
      // ---------------------------------------------------------- scout (both CTAs)
      // Runs ahead of the producer and counts the units that need not wait any more, so that a unit
      // whose operands have been there for a while costs the producer a look at shared memory and not a
      // global load and two fences (1.3 us between units).  Its word comes 0.1 us late, so it is asked
      // only where pairs have several units of a product (Params::scout): 8 x 1024 x 1024 bf16 206 ->
      // 198 us, 6 x 2048 x 2048 768 -> 734; one wave, 2048 x 2048, 193.5 without and 196.5 with it.
      Walk walk(a, table);
      Unit u{};
      for (uint32_t seq = 1; !*abort_flag && walk.next(u); ++seq) {
        if (!walk.ready(abort_flag)) {
          if (!*abort_flag) stop_pair(abort_flag, a.status);
          break;
        }
        asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(units_ready)), "r"(seq) : "memory");
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    wait_for_previous();  // no launch ends before the one that it overlapped
    if constexpr (Walk::kChained) {
      if (*abort_flag) Walk::gave_up(a);
    }
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

// [d2][d1][d0] with strides s1, s2 in bytes (multiples of 16); box {64, box_rows, mats}.
inline bool make_map(CUtensorMap* map, const void* base, bool bf16, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1,
                     uint64_t s2, int box_rows, int mats = 1) {
  const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1, s2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(mats)};
  return encode(map, base, bf16, 3, dims, strides, box);
}

// The same matrix for an MN-major operand: when d0 is a multiple of 64, a 4-D map
// [d2][d0 / 64][d1][64] whose box is 64 rows by `blocks` blocks of 64 contiguous elements; otherwise
// (a last partial block in such a map would reach past the end of the last row) make_map's, one
// block a box.  *is_4d says which: a load's rank has to be its map's.
inline bool make_mn_map(CUtensorMap* map, int* is_4d, int blocks, const void* base, bool bf16, uint64_t d0, uint64_t d1,
                        uint64_t d2, uint64_t s1, uint64_t s2, int mats = 1) {
  *is_4d = d0 % 64 == 0;
  if (!*is_4d) return make_map(map, base, bf16, d0, d1, d2, s1, s2, BK, mats);
  const cuuint64_t dims[4] = {64, d1, d0 / 64, d2}, strides[3] = {s1, 128, s2};
  const cuuint32_t box[4] = {64, BK, static_cast<cuuint32_t>(blocks), static_cast<cuuint32_t>(mats)};
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

// How a launch follows the one before it.  Every kernel starts while that one ends, and sets itself up.
// kAfter: it then waits for that launch (one token, 8 experts of 1024 x 1024: 10.2 -> 7.8 us a call in a
// graph).  kOverlap: it waits only before it uses the arrival counters.  kCooperative: kAfter, and all
// CTAs have to run at once, since units depend on one another (the launch is refused if they cannot).
enum Start { kAfter, kOverlap, kCooperative };

template <class Walk, int PLANES>
int launch(typename Walk::Params a, const Device& d, int pairs, Start start, cudaStream_t stream) {  // on `pairs` CTA pairs
  auto kernel = product_kernel<Walk, PLANES>;
  constexpr size_t smem = 1024 /*alignment*/ + Ring<PLANES>::BYTES + Walk::kEpiWarps * Ring<PLANES>::WARP_STASH + 256 /*barriers*/ + Walk::kTableBytes;
  static_assert(smem <= 232448, "shared memory budget");
  // No other kernel that holds tensor memory fits beside this one on an SM (the smallest takes two blocks of
  // 16 KB, newton_small_kernel), so a launch that starts early cannot take the columns this one is waiting for.
  static_assert(smem + 2 * 16384 > 232448, "alone on its SM");
  a.status = d.status;
  a.epi_wait_ns = epilogue_wait_ns();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(kThreadsOf<Walk>, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[2].id = cudaLaunchAttributeCooperative;
  attr[2].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = start == kCooperative ? 3 : 2;
  // The shared-memory limit is the function's, in this context: set on the first launch, and again
  // should a launch be refused (a new context after a device reset).
  static std::atomic<bool> ready[64] = {};
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

}  // namespace prod
}  // namespace oz
