// oz_grouped.cu -- matrix products grouped by expert with ragged sizes, and their gradients.
//
//   forward  Y_e = W_e^T X_e     D[n, row] = sum_k W_e[k, n] X[k, row]    both operands K-major
//   dgrad    dX_e = W_e dY_e     D[k, row] = sum_n W_e[k, n] dY[n, row]   W MN-major, dY K-major
//   wgrad    dW_e = X_e dY_e^T   D[k, n] = sum_row X[k, row] dY[n, row]   both MN-major, ragged sum
// (column-major: a token is a column of X, Y, dX, dY).  One launch each; the row offsets stay on
// the device, where every CTA builds the table of tiles from them.  Operands whose address or
// strides TMA cannot take (multiples of 16 bytes) are laid out in the workspace first.
#include "oz_products.cuh"

namespace oz {
namespace {

using namespace prod;

constexpr int kMaxParts = 160;  // parts of split tiles the workspace holds: about two a CTA pair
constexpr int kMaxUnsplit = 64;  // k-blocks of the longest sum that is never split (may_split)

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

enum Op { kForward, kDgrad, kWgrad };

// Deals out the tiles of all groups from the row offsets on the device.
//   forward, dgrad: a group's rows in equal tiles (a multiple of 32 rows, at most 256) by the
//     output's m; the group's tiles by row tile, so that a wave shares the rows and the weights.
//   wgrad: the output's tiles for every group; the sum runs over the group's rows.  Its k-blocks of 64
//     rows are aligned to the END of the rows, which are addressed as (offset within the group,
//     first row): the first block starts at a negative offset, where TMA reads zeros.  No row of a
//     neighbouring group ever enters a sum, so its NaNs cannot leak.
template <Op OP>
struct GroupedWalk {
  static constexpr bool kScaled = false, kChained = false;
  static constexpr int kEpiWarps = 8;
  static constexpr size_t kTableBytes = (2 * (OZ_MAX_GROUPS + 1) + 3) * 4;  // offsets, tile prefix, the split
  static constexpr bool A_MN = OP != kForward, B_MN = OP == kWgrad, RAGGED_SUM = OP == kWgrad;
  static constexpr int BOX = 32;  // ragged rows: the small box of B (the large one has HALF_N rows)

  struct Params {
    CUtensorMap tmA, tmB, tmB128;
    int M, N, K;   // contiguous extent of the output; wgrad: its rows; otherwise the sum's length
    int groups, rows, bn, max_parts, part_cols;
    int a_4d, b_4d, vec, out_type, after;
    uint32_t idesc;
    const int32_t* offsets;
    void* out;
    long long ld, stride;
    float* part;
    unsigned int* arrivals;
    int* status;
    unsigned long long epi_wait_ns;
  };

  const Params& a;
  const int *off, *prefix;
  int full, nsplit, total, idx, tiles_m, tiles_n;

  // Offsets are clamped to [0, rows] and to their predecessors, so that no access leaves the
  // matrices whatever they hold; offsets that needed it are reported.
  __device__ static void setup(const Params& a, int* table) {
    int* off = table;
    int* prefix = table + OZ_MAX_GROUPS + 1;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
      tma_prefetch_desc(&a.tmA);
      tma_prefetch_desc(&a.tmB);
      if (!B_MN) tma_prefetch_desc(&a.tmB128);
    }
    // A product after this one may set itself up on SMs that this one leaves idle; it waits here too.
    let_next_start();
    if (a.after) wait_for_previous();
    for (int i = threadIdx.x; i <= a.groups; i += blockDim.x) off[i] = a.offsets[i];
    __syncthreads();
    if (threadIdx.x >= 32) return;
    const int tiles_m = ceil_div(a.M, BM);
    int before = 0, sum = 0;
    bool bad = false;
    for (int b = 0; b <= a.groups; b += 32) {
      const int i = b + lane;
      const int given = i <= a.groups ? off[i] : 0;
      int v = max(0, min(given, a.rows));
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v = max(v, o);
      }
      v = max(v, before);
      bad |= i <= a.groups && v != given;
      int prev = __shfl_up_sync(0xFFFFFFFFu, v, 1);
      if (lane == 0) prev = before;
      before = __shfl_sync(0xFFFFFFFFu, v, 31);
      int t = (i >= 1 && i <= a.groups) ? ceil_div(v - prev, a.bn) * tiles_m : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, t, d);
        if (lane >= d) t += o;
      }
      if (i <= a.groups) {
        off[i] = v;
        prefix[i] = sum + t;
      }
      sum += __shfl_sync(0xFFFFFFFFu, t, 31);
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0 && blockIdx.x == 0) atomicExch(a.status, OZ_EINVAL);
    // Parts of the last wave's tiles: a lane weighs each count, the least cost (then count) wins.
    const int pairs = static_cast<int>(gridDim.x >> 1);
    const int tiles = RAGGED_SUM ? a.groups * tiles_m * ceil_div(a.N, a.bn) : sum;
    const int rest = tiles % pairs;
    const int nkb = ceil_div(RAGGED_SUM ? before : a.K, RAGGED_SUM ? BK * a.groups : BK);
    int cost = lane < kMaxSplit && (lane == 0 || a.max_parts)
                   ? split_cost(rest, nkb, pairs, a.max_parts, a.part_cols, lane + 1) : 1 << 30;
    cost = min(cost, (1 << 25)) * 32 + lane;
    cost = __reduce_min_sync(0xFFFFFFFFu, cost);
    if (lane == 0) {
      int* split = prefix + OZ_MAX_GROUPS + 1;
      split[0] = tiles;
      split[1] = tiles - rest;
      split[2] = (cost & 31) + 1;
    }
  }

  __device__ GroupedWalk(const Params& p, const int* table) : a(p), off(table), prefix(table + OZ_MAX_GROUPS + 1) {
    const int pairs = static_cast<int>(gridDim.x >> 1);
    const int* split = prefix + OZ_MAX_GROUPS + 1;
    tiles_m = ceil_div(a.M, BM);
    tiles_n = RAGGED_SUM ? ceil_div(a.N, a.bn) : 0;
    full = split[1];
    nsplit = split[2];
    total = full + (split[0] - full) * nsplit;
    idx = static_cast<int>(blockIdx.x >> 1) - pairs;
  }

  __device__ bool next(Unit& u) {
    idx += static_cast<int>(gridDim.x >> 1);
    if (idx >= total) return false;
    int tile = idx;
    u.split = 0;
    u.nsplit = 1;
    u.part = a.part;
    u.part_cols = a.part_cols;
    u.arrivals = a.arrivals;
    if (idx >= full && nsplit > 1) {
      const int r = (idx - full) / nsplit;
      tile = full + r;
      u.split = idx - full - r * nsplit;
      u.nsplit = nsplit;
      u.part = a.part + 2ll * r * nsplit * a.part_cols * HALF_M;
      u.arrivals = a.arrivals + 2 * r;
    }
    int group, nkb;
    if (RAGGED_SUM) {
      const int per = tiles_m * tiles_n;
      group = tile / per;
      const int r = tile - group * per, tn = r / tiles_m;
      u.m0 = (r - tn * tiles_m) * BM;
      u.n0 = u.orow = tn * a.bn;
      u.nn = min(a.bn, a.N - u.n0);
      const int len = off[group + 1] - off[group];
      nkb = ceil_div(len, BK);
      u.k0 = len - nkb * BK;
      u.zA = u.zB = off[group];
    } else {
      int lo = 0, hi = a.groups;  // prefix[group] <= tile < prefix[group + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= tile) lo = mid; else hi = mid;
      }
      group = lo;
      const int r = tile - prefix[group], tn = r / tiles_m;
      const int len = off[group + 1] - off[group];
      // equal tiles: as many as of full ones, with the least padding
      const int w = ceil_div(ceil_div(len, ceil_div(len, a.bn)), 32) * 32;
      u.m0 = (r - tn * tiles_m) * BM;
      u.n0 = u.orow = off[group] + tn * w;
      u.nn = min(w, len - tn * w);
      nkb = ceil_div(a.K, BK);
      u.k0 = 0;
      u.zA = group;
      u.zB = 0;
    }
    u.nmma = B_MN ? ceil_div(u.nn, 128) * 128 : ceil_div(u.nn, 32) * 32;
    u.kb0 = static_cast<int>(static_cast<long long>(nkb) * u.split / u.nsplit);
    u.kb1 = static_cast<int>(static_cast<long long>(nkb) * (u.split + 1) / u.nsplit);
    u.a_mn = A_MN;
    u.b_mn = B_MN;
    u.a_4d = a.a_4d;
    u.b_4d = a.b_4d;
    // Few copies a stage: their issue, not their bytes, is what a stage waits for first.
    const bool wide = u.nmma > 128;
    u.mapA = &a.tmA;
    u.mapB = !B_MN && wide ? &a.tmB128 : &a.tmB;
    u.box_b = wide ? HALF_N : BOX;
    u.boxes = B_MN ? (a.b_4d ? 1 : u.nmma / 128) : wide ? 1 : ceil_div(u.nmma / 2, BOX);
    u.box_bytes = B_MN ? (a.b_4d ? a.bn / 128 : 1) * MN_BLOCK : u.box_b * BK * 2;
    u.idesc = a.idesc;
    u.m_extent = a.M;
    u.out = static_cast<uint16_t*>(a.out) + (RAGGED_SUM ? group * a.stride : 0);
    u.ld = a.ld;
    u.out_type = a.out_type;
    u.vec = a.vec;
    u.sym = false;
    u.planes_out = 1;
    u.plane = 0;
    u.f = 1.0f;
    u.diag = 0.0f;
    return true;
  }

  // Rows that belong to no group are zero.
  __device__ void outside(int warp) const {
    if (RAGGED_SUM) return;
    const int lo = off[0], hi = off[a.groups], loose = lo + a.rows - hi;
    for (int i = static_cast<int>(blockIdx.x) * kEpiWarps + warp; i < loose; i += gridDim.x * kEpiWarps) {
      uint16_t* row = static_cast<uint16_t*>(a.out) + static_cast<long long>(i < lo ? i : hi + i - lo) * a.ld;
      for (int c = threadIdx.x & 31; c < a.M; c += 32) row[c] = 0;
    }
  }
};

struct Operand {
  const void* p;
  long long cols, rows, mats;  // contiguous extent, rows, matrices
  long long ld, stride;
  bool fits() const {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && (mats == 1 || stride % 8 == 0);
  }
  size_t repack_bytes() const {
    return fits() ? 0 : align256(2 * static_cast<size_t>(roundup(cols, 8)) * rows * mats);
  }
};

__global__ void zero_kernel(unsigned* words) {
  let_next_start();
  words[threadIdx.x] = 0;
}

// Operands laid out anew: [mats][rows][cols] of 16-bit elements to rows of ldo (a multiple of 8).  2^shift
// lanes a row, 8 elements a lane: the two aligned 16-byte vectors that hold them where both lie in
// the row, shifted into place, and single elements at its ends.  Both operands are one launch.  Bound by
// the bytes of a copy.  (1777 rows of 1001 and 7 experts of 1001 x 517, with their product: 18.6 us; 27.2 with a
// launch each and a division an element group.)
struct Repack {
  const uint16_t* in;
  long long ld, stride;
  uint16_t* out;
  int cols, ldo;
  long long rows, all;  // of a matrix, of all matrices
};

__global__ void __launch_bounds__(256) repack_kernel(const __grid_constant__ Repack first, const __grid_constant__ Repack second,
                                                     int shift) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & ((1 << shift) - 1);
  const long long step = static_cast<long long>(gridDim.x) * (256 >> shift);
  for (long long i = static_cast<long long>(blockIdx.x) * (256 >> shift) + (threadIdx.x >> shift); i < first.all + second.all;
       i += step) {
    const Repack& o = i < first.all ? first : second;
    const long long row = i < first.all ? i : i - first.all, mat = row / o.rows;
    const uint16_t* src = o.in + mat * o.stride + (row - mat * o.rows) * o.ld;
    uint16_t* dst = o.out + row * o.ldo;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / 2;  // elements past an aligned address
    for (int c = lane * 8; c < o.ldo; c += 8 << shift) {
      uint32_t w[8];
      if (c >= off && c - off + 16 <= o.cols) {
        const uint4* v = reinterpret_cast<const uint4*>(src + c - off);
        const uint4 x = v[0], y = v[1];
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
        if (off & 4) {
#pragma unroll
          for (int e = 0; e < 6; ++e) w[e] = w[e + 2];
        }
        if (off & 2) {
#pragma unroll
          for (int e = 0; e < 5; ++e) w[e] = w[e + 1];
        }
        if (off & 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = __funnelshift_r(w[e], w[e + 1], 16);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = c + 2 * e < o.cols ? src[c + 2 * e] : 0, hi = c + 2 * e + 1 < o.cols ? src[c + 2 * e + 1] : 0;
          w[e] = lo | (hi << 16);
        }
      }
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// The operands among a and b that TMA cannot take, laid out in the workspace.
int repack(Operand& a, Operand& b, uint8_t* ws, cudaStream_t stream) {
  Repack jobs[2] = {};
  int n = 0;
  for (Operand* o : {&a, &b}) {
    if (o->fits()) continue;
    uint16_t* out = reinterpret_cast<uint16_t*>(ws);
    const int ldo = static_cast<int>(roundup(o->cols, 8));
    jobs[n++] = Repack{static_cast<const uint16_t*>(o->p), o->ld, o->stride, out, static_cast<int>(o->cols), ldo, o->rows, o->rows * o->mats};
    ws += o->repack_bytes();
    *o = Operand{out, o->cols, o->rows, o->mats, ldo, static_cast<long long>(ldo) * o->rows};
  }
  if (n == 0) return OZ_OK;
  const int widest = jobs[0].ldo > jobs[1].ldo ? jobs[0].ldo : jobs[1].ldo;
  int shift = 0;
  while (shift < 5 && (8 << shift) < widest) ++shift;
  const long long per = 256 >> shift, blocks = (jobs[0].all + jobs[1].all + per - 1) / per;
  const unsigned grid = static_cast<unsigned>(blocks < 8192 ? blocks : 8192);
  return launch_overlapping(repack_kernel, dim3(grid), 256, 0, stream, jobs[0], jobs[1], shift) == cudaSuccess ? OZ_OK : OZ_ECUDA;
}

struct Problem {
  Op op;
  int n, k, rows, groups, dtype;
  Operand w, t;  // forward: W, X; dgrad: W, dY; wgrad: X (operand A), dY (operand B)
  const int32_t* offsets;
  void* out;
  int ldo;
  long long strideo;

  int m_out() const { return op == kForward ? n : k; }
  int bn() const { return op == kWgrad && n <= 128 ? 128 : 256; }
  // Whether tiles are left for a split is known on the device only, but parts need arrival counters
  // that a launch before the product's has to zero, and a rendezvous: 1.4 to 4.6 us (from the host, with the
  // allocation of a workspace, 3 to 8).  Parts win that back only when a sum is long.  In a graph, us unsplit / split,
  // one token of 8 experts with n = 1024, and 512 rows of one with n = 4096:
  //   k 1024:  8.4 / 11.3, 10.6 / 12.0    k 2048: 11.8 / 14.4, 15.0 / 19.6    k 4096: 18.4 / 19.9, 23.5 / 24.0
  //   k 6144: 25.4 / 25.3, 31.9 / 28.4    k 8192: 32.5 / 30.6, 40.5 / 33.9    k 16384: 60.5 / 53.0, 74.2 / 52.2
  bool may_split() const {
    const int blocks = op == kWgrad ? ceil_div(rows, BK * groups) : ceil_div(op == kForward ? k : n, BK);
    return blocks > kMaxUnsplit;
  }
  int part_cols() const { return op == kWgrad ? bn() : static_cast<int>(roundup(rows < bn() ? rows : bn(), 32)); }
  size_t split_bytes() const {
    if (!may_split()) return 0;
    return align256(sizeof(unsigned) * 2 * kMaxParts) + align256(sizeof(float) * 2 * HALF_M * part_cols() * kMaxParts);
  }
  int sum() const { return op == kForward ? k : op == kDgrad ? n : rows; }
  bool empty() const { return m_out() == 0 || (op == kWgrad ? n : rows) == 0; }
  bool has_operands() const { return out && offsets && (sum() == 0 || (w.p && t.p)); }
  size_t workspace() const { return split_bytes() + w.repack_bytes() + t.repack_bytes(); }
};

int check(int n, int k, int rows, int groups, int dtype, int ldw, long long stride_w, int ldk, int ldn) {
  if (n < 0 || k < 0 || rows < 0 || n > kMaxExtent || k > kMaxExtent || rows > kMaxExtent || groups < 1 || groups > OZ_MAX_GROUPS) return OZ_EINVAL;
  if (dtype != OZ_BF16 && dtype != OZ_F16) return OZ_EINVAL;
  if (ldw < (k > 1 ? k : 1) || ldk < (k > 1 ? k : 1) || ldn < (n > 1 ? n : 1)) return OZ_EINVAL;
  if (groups > 1 && stride_w < static_cast<long long>(ldw) * n) return OZ_EINVAL;
  return OZ_OK;
}

// The matrices outside every sum: zeros of the output.
int zero_output(const Problem& p, cudaStream_t stream) {
  const size_t width = 2 * static_cast<size_t>(p.m_out()), pitch = 2 * static_cast<size_t>(p.ldo);
  const int mats = p.op == kWgrad ? p.groups : 1, rows = p.op == kWgrad ? p.n : p.rows;
  for (int e = 0; e < mats; ++e)
    if (cudaMemset2DAsync(static_cast<uint8_t*>(p.out) + 2 * e * p.strideo, pitch, 0, width, rows, stream) != cudaSuccess)
      return OZ_ECUDA;
  return OZ_OK;
}

template <Op OP>
int launch_op(const Problem& p, float* part, unsigned* arrivals, const Device& dev, Start start, cudaStream_t stream) {
  typedef GroupedWalk<OP> Walk;
  const bool bf16 = p.dtype == OZ_BF16;
  typename Walk::Params a{};
  a.M = p.m_out();
  a.N = p.n;
  a.K = OP == kForward ? p.k : p.n;
  a.groups = p.groups;
  a.rows = p.rows;
  a.bn = p.bn();
  a.max_parts = part ? (kMaxParts < 2 * dev.pairs ? kMaxParts : 2 * dev.pairs) : 0;
  a.part_cols = p.part_cols();
  a.idesc = idesc_base(bf16, Walk::A_MN, Walk::B_MN);
  a.out_type = bf16 ? kOutBf16 : kOutF16;
  a.offsets = p.offsets;
  a.out = p.out;
  a.ld = p.ldo;
  a.stride = p.strideo;
  a.vec = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.ldo % 8 == 0 && (p.op != kWgrad || p.strideo % 8 == 0);
  a.after = start == kAfter;
  a.part = part;
  a.arrivals = arrivals;
  const Operand &w = p.w, &t = p.t;
  const uint64_t wl = 2ull * w.ld, tl = 2ull * t.ld;
  bool ok;
  if (OP == kWgrad) {  // rows as (offset within the group, the group's first row)
    ok = make_mn_map(&a.tmA, &a.a_4d, 2, w.p, bf16, w.cols, w.rows, w.rows, wl, wl) &&
         make_mn_map(&a.tmB, &a.b_4d, a.bn / 128, t.p, bf16, t.cols, t.rows, t.rows, tl, tl);
  } else {
    const uint64_t wm = w.mats > 1 ? 2ull * w.stride : wl * w.rows;
    ok = make_map(&a.tmB, t.p, bf16, t.cols, t.rows, 1, tl, tl * t.rows, Walk::BOX) &&
         (p.rows <= HALF_N || make_map(&a.tmB128, t.p, bf16, t.cols, t.rows, 1, tl, tl * t.rows, HALF_N)) &&
         (Walk::A_MN ? make_mn_map(&a.tmA, &a.a_4d, 2, w.p, bf16, w.cols, w.rows, w.mats, wl, wm)
                     : make_map(&a.tmA, w.p, bf16, w.cols, w.rows, w.mats, wl, wm, HALF_M));
  }
  if (p.rows <= HALF_N) a.tmB128 = a.tmB;  // no tile is that wide
  return ok ? launch<Walk, 1>(a, dev, dev.pairs, start, stream) : OZ_ECUDA;
}

int run(Problem p, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (p.empty()) return OZ_OK;
  if (!p.has_operands()) return OZ_EINVAL;
  if (p.sum() == 0) return zero_output(p, stream);
  const size_t need = p.workspace();
  if (need && (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))) return OZ_ENOMEM;
  Device dev;
  int rc;
  if ((rc = current_device(&dev))) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* part = nullptr;
  unsigned* arrivals = nullptr;
  if (p.may_split()) {
    arrivals = reinterpret_cast<unsigned*>(ws);
    part = reinterpret_cast<float*>(ws + align256(sizeof(unsigned) * 2 * kMaxParts));
    zero_kernel<<<1, 2 * kMaxParts, 0, stream>>>(arrivals);
    if (cudaGetLastError() != cudaSuccess) return OZ_ECUDA;
    ws += p.split_bytes();
  }
  // The product overlaps zero_kernel, which everything before it on the stream precedes; for anything
  // else before it, a repacked operand or a caller's launch, it waits.
  const Start start = arrivals && p.w.fits() && p.t.fits() ? kOverlap : kAfter;
  if ((rc = repack(p.w, p.t, ws, stream))) return rc;
  switch (p.op) {
    case kForward: return launch_op<kForward>(p, part, arrivals, dev, start, stream);
    case kDgrad: return launch_op<kDgrad>(p, part, arrivals, dev, start, stream);
    default: return launch_op<kWgrad>(p, part, arrivals, dev, start, stream);
  }
}

int run_allocating(const Problem& p, cudaStream_t stream) {
  const bool none = p.empty() || !p.has_operands() || p.sum() == 0;  // argument errors before any allocation
  const size_t bytes = none ? 0 : p.workspace();
  void* ws = nullptr;
  if (bytes) {
    keep_default_pool_cached();
    if (cudaMallocAsync(&ws, bytes, stream) != cudaSuccess) {
      cudaGetLastError();
      return OZ_ENOMEM;
    }
  }
  int rc = run(p, ws, bytes, stream);
  if (ws && cudaFreeAsync(ws, stream) != cudaSuccess && rc == OZ_OK) rc = OZ_ECUDA;
  return rc;
}

Problem forward(int n, int k, int rows, int groups, int dtype, const void* W, int ldw, long long sw, const void* X, int ldx,
                const int32_t* offsets, void* Y, int ldy) {
  return Problem{kForward, n, k, rows, groups, dtype, {W, k, n, groups, ldw, sw}, {X, k, rows, 1, ldx, 0}, offsets, Y, ldy, 0};
}
Problem dgrad(int n, int k, int rows, int groups, int dtype, const void* W, int ldw, long long sw, const void* dY, int lddy,
              const int32_t* offsets, void* dX, int lddx) {
  return Problem{kDgrad, n, k, rows, groups, dtype, {W, k, n, groups, ldw, sw}, {dY, n, rows, 1, lddy, 0}, offsets, dX, lddx, 0};
}
Problem wgrad(int n, int k, int rows, int groups, int dtype, const void* dY, int lddy, const void* X, int ldx,
              const int32_t* offsets, void* dW, int ldw, long long sw) {
  return Problem{kWgrad, n, k, rows, groups, dtype, {X, k, rows, 1, ldx, 0}, {dY, n, rows, 1, lddy, 0}, offsets, dW, ldw, sw};
}

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

size_t ozaki_grouped_gemm_workspace_bytes(int n, int k, int rows, int groups, int dtype, const void* W, int ldw,
                                          long long strideW, const void* X, int ldx) {
  if (check(n, k, rows, groups, dtype, ldw, strideW, ldx, n)) return 0;
  return forward(n, k, rows, groups, dtype, W, ldw, strideW, X, ldx, nullptr, nullptr, n).workspace();
}
size_t ozaki_grouped_gemm_dgrad_workspace_bytes(int n, int k, int rows, int groups, int dtype, const void* W, int ldw,
                                                long long strideW, const void* dY, int lddy) {
  if (check(n, k, rows, groups, dtype, ldw, strideW, k, lddy)) return 0;
  return dgrad(n, k, rows, groups, dtype, W, ldw, strideW, dY, lddy, nullptr, nullptr, k).workspace();
}
size_t ozaki_grouped_gemm_wgrad_workspace_bytes(int n, int k, int rows, int groups, int dtype, const void* dY, int lddy,
                                                const void* X, int ldx) {
  if (check(n, k, rows, groups, dtype, k, static_cast<long long>(k) * n, ldx, lddy)) return 0;
  return wgrad(n, k, rows, groups, dtype, dY, lddy, X, ldx, nullptr, nullptr, k, 0).workspace();
}

int ozaki_grouped_gemm_ws(int n, int k, int rows, int groups, int dtype, const void* W, int ldw, long long strideW,
                          const void* X, int ldx, const int32_t* offsets, void* Y, int ldy, void* workspace,
                          size_t ws_bytes, cudaStream_t stream) {
  const int rc = check(n, k, rows, groups, dtype, ldw, strideW, ldx, ldy);
  return rc ? rc : run(forward(n, k, rows, groups, dtype, W, ldw, strideW, X, ldx, offsets, Y, ldy), workspace, ws_bytes, stream);
}
int ozaki_grouped_gemm(int n, int k, int rows, int groups, int dtype, const void* W, int ldw, long long strideW,
                       const void* X, int ldx, const int32_t* offsets, void* Y, int ldy, cudaStream_t stream) {
  const int rc = check(n, k, rows, groups, dtype, ldw, strideW, ldx, ldy);
  return rc ? rc : run_allocating(forward(n, k, rows, groups, dtype, W, ldw, strideW, X, ldx, offsets, Y, ldy), stream);
}

int ozaki_grouped_gemm_dgrad_ws(int n, int k, int rows, int groups, int dtype, const void* W, int ldw, long long strideW,
                                const void* dY, int lddy, const int32_t* offsets, void* dX, int lddx, void* workspace,
                                size_t ws_bytes, cudaStream_t stream) {
  const int rc = check(n, k, rows, groups, dtype, ldw, strideW, lddx, lddy);
  return rc ? rc : run(dgrad(n, k, rows, groups, dtype, W, ldw, strideW, dY, lddy, offsets, dX, lddx), workspace, ws_bytes, stream);
}
int ozaki_grouped_gemm_dgrad(int n, int k, int rows, int groups, int dtype, const void* W, int ldw, long long strideW,
                             const void* dY, int lddy, const int32_t* offsets, void* dX, int lddx, cudaStream_t stream) {
  const int rc = check(n, k, rows, groups, dtype, ldw, strideW, lddx, lddy);
  return rc ? rc : run_allocating(dgrad(n, k, rows, groups, dtype, W, ldw, strideW, dY, lddy, offsets, dX, lddx), stream);
}

int ozaki_grouped_gemm_wgrad_ws(int n, int k, int rows, int groups, int dtype, const void* dY, int lddy, const void* X,
                                int ldx, const int32_t* offsets, void* dW, int ldw, long long strideW, void* workspace,
                                size_t ws_bytes, cudaStream_t stream) {
  const int rc = check(n, k, rows, groups, dtype, ldw, strideW, ldx, lddy);
  return rc ? rc : run(wgrad(n, k, rows, groups, dtype, dY, lddy, X, ldx, offsets, dW, ldw, strideW), workspace, ws_bytes, stream);
}
int ozaki_grouped_gemm_wgrad(int n, int k, int rows, int groups, int dtype, const void* dY, int lddy, const void* X,
                             int ldx, const int32_t* offsets, void* dW, int ldw, long long strideW, cudaStream_t stream) {
  const int rc = check(n, k, rows, groups, dtype, ldw, strideW, ldx, lddy);
  return rc ? rc : run_allocating(wgrad(n, k, rows, groups, dtype, dY, lddy, X, ldx, offsets, dW, ldw, strideW), stream);
}

}  // extern "C"
