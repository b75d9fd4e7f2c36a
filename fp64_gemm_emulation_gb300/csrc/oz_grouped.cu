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

constexpr int kMaxSplitUnits = 160;  // (tile, part) pairs the split workspace holds: about two a CTA pair

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

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

// Copies [mats][rows][cols] of 16-bit elements to rows of ldo (a multiple of 8): one thread per
// 8 output elements, 2-byte loads (the source has no alignment), one 16-byte store.
__global__ void repack_kernel(const uint16_t* __restrict__ in, long long ld, long long stride, uint16_t* __restrict__ out,
                              int cols, long long rows, long long mats, int ldo) {
  const int per = ldo / 8;
  const long long total = mats * rows * per;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long row = i / per;
    const int c = static_cast<int>(i - row * per) * 8;
    const long long mat = row / rows;
    const uint16_t* src = in + mat * stride + (row - mat * rows) * ld + c;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = c + 2 * e < cols ? src[2 * e] : 0, hi = c + 2 * e + 1 < cols ? src[2 * e + 1] : 0;
      w[e] = lo | (hi << 16);
    }
    *reinterpret_cast<uint4*>(out + row * ldo + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

int repack(Operand& o, uint8_t** ws, cudaStream_t stream) {
  if (o.fits()) return OZ_OK;
  uint16_t* out = reinterpret_cast<uint16_t*>(*ws);
  const int ldo = static_cast<int>(roundup(o.cols, 8));
  const long long total = o.mats * o.rows * (ldo / 8);
  const long long blocks = (total + 255) / 256;
  repack_kernel<<<static_cast<unsigned>(blocks < 8192 ? blocks : 8192), 256, 0, stream>>>(
      static_cast<const uint16_t*>(o.p), o.ld, o.stride, out, static_cast<int>(o.cols), o.rows, o.mats, ldo);
  if (cudaGetLastError() != cudaSuccess) return OZ_ECUDA;
  *ws += o.repack_bytes();
  o = Operand{out, o.cols, o.rows, o.mats, ldo, static_cast<long long>(ldo) * o.rows};
  return OZ_OK;
}

enum Op { kForward, kDgrad, kWgrad };

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
  int tiles_m() const { return ceil_div(m_out(), BM); }
  // Fewest tiles there can be (ragged rows: one tile in m), so whether a split is possible.
  bool may_split() const {
    const long long tiles = op == kWgrad ? static_cast<long long>(groups) * tiles_m() * ceil_div(n, bn()) : tiles_m();
    const long long blocks = op == kWgrad ? ceil_div(rows, BK * groups) : ceil_div(op == kForward ? k : n, BK);
    return tiles < kMaxSplitUnits && blocks > 1;
  }
  int part_cols() const { return op == kWgrad ? bn() : static_cast<int>(roundup(rows < bn() ? rows : bn(), 32)); }
  size_t split_bytes() const {
    if (!may_split()) return 0;
    return align256(sizeof(unsigned) * 2 * kMaxSplitUnits) + align256(sizeof(float) * 2 * HALF_M * part_cols() * kMaxSplitUnits);
  }
  size_t workspace() const { return split_bytes() + w.repack_bytes() + t.repack_bytes(); }
};

int check(int n, int k, int rows, int groups, int dtype, int ldw, long long stride_w, int ldk, int ldn) {
  if (n < 0 || k < 0 || rows < 0 || groups < 1 || groups > MAX_GROUPS) return OZ_EINVAL;
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

int run(Problem p, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  const int sum = p.op == kForward ? p.k : p.op == kDgrad ? p.n : p.rows;
  if (p.m_out() == 0 || (p.op == kWgrad ? p.n : p.rows) == 0) return OZ_OK;
  if (!p.out || !p.offsets) return OZ_EINVAL;
  if (sum == 0) return zero_output(p, stream);
  if (!p.w.p || !p.t.p) return OZ_EINVAL;
  const size_t need = p.workspace();
  if (need && (!workspace || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))) return OZ_ENOMEM;
  Device dev;
  int rc;
  if ((rc = current_device(&dev))) return rc;
  const int pairs = dev.pairs;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Args a{};
  if (p.may_split()) {
    a.counters = reinterpret_cast<unsigned*>(ws);
    a.part = reinterpret_cast<float*>(ws + align256(sizeof(unsigned) * 2 * kMaxSplitUnits));
    a.part_cols = p.part_cols();
    a.max_split_units = kMaxSplitUnits < 2 * pairs ? kMaxSplitUnits : 2 * pairs;
    if (cudaMemsetAsync(a.counters, 0, sizeof(unsigned) * 2 * kMaxSplitUnits, stream) != cudaSuccess) return OZ_ECUDA;
    ws += p.split_bytes();
  }
  if ((rc = repack(p.w, &ws, stream)) || (rc = repack(p.t, &ws, stream))) return rc;
  const bool bf16 = p.dtype == OZ_BF16;
  a.M = p.m_out();
  a.N = p.n;
  a.K = sum;
  a.groups = p.groups;
  a.rows = p.rows;
  a.bn = p.bn();
  a.nsplit = 1;
  a.chunk = 1 << 28;
  a.out_type = bf16 ? kOutBf16 : kOutF16;
  a.planes_out = 1;
  a.box_rows = BOX_ROWS;
  a.offsets = p.offsets;
  a.out = p.out;
  a.ld = p.ldo;
  a.stride = p.strideo;
  a.vec = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 && p.ldo % 8 == 0 && p.strideo % 8 == 0;
  a.alpha = 1.0f;
  CUtensorMap tmA, tmB, tmB128;
  const Operand &w = p.w, &t = p.t;
  const uint64_t wl = 2ull * w.ld, tl = 2ull * t.ld;
  if (p.op == kWgrad) {
    // rows addressed as (offset within the group, the group's first row)
    a.idesc = idesc_base(bf16, true, true);
    if (!make_mn_map(&tmA, &a.a_4d, 2, w.p, bf16, w.cols, w.rows, w.rows, wl, wl) ||
        !make_mn_map(&tmB, &a.b_4d, a.bn / 128, t.p, bf16, t.cols, t.rows, t.rows, tl, tl))
      return OZ_ECUDA;
    return launch<kRaggedK, true, true, 1>(tmA, tmB, tmB, a, dev, pairs, false, stream);
  }
  const uint64_t ws2 = w.mats > 1 ? 2ull * w.stride : wl * w.rows;
  if (!make_map(&tmB, t.p, bf16, t.cols, t.rows, 1, tl, tl * t.rows, BOX_ROWS) ||
      !make_map(&tmB128, t.p, bf16, t.cols, t.rows, 1, tl, tl * t.rows, HALF_N))
    return OZ_ECUDA;
  if (p.op == kForward) {
    a.idesc = idesc_base(bf16, false, false);
    if (!make_map(&tmA, w.p, bf16, w.cols, w.rows, w.mats, wl, ws2, HALF_M)) return OZ_ECUDA;
    return launch<kRaggedN, false, false, 1>(tmA, tmB, tmB128, a, dev, pairs, false, stream);
  }
  a.idesc = idesc_base(bf16, true, false);
  if (!make_mn_map(&tmA, &a.a_4d, 2, w.p, bf16, w.cols, w.rows, w.mats, wl, ws2)) return OZ_ECUDA;
  return launch<kRaggedN, true, false, 1>(tmA, tmB, tmB128, a, dev, pairs, false, stream);
}

int run_allocating(const Problem& p, cudaStream_t stream) {
  const size_t bytes = p.workspace();
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
