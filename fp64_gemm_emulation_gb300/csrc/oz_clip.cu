// oz_clip.cu -- the 2-norm over many tensors, and each of them times min(1, limit / (norm + eps)).
//
// Bound by memory: the tensors are read for the norm, and read again and written where that is below 1 or
// the results go elsewhere.  The tensors of a launch are in its parameters (no copy to the device), cut into
// chunks of equal length that CTAs take in turn.  Each CTA's sum of squares is a double at a place of its
// own, and every CTA of the second launch adds them all in the same order (at most 32 KB from the L2): the norm
// does not depend on timing, and there is no counter to be zeroed first.  The second launch goes through
// the chunks backwards: the first it meets are the last that were read, still in the L2.
// Measured: 6e8 bfloat16 values in 160 tensors 565 us, two readings and a writing at 6.4 TB/s.
//
// Squares: 32 elements at a time in FP32 where the largest of them is between 2^-50 and 2^55 (what the others
// then lose below 2^-126 is under 2^-26 of the sum), otherwise in FP64; the running sum is FP64 throughout.
#include <algorithm>
#include <utility>
#include <vector>

#include "oz_elements.cuh"
#include "oz_device.cuh"

namespace oz {
namespace {

constexpr int kThreads = 256, kResident = 5;  // CTAs of an SM: no more are launched, so that all get equally many chunks
// Elements of a chunk: enough for a CTA's 16-byte loads to follow each other, few enough for all CTAs to get some.
constexpr int kChunk = 16384, kLongChunk = 32768;
constexpr long long kLongTotal = 1ll << 27;    // elements of a launch from which on chunks are long
constexpr int kMaxSums = 4096;                 // CTAs whose sums the workspace holds

struct Tensor {
  const void* in;
  void* out;
  long long count;
  long long first;  // chunks before it in this launch
  int dtype, aligned;
};

template <int N>
struct ClipParams {
  Tensor t[N];
  int tensors;
  int first_sum, all_sums;  // where this launch's sums start; how many there are
  int chunk;                // elements
  long long chunks;
  double* sums;
  float limit, eps;
  float* norm;
};

template <class P>
__device__ __forceinline__ int tensor_of(const P& a, long long chunk) {
  int lo = 0, hi = a.tensors;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.t[mid].first <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// The squares of the eights v[0 .. N - 1].
template <class T, int N>
__device__ __forceinline__ double squares(const Eight<T> (&v)[N]) {
  float most = 0.0f, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = v[i].get(e);
      most = fmaxf(most, fabsf(x));
      sum = fmaf(x, x, sum);
    }
  }
  // (a NaN is not in most, but in sum)
  if (most == 0.0f || (most >= 8.8817842e-16f && most <= 3.6028797e16f)) return static_cast<double>(sum);
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // (unrolled: an index known only at run time would put v into memory)
      const double x = v[i].get(e);
      d = fma(x, x, d);
    }
  }
  return d;
}

// Four eights of a chunk of `count` elements, from c + i STEP on; zeros behind its end.
constexpr int kEights = 4, STEP = kThreads * 8;
template <class T>
__device__ __forceinline__ void load_eights(Eight<T> (&v)[kEights], const T* p, int c, int count, bool aligned) {
#pragma unroll
  for (int i = 0; i < kEights; ++i) {
    const int at = c + i * STEP;
    v[i] = aligned && at + 8 <= count ? load_eight(p + at) : gather_eight(p + at, 1, [&](int e) { return at + e < count; });
  }
}

template <class T>
__device__ __forceinline__ double chunk_squares(const Tensor& t, long long from, int chunk) {
  const T* p = static_cast<const T*>(t.in) + from;
  const int count = static_cast<int>(min(static_cast<long long>(chunk), t.count - from));
  double d = 0.0;
  for (int c = 8 * threadIdx.x; c < count; c += kEights * STEP) {
    Eight<T> v[kEights];
    load_eights(v, p, c, count, t.aligned);
    d += squares(v);
  }
  return d;
}

__device__ __forceinline__ double block_sum(double d, double* meet) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, s);
  if ((threadIdx.x & 31) == 0) meet[threadIdx.x >> 5] = d;
  __syncthreads();
  d = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) d += meet[w];
  __syncthreads();
  return d;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kResident) sum_kernel(const __grid_constant__ ClipParams<N> a) {
  __shared__ double meet[kThreads / 32];
  let_next_start();
  wait_for_previous();
  double d = 0.0;
  for (long long chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    const Tensor& t = a.t[tensor_of(a, chunk)];
    const long long from = (chunk - t.first) * a.chunk;
    d += t.dtype == OZ_F32 ? chunk_squares<float>(t, from, a.chunk)
         : t.dtype == OZ_BF16 ? chunk_squares<__nv_bfloat16>(t, from, a.chunk)
                              : chunk_squares<__half>(t, from, a.chunk);
  }
  d = block_sum(d, meet);
  if (threadIdx.x == 0) a.sums[a.first_sum + blockIdx.x] = d;
}

template <class T>
__device__ __forceinline__ void scale_chunk(const Tensor& t, long long from, int chunk, float f) {
  const T* p = static_cast<const T*>(t.in) + from;
  T* q = static_cast<T*>(t.out) + from;
  const int count = static_cast<int>(min(static_cast<long long>(chunk), t.count - from));
  for (int c = 8 * threadIdx.x; c < count; c += kEights * STEP) {
    Eight<T> v[kEights];  // all loads before the first store, which could be to the same memory
    load_eights(v, p, c, count, t.aligned);
#pragma unroll
    for (int i = 0; i < kEights; ++i) {
      const int at = c + i * STEP;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v[i].get(e) * f;
      if (t.aligned && at + 8 <= count) {
        store_eight(q + at, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at + e < count) from_float(x[e], q[at + e]);
      }
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kResident) scale_kernel(const __grid_constant__ ClipParams<N> a) {
  __shared__ double meet[kThreads / 32];
  let_next_start();
  wait_for_previous();
  double all = 0.0;
  for (int i = threadIdx.x; i < a.all_sums; i += kThreads) all += __ldcg(a.sums + i);
  const float norm = static_cast<float>(sqrt(block_sum(all, meet)));
  float f = a.limit / (norm + a.eps);
  // A NaN stays, but for 0 / 0 and Inf / Inf.
  if (f > 1.0f || norm == 0.0f || (norm == a.limit && isinf(norm))) f = 1.0f;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
  for (long long i = blockIdx.x; i < a.chunks; i += gridDim.x) {
    const long long chunk = a.chunks - 1 - i;
    const Tensor& t = a.t[tensor_of(a, chunk)];
    if (f == 1.0f && t.in == t.out) continue;
    const long long from = (chunk - t.first) * a.chunk;
    if (t.dtype == OZ_F32) scale_chunk<float>(t, from, a.chunk, f);
    else if (t.dtype == OZ_BF16) scale_chunk<__nv_bfloat16>(t, from, a.chunk, f);
    else scale_chunk<__half>(t, from, a.chunk, f);
  }
}

// Tensors of a launch: its parameters hold them all (at most 32764 bytes).
constexpr int kFew = 64, kMany = 640;

struct Work {
  int count;
  const int* dtypes;
  const void* const* in;
  void* const* out;
  const long long* counts;
};

template <int N>
int clip_launches(const Work& w, float limit, float eps, float* norm, uint8_t* ws, int sms, cudaStream_t stream) {
  ClipParams<N> a;
  a.sums = reinterpret_cast<double*>(ws);
  a.norm = norm;
  a.limit = limit;
  a.eps = eps;
  const int launches = w.count ? (w.count + N - 1) / N : 1;
  const int most = kMaxSums / launches < kResident * sms ? kMaxSums / launches : kResident * sms;
  int sums = 0;
  auto fill = [&](int l) {
    a.tensors = 0;
    a.chunks = 0;
    long long total = 0;
    for (int i = l * N; i < w.count && i < (l + 1) * N; ++i) total += w.counts[i];
    a.chunk = total >= kLongTotal ? kLongChunk : kChunk;
    for (int i = l * N; i < w.count && i < (l + 1) * N; ++i) {
      if (w.counts[i] == 0) continue;
      Tensor& t = a.t[a.tensors++];
      t.in = w.in[i];
      t.out = w.out[i];
      t.count = w.counts[i];
      t.first = a.chunks;
      t.dtype = w.dtypes[i];
      t.aligned = ((reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out)) & 15) == 0;
      a.chunks += (t.count + a.chunk - 1) / a.chunk;
    }
    const long long grid = a.chunks < most ? a.chunks : most;
    return static_cast<unsigned>(grid < 1 ? 1 : grid);
  };
  for (int l = 0; l < launches; ++l) {
    const unsigned grid = fill(l);
    a.first_sum = sums;
    sums += static_cast<int>(grid);
    if (launch_overlapping(sum_kernel<N>, dim3(grid), kThreads, 0, stream, a) != cudaSuccess) return OZ_ECUDA;
  }
  a.all_sums = sums;
  for (int l = launches - 1; l >= 0; --l) {  // each of them writes the norm, the same one
    const unsigned grid = fill(l);
    if (launch_overlapping(scale_kernel<N>, dim3(grid), kThreads, 0, stream, a) != cudaSuccess) return OZ_ECUDA;
  }
  return OZ_OK;
}

constexpr size_t kClipBytes = sizeof(double) * kMaxSums;
constexpr int kMaxTensors = kMany * 64;

}  // namespace
}  // namespace oz

using namespace oz;

extern "C" {

size_t ozaki_clip_grad_norm_workspace_bytes(void) { return kClipBytes; }

static int clip_check(const Work& w, float limit, float eps, const float* norm) try {
  if (w.count < 0 || w.count > kMaxTensors || !(limit >= 0.0f) || !(eps >= 0.0f) || !norm || (reinterpret_cast<uintptr_t>(norm) & 3)) return OZ_EINVAL;
  if (w.count && (!w.dtypes || !w.in || !w.out || !w.counts)) return OZ_EINVAL;
  for (int i = 0; i < w.count; ++i) {
    if (!element_bytes(w.dtypes[i]) || w.counts[i] < 0) return OZ_EINVAL;
    if (w.counts[i] && (!w.in[i] || !w.out[i] || !element_aligned(w.in[i], w.dtypes[i]) || !element_aligned(w.out[i], w.dtypes[i]))) return OZ_EINVAL;
  }
  // No two outputs may meet: a tensor that is listed twice would be scaled once or twice, as it happens.
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;
  spans.reserve(w.count);
  for (int i = 0; i < w.count; ++i) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(w.out[i]);
    if (w.counts[i]) spans.emplace_back(at, at + element_bytes(w.dtypes[i]) * static_cast<uintptr_t>(w.counts[i]));
  }
  if (!std::is_sorted(spans.begin(), spans.end())) std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].first < spans[i - 1].second) return OZ_EINVAL;
  return OZ_OK;
} catch (...) {  // no host memory
  return OZ_ENOMEM;
}

static int clip_run(const Work& w, float limit, float eps, float* norm, void* workspace, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return OZ_ECUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return w.count <= kFew ? clip_launches<kFew>(w, limit, eps, norm, ws, sms, stream) : clip_launches<kMany>(w, limit, eps, norm, ws, sms, stream);
}

int ozaki_clip_grad_norm_ws(int count, const int* dtypes, const void* const* grads, void* const* outs, const long long* counts,
                            float max_norm, float eps, float* norm, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  const Work w{count, dtypes, grads, outs, counts};
  const int rc = clip_check(w, max_norm, eps, norm);
  if (rc) return rc;
  if (!workspace || ws_bytes < kClipBytes || (reinterpret_cast<uintptr_t>(workspace) & 255)) return OZ_ENOMEM;
  return clip_run(w, max_norm, eps, norm, workspace, stream);
}

int ozaki_clip_grad_norm(int count, const int* dtypes, const void* const* grads, void* const* outs, const long long* counts,
                         float max_norm, float eps, float* norm, cudaStream_t stream) {
  const Work w{count, dtypes, grads, outs, counts};
  int rc = clip_check(w, max_norm, eps, norm);
  if (rc) return rc;
  void* ws = nullptr;
  keep_default_pool_cached();
  if (cudaMallocAsync(&ws, kClipBytes, stream) != cudaSuccess) {
    cudaGetLastError();
    return OZ_ENOMEM;
  }
  rc = clip_run(w, max_norm, eps, norm, ws, stream);
  if (cudaFreeAsync(ws, stream) != cudaSuccess && rc == OZ_OK) rc = OZ_ECUDA;
  return rc;
}

}  // extern "C"
