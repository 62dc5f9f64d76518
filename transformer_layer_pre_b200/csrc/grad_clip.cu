// grad_clip.cu — global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over every tensor of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// Two launches.  The first gives every block a fixed set of chunks of the
// listed tensors and leaves one float64 sum of squares per block; the second
// sums those in block order (every block the same few kilobytes, so no third
// launch and no atomics: the result is bitwise reproducible), derives the
// factor and scales the tensors, its chunks in reverse order so that the ones
// the norm read last still come from L2.  When nothing is clipped in place
// the second launch ends after the sum.
//
// Squares are float64: a float32 square overflows from |g| = 1.8e19 and
// vanishes below 1e-23, and the conversions and FP64 FMAs (one each per value)
// stay below the rate at which HBM delivers float32 values.  16-bit values come
// twice as fast, and there the conversions begin to count: 302 M values, the norm
// alone 206 us of float32 (5.9 TB/s) and 120 us of 16 bits (5.0 TB/s).
// Bound: HBM; the norm has to be known before anything is scaled, so what
// exceeds L2 is read twice and written once.  24 layers of hidden 1024 (302 M
// float32, 2.42 GB read and written once): 608 us, three passes at 5.97 TB/s,
// 0.91 of the measured copy rate; the same number of 16-bit values 312 us, 5.8
// TB/s.  108 odd bf16 tensors, 98 MB, out of place: 27 us
// on the device (the norm's read from HBM, the scaling's from L2), and the 108 tensors' checks and addresses 45 us on the host.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>
#include <memory>
#include <new>
#include <utility>

#include "../../include/tlp.h"
#include "kernels.h"
#include "profile.h"

namespace tlp {
namespace {

constexpr int kClipThreads = 512;
constexpr int kClipUnroll = 4;                       // 16-byte loads in flight per thread
constexpr int kClipMaxBlocks = 148 * 4;              // four blocks of 512 threads per SM
constexpr int kClipChunkBytes = kClipThreads * kClipUnroll * 16;   // 32 KB: one round of a block

struct ClipTensor {
  const void* in;
  void* out;
  uint64_t n;          // elements
  uint64_t chunk0;     // chunks of the tensors before it
};
// Kernel parameters hold the list (32,764 bytes at most); a longer one runs
// as several launches.  Small lists use a small parameter block: the launch
// copies it whole.
template <int CAP>
struct ClipList {
  ClipTensor t[CAP];
  uint64_t chunks;
  int count;
};

// The tensor that chunk c belongs to (block-uniform binary search).
template <int CAP>
__device__ __forceinline__ int find_tensor(const ClipList<CAP>& l, uint64_t c) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.t[mid].chunk0 <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Chunk c of a tensor: elements [begin, end), cut where addresses of `in`
// are 16-byte aligned (the tensor's ragged head joins its first chunk).
template <typename T>
__device__ __forceinline__ void chunk_range(const ClipTensor& t, uint64_t c, uint64_t& begin, uint64_t& end) {
  constexpr uint64_t per = kClipChunkBytes / sizeof(T);
  const uint64_t head = ((16 - (reinterpret_cast<uintptr_t>(t.in) & 15)) & 15) / sizeof(T);
  const uint64_t k = c - t.chunk0;
  begin = k == 0 ? 0 : head + k * per;
  end = head + (k + 1) * per;
  if (end > t.n) end = t.n;
}

__device__ __forceinline__ double block_sum_f64(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kClipThreads / 32; ++w) s += red[w];
  return s;
}

template <typename T>
__device__ __forceinline__ double square_sum16(const uint4& r) {
  const T* h = reinterpret_cast<const T*>(&r);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) {
    const double x = (double)to_f(h[i]);
    s = fma(x, x, s);
  }
  return s;
}

template <typename T, int CAP>
__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const __grid_constant__ ClipList<CAP> l, double* part) {
  __shared__ double red[kClipThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  double acc = 0.0;
  for (uint64_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const ClipTensor& t = l.t[find_tensor(l, c)];
    uint64_t b, e;
    chunk_range<T>(t, c, b, e);
    const T* p = static_cast<const T*>(t.in);
    // ragged head (first chunk of an unaligned tensor) and tail, one value per thread
    const uint64_t head = ((16 - (reinterpret_cast<uintptr_t>(p + b) & 15)) & 15) / sizeof(T);
    const uint64_t vb = b + head < e ? b + head : e;
    const uint64_t vecs = (e - vb) / (16 / sizeof(T));
    const uint64_t te = vb + vecs * (16 / sizeof(T));
    const uint4* v = reinterpret_cast<const uint4*>(p + vb);
    uint4 r[kClipUnroll];
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) {
      const uint64_t i = threadIdx.x + u * kClipThreads;
      r[u] = i < vecs ? v[i] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) acc += square_sum16<T>(r[u]);
    if (b + threadIdx.x < vb) {
      const double x = (double)to_f(p[b + threadIdx.x]);
      acc = fma(x, x, acc);
    }
    if (te + threadIdx.x < e) {
      const double x = (double)to_f(p[te + threadIdx.x]);
      acc = fma(x, x, acc);
    }
  }
  const double s = block_sum_f64(acc, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ uint4 scale16(const uint4& r, float f) {
  uint4 o;
  const T* h = reinterpret_cast<const T*>(&r);
  T* q = reinterpret_cast<T*>(&o);
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) q[i] = from_f<T>(to_f(h[i]) * f);
  return o;
}

template <typename T, int CAP>
__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipList<CAP> l, const double* part, int nparts, double max_norm,
                      float* norm_out, int in_place) {
  __shared__ double red[kClipThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  double acc = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kClipThreads) acc += part[i];
  const double norm = sqrt(block_sum_f64(acc, red));
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out) *norm_out = (float)norm;
  const double ratio = max_norm / (norm + 1e-6);
  // NaN stays NaN; without a limit there is nothing to scale, whatever the norm
  const float f = ratio > 1.0 || max_norm == INFINITY ? 1.0f : (float)ratio;
  if (in_place && f == 1.0f) return;
  for (uint64_t k = blockIdx.x; k < l.chunks; k += gridDim.x) {
    const uint64_t c = l.chunks - 1 - k;
    const ClipTensor& t = l.t[find_tensor(l, c)];
    uint64_t b, e;
    chunk_range<T>(t, c, b, e);
    const T* p = static_cast<const T*>(t.in);
    T* o = static_cast<T*>(t.out);
    if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) {
      // input and output aligned differently: value by value
      for (uint64_t i = b + threadIdx.x; i < e; i += kClipThreads) o[i] = from_f<T>(to_f(p[i]) * f);
      continue;
    }
    const uint64_t head = ((16 - (reinterpret_cast<uintptr_t>(p + b) & 15)) & 15) / sizeof(T);
    const uint64_t vb = b + head < e ? b + head : e;
    const uint64_t vecs = (e - vb) / (16 / sizeof(T));
    const uint64_t te = vb + vecs * (16 / sizeof(T));
    const uint4* v = reinterpret_cast<const uint4*>(p + vb);
    uint4* w = reinterpret_cast<uint4*>(o + vb);
    uint4 r[kClipUnroll];
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) {
      const uint64_t i = threadIdx.x + u * kClipThreads;
      if (i < vecs) r[u] = v[i];
    }
#pragma unroll
    for (int u = 0; u < kClipUnroll; ++u) {
      const uint64_t i = threadIdx.x + u * kClipThreads;
      if (i < vecs) w[i] = scale16<T>(r[u], f);
    }
    if (b + threadIdx.x < vb) o[b + threadIdx.x] = from_f<T>(to_f(p[b + threadIdx.x]) * f);
    if (te + threadIdx.x < e) o[te + threadIdx.x] = from_f<T>(to_f(p[te + threadIdx.x]) * f);
  }
}

size_t elem_size(int dt) { return dt == DT_F32 ? 4 : 2; }

// Fills l with tensors [first, ...) of the call; returns the first one left out.
template <int CAP>
int fill(ClipList<CAP>& l, int dt, int count, const void* const* in, void* const* out, const uint64_t* n, int first) {
  const uint64_t es = elem_size(dt), per = kClipChunkBytes / es;
  l.count = 0;
  l.chunks = 0;
  int i = first;
  for (; i < count && l.count < CAP; ++i) {
    if (n[i] == 0) continue;
    const uint64_t head = ((16 - (reinterpret_cast<uintptr_t>(in[i]) & 15)) & 15) / es;
    l.t[l.count++] = {in[i], out[i], n[i], l.chunks};
    l.chunks += n[i] > head ? (n[i] - head + per - 1) / per : 1;
  }
  return i;
}

int grid_of(uint64_t chunks) { return (int)std::min<uint64_t>(std::max<uint64_t>(chunks, 1), kClipMaxBlocks); }

template <typename T, int CAP>
void run(int dt, int count, const void* const* in, void* const* out, const uint64_t* n, double max_norm, float* norm,
         int in_place, double* ws, cudaStream_t s) {
  ClipList<CAP> l;
  int parts = 0;
  for (int i = 0; i < count || parts == 0;) {
    i = fill<CAP>(l, dt, count, in, out, n, i);
    const int grid = grid_of(l.chunks);
    launch_pdl(clip_norm_kernel<T, CAP>, grid, kClipThreads, 0, s, l, ws + parts);
    count_launch();
    parts += grid;
  }
  bool first = true;
  for (int i = 0; i < count || first;) {
    i = fill<CAP>(l, dt, count, in, out, n, i);
    launch_pdl(clip_scale_kernel<T, CAP>, grid_of(l.chunks), kClipThreads, 0, s, l, (const double*)ws, parts, max_norm,
               first ? norm : nullptr, in_place);
    count_launch();
    first = false;
  }
}

constexpr int kCapSmall = 24, kCapMid = 320, kCapLarge = 1000;
static_assert(sizeof(ClipList<kCapLarge>) + 64 <= 32764, "the tensor list exceeds the kernel parameter space");

template <typename T>
void run_t(int dt, int count, const void* const* in, void* const* out, const uint64_t* n, double max_norm, float* norm,
           int in_place, double* ws, cudaStream_t s) {
  if (count <= kCapSmall) run<T, kCapSmall>(dt, count, in, out, n, max_norm, norm, in_place, ws, s);
  else if (count <= kCapMid) run<T, kCapMid>(dt, count, in, out, n, max_norm, norm, in_place, ws, s);
  else run<T, kCapLarge>(dt, count, in, out, n, max_norm, norm, in_place, ws, s);
}

// Whether no output shares memory with another tensor of the call (its own
// input at the same address apart).
bool separate(int count, const void* const* in, void* const* out, const uint64_t* n, uint64_t es) {
  using Range = std::pair<uintptr_t, uintptr_t>;
  constexpr int kStack = 256;
  Range few[kStack];
  std::unique_ptr<Range[]> many(count > kStack ? new (std::nothrow) Range[count] : nullptr);
  if (count > kStack && !many) return false;
  Range* r = many ? many.get() : few;
  int m = 0;
  bool sorted = true;
  for (int i = 0; i < count; ++i) {
    if (n[i] == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(out[i]);
    r[m] = {p, p + n[i] * es};
    sorted = sorted && (m == 0 || r[m - 1].first <= p);
    ++m;
  }
  if (!sorted) std::sort(r, r + m);
  for (int i = 1; i < m; ++i)
    if (r[i].first < r[i - 1].second) return false;
  for (int i = 0; i < count; ++i) {
    if (n[i] == 0 || in[i] == out[i]) continue;
    const uintptr_t b = reinterpret_cast<uintptr_t>(in[i]), e = b + n[i] * es;
    // the outputs are in order and apart: the first that ends behind the input's start
    const Range* x = std::upper_bound(r, r + m, b, [](uintptr_t at, const Range& y) { return at < y.second; });
    if (x != r + m && x->first < e) return false;
  }
  return true;
}

}  // namespace
}  // namespace tlp

using namespace tlp;

extern "C" {

size_t tl_clip_workspace_bytes(int count) {
  if (count < 0) return 0;
  return (size_t)((count + kCapLarge - 1) / kCapLarge + 1) * kClipMaxBlocks * sizeof(double);
}

tl_status tl_clip_grad_norm(int dtype, int count, const void* const* in, void* const* out, const uint64_t* n,
                            float max_norm, float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype < TL_F32 || dtype > TL_BF16 || count < 0 || !norm || !workspace) return TL_EINVAL;
  if (count > 0 && (!in || !out || !n)) return TL_EINVAL;
  if (!(max_norm >= 0.0f)) return TL_EINVAL;
  if (workspace_bytes < tl_clip_workspace_bytes(count) || (reinterpret_cast<uintptr_t>(workspace) & 7)) return TL_EINVAL;
  if (reinterpret_cast<uintptr_t>(norm) & 3) return TL_EINVAL;
  const uint64_t es = elem_size(dtype);
  int in_place = 1;
  for (int i = 0; i < count; ++i) {
    if (n[i] == 0) continue;
    if (!in[i] || !out[i] || n[i] > (1ull << 48)) return TL_EINVAL;
    if ((reinterpret_cast<uintptr_t>(in[i]) | reinterpret_cast<uintptr_t>(out[i])) & (es - 1)) return TL_EINVAL;
    if (in[i] != out[i]) in_place = 0;
  }
  if (!separate(count, in, out, n, es)) return TL_EINVAL;
  if (cudaPeekAtLastError() != cudaSuccess) {
    cudaGetLastError();
    return TL_ECUDA;
  }
  cudaStream_t s = (cudaStream_t)stream;
  ProfScope p_(PC_ROWWISE, s);
  double* ws = static_cast<double*>(workspace);
  if (dtype == TL_F32) run_t<float>(dtype, count, in, out, n, max_norm, norm, in_place, ws, s);
  else if (dtype == TL_F16) run_t<half_t>(dtype, count, in, out, n, max_norm, norm, in_place, ws, s);
  else run_t<bf16_t>(dtype, count, in, out, n, max_norm, norm, in_place, ws, s);
  return cudaGetLastError() == cudaSuccess ? TL_OK : TL_ECUDA;
}

}  // extern "C"
