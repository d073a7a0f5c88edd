// clip.cu -- the norm of many tensors together, and their scaling down to a limit:
//   norm = sqrt(sum g^2), out = g min(1, max_norm / (norm + 1e-6)).
//
// Two launches: the blocks' sums of squares, then the scaling, each of whose blocks adds those sums
// again in their order (no atomics, so equal inputs give equal bits; a few KB from L2).  The
// tensors' addresses are launch arguments, so a captured graph holds them and nothing is copied.

#include <algorithm>

#include "dspark.h"
#include "step.h"
#include "typed.cuh"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 512;
constexpr int kChunk = 16384;  // elements of one tensor that a block takes at a time

// The tensors of one launch.
template <int CAP>
struct ClipList {
  const void* in[CAP];
  void* out[CAP];
  int64_t numel[CAP];
  int64_t first[CAP + 1];  // chunks before each tensor
  uint8_t bf16_in[CAP], wide[CAP];  // its type; both addresses allow vectors of eight
  int count;
};

// The tensor that chunk c lies in.
template <int CAP>
__device__ __forceinline__ int tensor_of(const ClipList<CAP>& l, int64_t c) {
  int lo = 0, hi = l.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    (l.first[mid] <= c ? lo : hi) = mid;
  }
  return lo;
}

// Sum over the block, on every thread.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double warps[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += warps[i];
  return s;
}

template <typename T>
__device__ __forceinline__ void add_squares(const T* p, int n, bool wide, float (&s)[8]) {
  if (wide) {
    const int n8 = n / 8;
#pragma unroll 4
    for (int i = threadIdx.x; i < n8; i += kThreads) {
      Raw8<T> r;
      float v[8];
      r.load(p + 8 * i);
      r.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = fmaf(v[j], v[j], s[j]);
    }
    const int i = n8 * 8 + threadIdx.x;
    if (i < n) s[0] = fmaf(load1(p + i), load1(p + i), s[0]);
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float v = load1(p + i);
      s[0] = fmaf(v, v, s[0]);
    }
  }
}

// The sums are of 32 bits within a thread (eight of them, a few dozen squares each and chunk) and of
// 64 beyond.
template <int CAP>
__global__ void __launch_bounds__(kThreads)
    clip_squares_kernel(const __grid_constant__ ClipList<CAP> l, double* partial, bool add) {
  double total = 0.0;
  for (int64_t c = blockIdx.x; c < l.first[l.count]; c += gridDim.x) {
    const int t = tensor_of(l, c);
    const int64_t at = (c - l.first[t]) * kChunk;
    const int n = static_cast<int>(min(static_cast<int64_t>(kChunk), l.numel[t] - at));
    float s[8] = {};
    if (l.bf16_in[t])
      add_squares(static_cast<const bf16*>(l.in[t]) + at, n, l.wide[t], s);
    else
      add_squares(static_cast<const float*>(l.in[t]) + at, n, l.wide[t], s);
    total += static_cast<double>(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
  }
  total = block_sum(total);
  if (threadIdx.x == 0) partial[blockIdx.x] = total + (add ? partial[blockIdx.x] : 0.0);
}

__device__ __forceinline__ double norm_of(const double* partial, int parts) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += partial[i];
  return sqrt(block_sum(v));
}

__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const double* partial, int parts, float* norm) {
  const double v = norm_of(partial, parts);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* p, T* q, int n, bool wide, float c) {
  if (wide) {
    const int n8 = n / 8;
#pragma unroll 4
    for (int i = threadIdx.x; i < n8; i += kThreads) {
      Raw8<T> r;
      float v[8];
      r.load(p + 8 * i);
      r.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= c;
      store8(q + 8 * i, v);
    }
    const int i = n8 * 8 + threadIdx.x;
    if (i < n) store1(q + i, load1(p + i) * c);
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) store1(q + i, load1(p + i) * c);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    clip_scale_kernel(const __grid_constant__ ClipList<CAP> l, const double* partial, int parts,
                      float max_norm, float* norm) {
  const double total = norm_of(partial, parts);
  double coef = static_cast<double>(max_norm) / (total + 1e-6);
  if (coef > 1.0) coef = 1.0;  // (a NaN stays one)
  const float c = static_cast<float>(coef);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  const int64_t chunks = l.first[l.count];
  // from the end: what was read last is still in L2
  for (int64_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const int64_t at_chunk = chunks - 1 - k;
    const int t = tensor_of(l, at_chunk);
    if (c == 1.f && l.in[t] == l.out[t]) continue;
    const int64_t at = (at_chunk - l.first[t]) * kChunk;
    const int n = static_cast<int>(min(static_cast<int64_t>(kChunk), l.numel[t] - at));
    if (l.bf16_in[t])
      scale_chunk(static_cast<const bf16*>(l.in[t]) + at, static_cast<bf16*>(l.out[t]) + at, n,
                  l.wide[t], c);
    else
      scale_chunk(static_cast<const float*>(l.in[t]) + at, static_cast<float*>(l.out[t]) + at, n,
                  l.wide[t], c);
  }
}

template <int CAP>
void fill(ClipList<CAP>& l, const ClipArgs& a, int t0, int n) {
  l.count = n;
  l.first[0] = 0;
  for (int i = 0; i < n; ++i) {
    l.in[i] = a.in[t0 + i];
    l.out[i] = a.out != nullptr ? a.out[t0 + i] : nullptr;
    l.numel[i] = a.numel[t0 + i];
    l.first[i + 1] = l.first[i] + (a.numel[t0 + i] + kChunk - 1) / kChunk;
    l.bf16_in[i] = a.dtypes[t0 + i] == DSPARK_BF16;
    l.wide[i] = rows_of_8(l.in[i], 0, a.dtypes[t0 + i]) && rows_of_8(l.out[i], 0, a.dtypes[t0 + i]);
  }
}

template <int CAP>
cudaError_t clip(const ClipArgs& a, int* launches, cudaStream_t stream) {
  const int parts = clip_partials(a.num_sms);
  ClipList<CAP> l;
  int t0 = 0;
  do {  // (no tensors: sums of nothing)
    const int n = std::min(CAP, a.count - t0);
    fill(l, a, t0, n);
    clip_squares_kernel<CAP><<<parts, kThreads, 0, stream>>>(l, a.partial, t0 > 0);
    *launches += 1;
    t0 += n;
  } while (t0 < a.count);
  if (a.out == nullptr) {
    clip_norm_kernel<<<1, kThreads, 0, stream>>>(a.partial, parts, a.norm);
    *launches += 1;
    return cudaGetLastError();
  }
  t0 = 0;
  do {
    const int n = std::min(CAP, a.count - t0);
    if (a.count > CAP) fill(l, a, t0, n);
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(parts, l.first[n]));
    clip_scale_kernel<CAP><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
        l, a.partial, parts, a.max_norm, t0 == 0 ? a.norm : nullptr);
    *launches += 1;
    t0 += n;
  } while (t0 < a.count);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_clip(const ClipArgs& a, int* launches, cudaStream_t stream) {
  // a short list makes short launch arguments (2 KB instead of 17)
  return a.count <= 64 ? clip<64>(a, launches, stream) : clip<kClipMaxTensors>(a, launches, stream);
}

}  // namespace dspark
