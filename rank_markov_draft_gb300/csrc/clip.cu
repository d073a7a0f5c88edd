// clip.cu -- the norm of many tensors together, and their scaling down to a limit:
//   norm = sqrt(sum g^2), out = g min(1, max_norm / (norm + 1e-6)).
//
// Two launches: the blocks' sums of squares, then the scaling, each of whose blocks adds those sums
// again in their order (no atomics, so equal inputs give equal bits; a few KB from L2). The tensors'
// addresses are launch arguments, so a captured graph holds them and nothing is copied.
//
// DRAM bounds it: 320 MB are read twice and written once in 157 us (6.1 TB/s), 36 MB that L2 holds in
// 26. Each block takes an equal stretch of all tensors, in straight loops of four vectors a thread, and
// goes back over it from its end (chunks two ahead with a search for each one's tensor took 167 us,
// L2 hints for what is read last 188).

#include <algorithm>
#include <type_traits>

#include "dependent.h"
#include "dspark.h"
#include "sm103.cuh"
#include "step.h"
#include "typed.cuh"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256, kBlocks = 4;  // of an SM
constexpr int kChunk = 8 * kThreads;        // elements, eight a thread: the grain of the blocks' stretches
constexpr int kAhead = 4;                   // vectors under way a thread
constexpr int kAdds = 32;                   // squares that a thread adds up in 32 bits

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

// f(t, first, n) for each tensor in this block's equal stretch of all chunks: n elements from `first`.
template <bool DOWN, int CAP, typename F>
__device__ __forceinline__ void for_stretch(const ClipList<CAP>& l, F f) {
  const int64_t chunks = l.first[l.count];
  const int64_t begin = chunks * blockIdx.x / gridDim.x, end = chunks * (blockIdx.x + 1) / gridDim.x;
  if (begin >= end) return;
  const int64_t from = DOWN ? end - 1 : begin;
  int lo = 0, hi = l.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    (l.first[mid] <= from ? lo : hi) = mid;
  }
  for (int t = lo; t >= 0 && t < l.count; t += DOWN ? -1 : 1) {
    const int64_t c0 = max(begin, l.first[t]), c1 = min(end, l.first[t + 1]);
    if (c0 >= c1) {
      if (DOWN ? l.first[t + 1] <= begin : l.first[t] >= end) break;
      continue;  // (a tensor of no elements)
    }
    const int64_t first = (c0 - l.first[t]) * kChunk;
    f(t, first, min(l.numel[t], (c1 - l.first[t]) * kChunk) - first);
  }
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

// A thread's sum of squares: of 32 bits for kAdds of them in each of eight sums, of 64 beyond.
struct Squares {
  double total = 0.0;
  float s[8] = {};
  int adds = 0;

  __device__ __forceinline__ void fold() {
    total += static_cast<double>(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.f;
    adds = 0;
  }
  template <typename T>
  __device__ __forceinline__ void add(const T* p, int64_t n, bool wide) {
    int64_t i = 8 * static_cast<int>(threadIdx.x);
    if (wide) {
      for (; i + (kAhead - 1) * kChunk + 8 <= n; i += kAhead * kChunk) {
        Raw8<T> r[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) r[k].load(p + i + k * kChunk);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          float v[8];
          r[k].get(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] = fmaf(v[j], v[j], s[j]);
        }
        if ((adds += kAhead) > kAdds - kAhead) fold();
      }
      for (; i + 8 <= n; i += kChunk) {
        Raw8<T> r;
        float v[8];
        r.load(p + i);
        r.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = fmaf(v[j], v[j], s[j]);
        if (++adds > kAdds - kAhead) fold();
      }
    }
    for (; i < n; i += kChunk) {  // the last few, or rows that allow no vectors
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < n) s[j] = fmaf(load1(p + i + j), load1(p + i + j), s[j]);
      if (++adds > kAdds - kAhead) fold();
    }
  }
};

template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocks)
    clip_squares_kernel(const __grid_constant__ ClipList<CAP> l, double* partial, bool add) {
  griddep_launch_dependents();
  Squares q;
  for_stretch<false>(l, [&](int t, int64_t first, int64_t n) {
    if (l.bf16_in[t])
      q.add(static_cast<const bf16*>(l.in[t]) + first, n, l.wide[t]);
    else
      q.add(static_cast<const float*>(l.in[t]) + first, n, l.wide[t]);
  });
  q.fold();
  const double total = block_sum(q.total);
  if (threadIdx.x == 0) partial[blockIdx.x] = total + (add ? partial[blockIdx.x] : 0.0);
}

__device__ __forceinline__ double norm_of(const double* partial, int parts) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += partial[i];
  return sqrt(block_sum(v));
}

__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const double* partial, int parts, float* norm) {
  griddep_wait();
  const double v = norm_of(partial, parts);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

// out = c in, from the end.
template <typename T>
__device__ __forceinline__ void scale_down(const T* in, T* out, int64_t n, bool wide, float c) {
  int64_t i = (n - 1) / kChunk * kChunk + 8 * static_cast<int>(threadIdx.x);
  auto slow = [&]() {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) store1(out + i + j, load1(in + i + j) * c);
  };
  if (!wide) {
    for (; i >= 0; i -= kChunk) slow();
    return;
  }
  if (i + 8 > n) {
    slow();
    i -= kChunk;
  }
  auto vectors = [&](auto count) {
    constexpr int kCount = decltype(count)::value;
    Raw8<T> r[kCount];
#pragma unroll
    for (int k = 0; k < kCount; ++k) r[k].load(in + i - k * kChunk);
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      float v[8];
      r[k].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= c;
      store8(out + i - k * kChunk, v);
    }
    i -= kCount * kChunk;
  };
  while (i >= (kAhead - 1) * kChunk) vectors(std::integral_constant<int, kAhead>());
  while (i >= 0) vectors(std::integral_constant<int, 1>());
}

// From the end of each block's stretch: what was read last is still in L2.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kBlocks)
    clip_scale_kernel(const __grid_constant__ ClipList<CAP> l, const double* partial, int parts,
                      float max_norm, float* norm) {
  griddep_wait();
  const double total = norm_of(partial, parts);
  double coef = static_cast<double>(max_norm) / (total + 1e-6);
  if (coef > 1.0) coef = 1.0;  // (a NaN stays one)
  const float c = static_cast<float>(coef);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  for_stretch<true>(l, [&](int t, int64_t first, int64_t n) {
    if (c == 1.f && l.in[t] == l.out[t]) return;
    if (l.bf16_in[t])
      scale_down(static_cast<const bf16*>(l.in[t]) + first, static_cast<bf16*>(l.out[t]) + first, n, l.wide[t], c);
    else
      scale_down(static_cast<const float*>(l.in[t]) + first, static_cast<float*>(l.out[t]) + first, n, l.wide[t], c);
  });
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
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.out == nullptr) {
    e = launch_kernel({dim3(1), kThreads}, stream, clip_norm_kernel, a.partial, parts, a.norm);
    if (e == cudaSuccess) *launches += 1;
    return e;
  }
  t0 = 0;
  do {
    const int n = std::min(CAP, a.count - t0);
    if (a.count > CAP) fill(l, a, t0, n);
    e = launch_kernel({dim3(parts), kThreads}, stream, clip_scale_kernel<CAP>, l, a.partial, parts, a.max_norm,
                      t0 == 0 ? a.norm : nullptr);
    if (e != cudaSuccess) return e;
    *launches += 1;
    t0 += n;
  } while (t0 < a.count);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_clip(const ClipArgs& a, int* launches, cudaStream_t stream) {
  // a short list makes short launch arguments (2 KB instead of 17)
  return a.count <= 64 ? clip<64>(a, launches, stream) : clip<kClipMaxTensors>(a, launches, stream);
}

}  // namespace dspark
