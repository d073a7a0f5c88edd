// clip.cu -- the norm of many tensors together, and their scaling down to a limit:
//   norm = sqrt(sum g^2), out = g min(1, max_norm / (norm + 1e-6)).
//
// Two launches: the blocks' sums of squares, then the scaling, each of whose blocks adds those sums
// again in their order (no atomics, so equal inputs give equal bits; a few KB from L2).  The
// tensors' addresses are launch arguments, so a captured graph holds them and nothing is copied.

#include <algorithm>

#include "dependent.h"
#include "dspark.h"
#include "sm103.cuh"
#include "step.h"
#include "typed.cuh"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 512;
constexpr int kChunk = 8 * kThreads;  // elements of one tensor that a block takes at a time, eight a thread
constexpr int kAhead = 2;             // chunks under way a block
constexpr int kAdds = 32;             // squares that a thread adds up in 32 bits

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

// A block's chunks: an equal stretch of all of them, walked up or down.
template <int CAP>
struct Walk {
  const ClipList<CAP>& l;
  int64_t begin, end;
  int t;  // tensor of the chunk asked for last

  __device__ __forceinline__ explicit Walk(const ClipList<CAP>& list) : l(list) {
    const int64_t chunks = l.first[l.count];
    begin = chunks * blockIdx.x / gridDim.x;
    end = chunks * (blockIdx.x + 1) / gridDim.x;
    t = 0;
  }
  // to the tensor of chunk c
  __device__ __forceinline__ void find(int64_t c) {
    int lo = 0, hi = l.count;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      (l.first[mid] <= c ? lo : hi) = mid;
    }
    t = lo;
  }
  __device__ __forceinline__ void follow(int64_t c) {  // the same for a neighbour of the last
    while (l.first[t + 1] <= c) ++t;
    while (l.first[t] > c) --t;
  }
};

// This thread's part of a chunk.
struct Piece {
  Raw8<float> f;
  Raw8<bf16> h;
  int t, n;       // its tensor; elements (< 8: a tail or a tensor without vectors)
  int64_t at;     // the first
  float v[8];     // of those

  template <int CAP>
  __device__ __forceinline__ void load(Walk<CAP>& w, int64_t c) {
    n = 0;
    if (c < w.begin || c >= w.end) return;
    w.follow(c);
    t = w.t;
    const int64_t rest = w.l.numel[t] - (c - w.l.first[t]) * kChunk;
    at = (c - w.l.first[t]) * kChunk + 8 * threadIdx.x;
    const int64_t mine = rest - 8 * static_cast<int>(threadIdx.x);
    n = mine >= 8 ? 8 : (mine > 0 ? static_cast<int>(mine) : 0);
    if (n == 8 && w.l.wide[t]) {
      if (w.l.bf16_in[t])
        h.load(static_cast<const bf16*>(w.l.in[t]) + at);
      else
        f.load(static_cast<const float*>(w.l.in[t]) + at);
    }
  }
  template <int CAP>
  __device__ __forceinline__ void get(const Walk<CAP>& w) {
    const bool is_bf16 = w.l.bf16_in[t];
    if (n == 8 && w.l.wide[t]) {
      is_bf16 ? h.get(v) : f.get(v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = 0.f;
        if (j < n) v[j] = is_bf16 ? load1(static_cast<const bf16*>(w.l.in[t]) + at + j) : load1(static_cast<const float*>(w.l.in[t]) + at + j);
      }
    }
  }
  template <int CAP>
  __device__ __forceinline__ void put(const Walk<CAP>& w, float c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= c;
    const bool is_bf16 = w.l.bf16_in[t];
    if (n == 8 && w.l.wide[t]) {
      is_bf16 ? store8(static_cast<bf16*>(w.l.out[t]) + at, v) : store8(static_cast<float*>(w.l.out[t]) + at, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) is_bf16 ? store1(static_cast<bf16*>(w.l.out[t]) + at + j, v[j]) : store1(static_cast<float*>(w.l.out[t]) + at + j, v[j]);
    }
  }
};

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

template <int CAP>
__global__ void __launch_bounds__(kThreads, 2)
    clip_squares_kernel(const __grid_constant__ ClipList<CAP> l, double* partial, bool add) {
  griddep_launch_dependents();
  Walk<CAP> w(l);
  if (w.begin < w.end) w.find(w.begin);
  double total = 0.0;
  float s[8] = {};
  int adds = 0;
  auto fold = [&]() {
    total += static_cast<double>(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.f;
    adds = 0;
  };
  Piece p[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) p[k].load(w, w.begin + k);
  for (int64_t c = w.begin; c < w.end; c += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (p[k].n > 0) {
        p[k].get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = fmaf(p[k].v[j], p[k].v[j], s[j]);
      }
      p[k].load(w, c + kAhead + k);
    }
    if ((adds += kAhead) == kAdds) fold();
  }
  fold();
  total = block_sum(total);
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

// From the end of each block's stretch: what was read last is still in L2.
template <int CAP>
__global__ void __launch_bounds__(kThreads, 2)
    clip_scale_kernel(const __grid_constant__ ClipList<CAP> l, const double* partial, int parts,
                      float max_norm, float* norm) {
  Walk<CAP> w(l);
  if (w.begin < w.end) w.find(w.end - 1);
  griddep_wait();
  Piece p[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) p[k].load(w, w.end - 1 - k);
  const double total = norm_of(partial, parts);
  double coef = static_cast<double>(max_norm) / (total + 1e-6);
  if (coef > 1.0) coef = 1.0;  // (a NaN stays one)
  const float f = static_cast<float>(coef);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  for (int64_t c = w.end - 1; c >= w.begin; c -= kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (p[k].n > 0 && (f != 1.f || l.in[p[k].t] != l.out[p[k].t])) {
        p[k].get(w);
        p[k].put(w, f);
      }
      p[k].load(w, c - kAhead - k);
    }
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
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.out == nullptr) {
    e = launch_dependent(clip_norm_kernel, dim3(1), kThreads, stream, a.partial, parts, a.norm);
    if (e == cudaSuccess) *launches += 1;
    return e;
  }
  t0 = 0;
  do {
    const int n = std::min(CAP, a.count - t0);
    if (a.count > CAP) fill(l, a, t0, n);
    e = launch_dependent(clip_scale_kernel<CAP>, dim3(parts), kThreads, stream, l, a.partial, parts,
                         a.max_norm, t0 == 0 ? a.norm : nullptr);
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
