// rnn_scan.cu -- the RNN head's gated linear recurrence over given sequences, and its
// gradients.
//
// Source: DSpark explainer, "The RNN head"; the equations are this library's reading (as for
// the RNN draft):  a = sigmoid(za), g = sigmoid(zg) (1 where zg is absent),
//   s_t = a_t s_{t-1} + g_t e_t                         (channel by channel)
// and backwards, with ds the gradient of the states used outside the recurrence,
//   delta_t = ds_t + a_{t+1} delta_{t+1}  (delta_{L-1} = ds_{L-1} + ds_last)
//   dza_t = delta_t s_{t-1} a_t (1 - a_t),  dzg_t = delta_t e_t g_t (1 - g_t)
//   de_t = delta_t g_t,  ds0 = a_0 delta_0.
// A reset at t makes a_t zero.  A decay of exactly zero drops the earlier state, whatever it
// holds (an infinity or NaN before a reset stays before it).

#include <cstdint>
#include <cuda_bf16.h>

#include "internal.h"
#include "sm103.cuh"

namespace dspark {
namespace {

constexpr int kRsThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) {
  return __uint_as_float(static_cast<uint32_t>(x) << 16);
}
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// sigmoid(z) and 1 - sigmoid(z), each to full relative precision
__device__ __forceinline__ void gate(float z, float& a, float& rest) {
  const float t = exp2f(-z * kLog2e);
  a = 1.f / (1.f + t);
  rest = t <= 1.f ? t * a : 1.f - a;
}

template <typename T>
__global__ void __launch_bounds__(kRsThreads) rnn_scan_kernel(const RnnScanArgs p) {
  const int64_t lane = static_cast<int64_t>(blockIdx.x) * kRsThreads + threadIdx.x;
  if (lane >= p.N * p.D) return;
  const int64_t n = lane / p.D;
  const int d = static_cast<int>(lane - n * p.D);
  float s = p.s0 != nullptr ? p.s0[lane] : 0.f;
  for (int64_t t = 0; t < p.L; ++t) {
    const int64_t r = n * p.L + t;
    float a, g = 1.f, rest;
    gate(to_f32(static_cast<const T*>(p.za)[r * p.ld_za + d]), a, rest);
    if (p.zg != nullptr) gate(to_f32(static_cast<const T*>(p.zg)[r * p.ld_zg + d]), g, rest);
    if (p.reset != nullptr && p.reset[r] != 0) a = 0.f;
    const float b = g * to_f32(static_cast<const T*>(p.e)[r * p.ld_e + d]);
    s = a == 0.f ? b : fmaf(a, s, b);
    put(static_cast<T*>(p.s) + r * p.D + d, s);
  }
  if (p.s_last != nullptr) p.s_last[lane] = s;
}

template <typename T>
__global__ void __launch_bounds__(kRsThreads) rnn_scan_grad_kernel(const RnnScanGradArgs p) {
  const int64_t lane = static_cast<int64_t>(blockIdx.x) * kRsThreads + threadIdx.x;
  if (lane >= p.N * p.D) return;
  const int64_t n = lane / p.D;
  const int d = static_cast<int>(lane - n * p.D);
  float delta = p.ds_last != nullptr ? p.ds_last[lane] : 0.f;
  for (int64_t t = p.L - 1; t >= 0; --t) {
    const int64_t r = n * p.L + t;
    float a, na, g = 1.f, ng = 0.f;
    gate(to_f32(static_cast<const T*>(p.za)[r * p.ld_za + d]), a, na);
    if (p.zg != nullptr) gate(to_f32(static_cast<const T*>(p.zg)[r * p.ld_zg + d]), g, ng);
    if (p.reset != nullptr && p.reset[r] != 0) a = 0.f;
    const float e = to_f32(static_cast<const T*>(p.e)[r * p.ld_e + d]);
    float prev = 0.f;
    if (t > 0)
      prev = to_f32(static_cast<const T*>(p.s)[(r - 1) * p.D + d]);
    else if (p.s0 != nullptr)
      prev = p.s0[lane];
    delta += to_f32(static_cast<const T*>(p.ds)[r * p.D + d]);
    put(static_cast<T*>(p.dza) + r * p.ld_dza + d, a == 0.f ? 0.f : delta * prev * a * na);
    if (p.dzg != nullptr) put(static_cast<T*>(p.dzg) + r * p.ld_dzg + d, delta * e * g * ng);
    put(static_cast<T*>(p.de) + r * p.D + d, delta * g);
    delta = a == 0.f ? 0.f : a * delta;
  }
  if (p.ds0 != nullptr) p.ds0[lane] = delta;
}

}  // namespace

cudaError_t launch_rnn_scan(const RnnScanArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((a.N * a.D + kRsThreads - 1) / kRsThreads);
  if (a.dtype == DSPARK_F32)
    rnn_scan_kernel<float><<<grid, kRsThreads, 0, stream>>>(a);
  else
    rnn_scan_kernel<uint16_t><<<grid, kRsThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_rnn_scan_grad(const RnnScanGradArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((a.N * a.D + kRsThreads - 1) / kRsThreads);
  if (a.dtype == DSPARK_F32)
    rnn_scan_grad_kernel<float><<<grid, kRsThreads, 0, stream>>>(a);
  else
    rnn_scan_grad_kernel<uint16_t><<<grid, kRsThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dspark
