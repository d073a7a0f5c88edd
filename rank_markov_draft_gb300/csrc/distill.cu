// distill.cu -- distillation of the draft head from a teacher's top logits: the loss of each
// row and its gradient with respect to the student's logits.
//
// Source: DSpark explainer, "How DSpark is trained" (cross entropy and total variation against
// the target's distribution, weights 0.1 and 0.9, position weights exp(-(k - 1) / gamma)).
// The events are the teacher's k tokens and "the rest":
//   p_i = (1 - rho) softmax(t / T)_i, p_rest = rho;  q = softmax(s / T), q_rest = sum outside
//   KL = sum_i p_i ln(p_i / q_i) + rho ln(rho / q_rest)
//   TV = (sum_i |p_i - q_i| + |rho - q_rest|) / 2,   loss = w (a_kl KL + a_tv TV)
// With S = sum_i sgn(q_i - p_i) q_i + sgn(q_rest - rho) q_rest, the derivative by logit v is
//   teacher's token i:  w / T [a_kl (q_i - p_i) + a_tv / 2 (sgn_i - S) q_i]
//   any other token:    w / T o_v [a_kl (q_rest - rho) + a_tv / 2 (sgn_rest - S) q_rest]
// with o the softmax over the other tokens alone.  The outside sum is taken without the
// teacher's tokens rather than as 1 - sum_i q_i, which cancels when the student agrees.

#include <cstdint>
#include <cuda_bf16.h>

#include "internal.h"
#include "sm103.cuh"

namespace dspark {
namespace {

constexpr int kDtThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) {
  return __uint_as_float(static_cast<uint32_t>(x) << 16);
}
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// The larger of two values, NaN if either is (so that a row of NaN is not taken for a masked one).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Block-wide maximum or sum; every thread gets the result (two barriers).
template <bool kMax>
__device__ float block_reduce(float x, float* sm) {
  for (int off = 16; off > 0; off >>= 1) {
    const float y = __shfl_xor_sync(0xFFFFFFFFu, x, off);
    x = kMax ? max_nan(x, y) : x + y;
  }
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sm[0];
  for (int w = 1; w < kDtThreads / 32; ++w) x = kMax ? max_nan(x, sm[w]) : x + sm[w];
  __syncthreads();
  return x;
}

// The sign of q_i - p_i where 32 bits cannot tell: the two sides in 64 bits.
__device__ __noinline__ float sign64(double qi, double pi) {
  return qi > pi ? 1.f : (qi < pi ? -1.f : 0.f);
}

template <typename T>
__global__ void __launch_bounds__(kDtThreads) distill_kernel(const DistillArgs a) {
  const int64_t n = blockIdx.x;
  const int tid = threadIdx.x, V = a.V, k = a.k;
  const T* row = static_cast<const T*>(a.logits) + n * a.ld;
  T* grad = a.grad != nullptr ? static_cast<T*>(a.grad) + n * a.ld_grad : nullptr;
  const float c = kLog2e / a.temperature;
  __shared__ int s_id[kMaxTeacher];
  __shared__ float s_g[kMaxTeacher], s_red[kDtThreads / 32];
  const float w = a.row_weight != nullptr ? __ldg(a.row_weight + n) : 1.f;
  // the teacher's slot of this thread
  int id = -1;
  float t = -INFINITY, s = -INFINITY;
  if (w != 0.f) {
    if (tid < k) {
      id = __ldg(a.teacher_ids + n * k + tid);
      if (id >= V) {
        record_error(a.status, kStatusDeviceOob);
        id = -1;
      }
      s_id[tid] = id;
    }
    __syncthreads();
    for (int i = 0; i < tid && tid < k; ++i)
      if (s_id[i] == id) id = -1;  // a repeated token's first slot counts
    __syncthreads();
    if (tid < k) s_id[tid] = id;
    if (id >= 0) {
      t = __ldg(a.teacher_logits + n * k + tid);
      s = to_f32(row[id]);
    }
    __syncthreads();
  }
  auto listed = [&](int v) {
    for (int i = 0; i < k; ++i)
      if (s_id[i] == v) return true;
    return false;
  };
  float m_out = -INFINITY;
  if (w != 0.f)
    for (int v = tid; v < V; v += kDtThreads)
      if (!listed(v)) m_out = max_nan(m_out, to_f32(row[v]));
  m_out = block_reduce<true>(m_out, s_red);
  const float t_top = block_reduce<true>(t, s_red);
  const float top = max_nan(m_out, block_reduce<true>(s, s_red));
  if (w == 0.f || t_top == -INFINITY || top == -INFINITY) {
    if (tid == 0) {
      a.loss[n] = 0.f;
      if (a.tv != nullptr) a.tv[n] = 0.f;
    }
    if (grad != nullptr)
      for (int v = tid; v < V; v += kDtThreads) put(grad + v, 0.f);
    return;
  }
  float sum = 0.f;
  for (int v = tid; v < V; v += kDtThreads) {
    const float x = to_f32(row[v]);
    if (x != -INFINITY && !listed(v)) sum += exp2f((x - m_out) * c);
  }
  const float sum_out = block_reduce<false>(sum, s_red);
  const float yi = id >= 0 ? (s - top) * c : -INFINITY;
  const float xi = id >= 0 ? (t - t_top) * c : -INFINITY;
  const float scale_out = m_out == -INFINITY ? 0.f : exp2f((m_out - top) * c);
  const float total = block_reduce<false>(exp2f(yi), s_red) + sum_out * scale_out;
  const float sum_t = block_reduce<false>(exp2f(xi), s_red);
  const float rho = a.teacher_rest != nullptr ? fminf(fmaxf(__ldg(a.teacher_rest + n), 0.f), 1.f)
                                              : 0.f;
  const float q = exp2f(yi) / total, q_rest = sum_out * scale_out / total;
  const float p = exp2f(xi) / sum_t * (1.f - rho);
  const float sgn_r = q_rest > rho ? 1.f : (q_rest < rho ? -1.f : 0.f);
  float sgn = q > p ? 1.f : (q < p ? -1.f : 0.f);
  if (id >= 0 && fabsf(q - p) < 1e-5f * p)
    sgn = sign64(exp((static_cast<double>(s) - top) / a.temperature) / total,
                 exp((static_cast<double>(t) - t_top) / a.temperature) / sum_t * (1.0 - rho));
  if (id < 0) sgn = 0.f;
  const float S = block_reduce<false>(sgn * q, s_red) + sgn_r * q_rest;
  const float kl_i = p > 0.f ? p * ((xi - yi) + (log2f(total) - log2f(sum_t)) + log2f(1.f - rho))
                             : 0.f;
  float kl = block_reduce<false>(kl_i, s_red) * kLn2;
  const float tv = 0.5f * (block_reduce<false>(fabsf(p - q), s_red) + fabsf(rho - q_rest));
  if (rho > 0.f)
    kl += rho * kLn2 *
          (log2f(rho) - (log2f(sum_out) + (m_out - top) * c) + log2f(total));
  if (tid == 0) {
    a.loss[n] = w * ((a.alpha_kl != 0.f ? a.alpha_kl * kl : 0.f) + a.alpha_tv * tv);
    if (a.tv != nullptr) a.tv[n] = tv;
  }
  if (grad == nullptr) return;
  const float wt = w / a.temperature;
  const float out = wt * (a.alpha_kl * (q_rest - rho) + 0.5f * a.alpha_tv * (sgn_r - S) * q_rest) /
                    sum_out;
  if (tid < k) s_g[tid] = wt * (a.alpha_kl * (q - p) + 0.5f * a.alpha_tv * (sgn - S) * q);
  __syncthreads();
  for (int v = tid; v < V; v += kDtThreads) {
    const float x = to_f32(row[v]);
    float g = x == -INFINITY ? 0.f : out * exp2f((x - m_out) * c);
    for (int i = 0; i < k; ++i)
      if (s_id[i] == v) g = s_g[i];
    put(grad + v, g);
  }
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
  const unsigned rows = static_cast<unsigned>(a.N);
  if (a.dtype == DSPARK_F32)
    distill_kernel<float><<<rows, kDtThreads, 0, stream>>>(a);
  else
    distill_kernel<uint16_t><<<rows, kDtThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dspark
