// linear.cu -- y = act(x W + bias) + residual, and the gradients of x, W and the bias.
//
// The heads' projections (h Wa, h Wg) and calibrated logits (U + s W2), forward and backward.

#include <algorithm>

#include "dspark.h"
#include "step.h"
#include "typed.cuh"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

__device__ float act_value(int act, float z) {
  switch (act) {
    case DSPARK_ACT_SIGMOID: return 1.f / (1.f + expf(-z));
    case DSPARK_ACT_TANH: return tanhf(z);
    case DSPARK_ACT_RELU: return z < 0.f ? 0.f : z;
    case DSPARK_ACT_SILU: return z / (1.f + expf(-z));
    case DSPARK_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678f));
    default: return z;
  }
}

__device__ float act_slope(int act, float z) {
  switch (act) {
    case DSPARK_ACT_SIGMOID: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f - s);
    }
    case DSPARK_ACT_TANH: {
      const float t = tanhf(z);
      return 1.f - t * t;
    }
    case DSPARK_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case DSPARK_ACT_SILU: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + z * (1.f - s));
    }
    case DSPARK_ACT_GELU:
      return 0.5f * (1.f + erff(z * 0.70710678f)) + z * expf(-0.5f * z * z) * 0.39894228f;
    default: return 1.f;
  }
}

__device__ __forceinline__ float load_as(const void* p, int dtype, int64_t i) {
  return dtype == DSPARK_F32 ? static_cast<const float*>(p)[i]
                             : __bfloat162float(static_cast<const bf16*>(p)[i]);
}
__device__ __forceinline__ void store_as(void* p, int dtype, int64_t i, float v) {
  if (dtype == DSPARK_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<bf16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float slope_times(const LinearGradArgs& a, int64_t m, int64_t n) {
  const float dy = load_as(a.dy, a.dy_dtype, m * a.ld_dy + n);
  return a.act == DSPARK_ACT_NONE
             ? dy
             : dy * act_slope(a.act, load_as(a.pre, a.pre_dtype, m * a.ld_pre + n));
}

// A 64 x 64 tile of sum_k A(i, k) B(k, j), 16 elements a thread.
constexpr int kTile = 64, kDeep = 16;
template <typename FA, typename FB, typename FO>
__device__ __forceinline__ void tile_product(int64_t I, int64_t J, int64_t Kc, FA A, FB B, FO out) {
  __shared__ float sa[kDeep][kTile + 1], sb[kDeep][kTile + 1];
  const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kTile, j0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < Kc; k0 += kDeep) {
    for (int e = threadIdx.x; e < kDeep * kTile; e += 256) {
      const int k = e / kTile, r = e % kTile;
      sa[k][r] = k0 + k < Kc && i0 + r < I ? A(i0 + r, k0 + k) : 0.f;
      sb[k][r] = k0 + k < Kc && j0 + r < J ? B(k0 + k, j0 + r) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = i0 + ty * 4 + i, c = j0 + tx + 16 * j;
      if (r < I && c < J) out(r, c, acc[i][j]);
    }
}

__global__ void __launch_bounds__(256) linear_kernel(LinearArgs a) {
  const bf16 *x = reinterpret_cast<const bf16*>(a.x), *W = reinterpret_cast<const bf16*>(a.W);
  tile_product(
      a.M, a.N, a.K, [&](int64_t m, int64_t k) { return load1(x + m * a.ld_x + k); },
      [&](int64_t k, int64_t n) { return load1(W + k * a.ld_w + n); },
      [&](int64_t m, int64_t n, float z) {
        if (a.bias != nullptr) z += a.bias[n];
        if (a.pre != nullptr) store_as(a.pre, a.y_dtype, m * a.ld_pre + n, z);
        z = act_value(a.act, z);
        if (a.residual != nullptr) z += load_as(a.residual, a.res_dtype, m * a.ld_res + n);
        store_as(a.y, a.y_dtype, m * a.ld_y + n, z);
      });
}

__global__ void __launch_bounds__(256) linear_dx_kernel(LinearGradArgs a) {
  const bf16* W = reinterpret_cast<const bf16*>(a.W);
  tile_product(
      a.M, a.K, a.N, [&](int64_t m, int64_t n) { return slope_times(a, m, n); },
      [&](int64_t n, int64_t k) { return load1(W + k * a.ld_w + n); },
      [&](int64_t m, int64_t k, float v) { store_as(a.dx, a.dx_dtype, m * a.ld_dx + k, v); });
}

__global__ void __launch_bounds__(256) linear_dw_kernel(LinearGradArgs a) {
  const bf16* x = reinterpret_cast<const bf16*>(a.x);
  tile_product(
      a.K, a.N, a.M, [&](int64_t k, int64_t m) { return load1(x + m * a.ld_x + k); },
      [&](int64_t m, int64_t n) { return slope_times(a, m, n); },
      [&](int64_t k, int64_t n, float v) { store_as(a.dW, a.dw_dtype, k * a.ld_dw + n, v); });
}

__global__ void __launch_bounds__(256) linear_dbias_kernel(LinearGradArgs a) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  float s = 0.f;
  for (int64_t m = 0; m < a.M; ++m) s += slope_times(a, m, n);
  a.dbias[n] = s;
}

dim3 tiles(int64_t I, int64_t J) {
  return dim3(static_cast<unsigned>((J + kTile - 1) / kTile), static_cast<unsigned>((I + kTile - 1) / kTile));
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, int* launches, cudaStream_t stream) {
  if (a.M == 0) return cudaSuccess;
  linear_kernel<<<tiles(a.M, a.N), 256, 0, stream>>>(a);
  *launches += 1;
  return cudaGetLastError();
}

cudaError_t launch_linear_grad(const LinearGradArgs& a, int* launches, cudaStream_t stream) {
  if (a.dx != nullptr && a.M > 0) {
    linear_dx_kernel<<<tiles(a.M, a.K), 256, 0, stream>>>(a);
    *launches += 1;
  }
  if (a.dW != nullptr) {
    linear_dw_kernel<<<tiles(a.K, a.N), 256, 0, stream>>>(a);
    *launches += 1;
  }
  if (a.dbias != nullptr) {
    linear_dbias_kernel<<<(a.N + 255) / 256, 256, 0, stream>>>(a);
    *launches += 1;
  }
  return cudaGetLastError();
}

}  // namespace dspark
