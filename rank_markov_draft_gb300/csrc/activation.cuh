// activation.cuh -- the linear layers' activations and their slopes, in fp32 by CUDA's functions.
#pragma once

#include <type_traits>

#include "dspark.h"

namespace dspark {

// 1 / (1 + e^-z) without cancellation or overflow, right to four units in the last place (the
// exponential to one, the quick division of numbers up to 2 by ones of 1 to 2 to two).
__device__ __forceinline__ float sigmoid_of(float z) {
  const float e = expf(-fabsf(z));
  return __fdividef(z < 0.f ? e : 1.f, 1.f + e);
}
// The same by the quick exponential, right to 2 + 1.2 |z| units in the last place of e^-z (which counts where
// z < 0; elsewhere 1 is the larger summand), and 0 below 2^-126: for outputs of bf16, of whose steps that is
// less than a three-hundredth. (1825 x 256 x 35840 with sigmoid to bf16 takes 80 us; with expf 99.)
__device__ __forceinline__ float quick_sigmoid_of(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

template <int ACT, bool QUICK>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == DSPARK_ACT_SIGMOID) return QUICK ? quick_sigmoid_of(z) : sigmoid_of(z);
  if constexpr (ACT == DSPARK_ACT_TANH) return tanhf(z);
  if constexpr (ACT == DSPARK_ACT_RELU) return z < 0.f ? 0.f : z;  // (a NaN stays one)
  if constexpr (ACT == DSPARK_ACT_SILU) return QUICK ? __fdividef(z, 1.f + __expf(-z)) : z * sigmoid_of(z);
  if constexpr (ACT == DSPARK_ACT_GELU) return 0.5f * z * erfcf(z * -0.70710678f);
  return z;
}

// Slopes without a difference from 1, of which saturated arguments would leave nothing: s (1 - s) is
// e / (1 + e)^2 with e = e^-|z|, and 1 - tanh^2 four times that of 2 z. Both are right to five units in the last place.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == DSPARK_ACT_SIGMOID) {
    const float e = expf(-fabsf(z)), d = 1.f + e;
    return __fdividef(e, d * d);
  }
  if constexpr (ACT == DSPARK_ACT_TANH) {
    const float e = expf(-2.f * fabsf(z)), d = 1.f + e;
    return __fdividef(4.f * e, d * d);
  }
  if constexpr (ACT == DSPARK_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == DSPARK_ACT_SILU) {  // s (1 + z (1 - s))
    const float e = expf(-fabsf(z)), large = __fdividef(1.f, 1.f + e), small = e * large;
    return (z < 0.f ? small : large) * fmaf(z, z < 0.f ? large : small, 1.f);
  }
  if constexpr (ACT == DSPARK_ACT_GELU)
    return 0.5f * erfcf(z * -0.70710678f) + z * expf(-0.5f * z * z) * 0.39894228f;
  return 1.f;
}

// f with the activation as a constant: one branch for many elements.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case DSPARK_ACT_SIGMOID: f(std::integral_constant<int, DSPARK_ACT_SIGMOID>()); break;
    case DSPARK_ACT_TANH: f(std::integral_constant<int, DSPARK_ACT_TANH>()); break;
    case DSPARK_ACT_RELU: f(std::integral_constant<int, DSPARK_ACT_RELU>()); break;
    case DSPARK_ACT_SILU: f(std::integral_constant<int, DSPARK_ACT_SILU>()); break;
    case DSPARK_ACT_GELU: f(std::integral_constant<int, DSPARK_ACT_GELU>()); break;
    default: break;
  }
}

}  // namespace dspark
