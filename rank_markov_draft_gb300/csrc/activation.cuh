// activation.cuh -- the linear layers' activations and their slopes, in fp32 by CUDA's functions.
#pragma once

#include "dspark.h"

namespace dspark {

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case DSPARK_ACT_SIGMOID: return 1.f / (1.f + expf(-z));
    case DSPARK_ACT_TANH: return tanhf(z);
    case DSPARK_ACT_RELU: return z < 0.f ? 0.f : z;  // (a NaN stays one)
    case DSPARK_ACT_SILU: return z / (1.f + expf(-z));
    case DSPARK_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678f);
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(int act, float z) {
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
      return 0.5f * erfcf(z * -0.70710678f) + z * expf(-0.5f * z * z) * 0.39894228f;
    default: return 1.f;
  }
}

}  // namespace dspark
