// step.h -- host/device interface between the C ABI (api.cu) and the operators of the training step
// around the heads (embed.cu, clip.cu, linear.cu).  Not part of the public boundary.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "smem_optin.h"

namespace dspark {

// Scratch that the calls of a context share.
constexpr int64_t kStepScratchBytes = 32 << 20;

// ---- embedding rows and their gradient (embed.cu)
struct EmbedArgs {
  const void* table;  // [V, D] of table_dtype, rows ld_table apart
  const int32_t* ids; // [N]
  int64_t N, ld_table, ld_out;
  int V, D, table_dtype, out_dtype;
  float scale;
  void* out;          // [N, D] of out_dtype, rows ld_out apart
  int* status;
};
cudaError_t launch_embed(const EmbedArgs& a, int* launches, cudaStream_t stream);

constexpr int64_t kEmbedGradMaxRows = 1 << 20;  // of one call
struct EmbedGradArgs {
  const int32_t* ids;  // [N]
  const void* de;      // [N, D] of de_dtype, rows ld_de apart
  int64_t N, ld_de, ld_grad;
  int V, D, de_dtype, grad_dtype;
  float scale;
  bool accumulate;
  void* grad;          // [V, D] of grad_dtype, rows ld_grad apart
  int* status;
};
constexpr int kEmbedGradMaxWidth = 1 << 16;  // of D: 256 slices of columns
struct EmbedGradLaunch {
  uint8_t* scratch;  // [kStepScratchBytes]
  int num_sms;
  SmemOptIn* opt_in;
  int* launches;     // host: kernels launched (added to)
};
cudaError_t launch_embed_grad(const EmbedGradArgs& a, const EmbedGradLaunch& c, cudaStream_t stream);

// ---- global norm and clipping (clip.cu)
constexpr int kClipMaxTensors = 512;  // of one launch
struct ClipArgs {
  const void* const* in;  // host [count]
  void* const* out;       // host [count], or null: only the norm
  const int64_t* numel;   // host [count]
  const int32_t* dtypes;  // host [count]
  int count;
  float max_norm;
  float* norm;            // device scalar
  double* partial;        // context scratch: [clip_partials(num_sms)]
  int num_sms;
};
constexpr int clip_partials(int num_sms) { return 4 * num_sms; }
cudaError_t launch_clip(const ClipArgs& a, int* launches, cudaStream_t stream);

// ---- products with an epilogue (linear.cu)
constexpr int kLinearMaxWidth = 1 << 22;  // of K and N: a row of column sums fits half the scratch
struct LinearArgs {
  const uint16_t *x, *W;    // [M, K], [K, N] bf16
  const float* bias;        // [N] or null
  const void* residual;     // [M, N] or null
  int64_t M, ld_x, ld_w, ld_res, ld_y, ld_pre;
  int K, N, act, res_dtype, y_dtype;
  void* y;                  // [M, N] of y_dtype
  void* pre;                // [M, N] of y_dtype, or null
};
struct LinearGradArgs {
  const uint16_t *x, *W;
  const void *dy, *pre;     // [M, N] of dy_dtype; of pre_dtype (null: no activation)
  int64_t M, ld_x, ld_w, ld_dy, ld_pre, ld_dx, ld_dw;
  int K, N, act, dy_dtype, pre_dtype, dx_dtype, dw_dtype;
  void *dx, *dW;            // [M, K], [K, N]; each may be null
  float* dbias;             // [N] or null
};
// What a context gives its launches.
struct LinearLaunch {
  float* scratch;     // [kStepScratchBytes]
  int num_sms;
  int* status;
  uint64_t timeout_ns;
  int debug_skip_cta; // testing: the block of each product that loads nothing (-1: none)
  SmemOptIn* opt_in;
  int* launches;      // host: kernels launched (added to)
};
// Bytes that a call needs of its caller.
int64_t linear_workspace(const LinearArgs& a);
int64_t linear_grad_workspace(const LinearGradArgs& a);
cudaError_t launch_linear(const LinearArgs& a, const LinearLaunch& c, void* workspace, cudaStream_t stream);
cudaError_t launch_linear_grad(const LinearGradArgs& a, const LinearLaunch& c, void* workspace,
                               cudaStream_t stream);

}  // namespace dspark
