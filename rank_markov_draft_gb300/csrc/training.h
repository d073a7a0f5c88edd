// training.h -- host/device interface between the C ABI (api.cu) and the training and verification
// operators (verify_probs.cu, distill.cu, rnn_scan.cu).  Not part of the public boundary.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "smem_optin.h"

namespace dspark {

// ---- verification from given probabilities and random numbers (verify_probs.cu)
struct VerifyProbsArgs {
  const float* P;           // [B, K+1, V]
  const float* Q;           // [B, K, V] (m = 0)
  const int32_t* cand;      // [B, K, m] (m > 0)
  const float* cand_q;      // [B, K, m]
  const int32_t* tokens;    // [B, K]
  const float* u_accept;    // [B, K]
  const float* u_draw;      // [B]
  const int32_t* ell;       // [B] or null: K
  int m, B, K, V;
  int32_t* n_acc;           // [B]
  int32_t* next_token;      // [B]
  float* accept_prob;       // [B, K] or null
  int* status;
  float* sums;              // context scratch: [kVpMaxRequests][128 segments] x (hi, lo)
  int* count;               // [kVpMaxRequests] CTAs done, zero between calls
};
constexpr int kVpMaxRequests = 1024;  // of one launch
constexpr int kVpMaxCtas = 16;        // of a request
cudaError_t launch_verify_probs(const VerifyProbsArgs& a, SmemOptIn& opt_in, int* launches,
                                cudaStream_t stream);

// ---- distillation from a teacher's top logits (distill.cu)
constexpr int kMaxTeacher = 256;  // teacher tokens (and draft candidates) a row
constexpr int kLongMaxRows = 2048, kLongMaxSegments = 128;  // of one launch, of a row
struct LongScratch {               // rows of several segments
  unsigned long long* part;        // [kLongMaxRows][kLongMaxSegments][2] tagged maximum and sum
  unsigned long long* coef;        // [kLongMaxRows][3] tagged coefficient, maximum, any outside
  int2* list;                      // [kLongMaxRows][kMaxTeacher] tokens and their gradients
  uint32_t* epoch;                 // tag of the last launch
  uint32_t* done;                  // CTAs done, zero between launches (the last word)
};
constexpr size_t kLongScratchBytes =
    static_cast<size_t>(kLongMaxRows) * (kLongMaxSegments * 16 + 3 * 8 + kMaxTeacher * 8) + 8;
struct DistillArgs {
  const void* logits;           // [N, V] of dtype, rows ld apart
  const int32_t* teacher_ids;   // [N, k]
  const float* teacher_logits;  // [N, k]
  const float* teacher_rest;    // [N] or null: 0
  const float* row_weight;      // [N] or null: 1
  int64_t N, ld, ld_grad;
  int V, k, dtype;
  float temperature, alpha_kl, alpha_tv;
  float* loss;                  // [N]
  float* tv;                    // [N] or null
  void* grad;                   // [N, V] of dtype, rows ld_grad apart, or null
  int* status;
  uint64_t timeout_ns;
  int debug_skip_cta;           // long rows: the CTA that publishes no first sums (-1: none)
  LongScratch scratch;
};
// extra_smem: testing, beyond what a long row's launch may have
cudaError_t launch_distill(const DistillArgs& a, int num_sms, uint32_t extra_smem,
                           SmemOptIn& opt_in, int* launches, cudaStream_t stream);

// ---- the RNN head's recurrence over given sequences (rnn_scan.cu)
struct RnnScanArgs {
  const void *za, *zg, *e;   // [N, L, D] of dtype, rows ld_* apart; zg may be null
  int64_t ld_za, ld_zg, ld_e;
  const float* s0;           // [N, D] or null
  const uint8_t* reset;      // [N, L] or null
  int64_t N, L;
  int D, dtype;
  void* s;                   // [N, L, D]
  float* s_last;             // [N, D] or null
};
struct RnnScanGradArgs {
  const void *za, *zg, *e, *s, *ds;
  int64_t ld_za, ld_zg, ld_e, ld_dza, ld_dzg;
  const float* s0;
  const uint8_t* reset;
  const float* ds_last;      // [N, D] or null
  int64_t N, L;
  int D, dtype;
  void *dza, *dzg, *de;
  float* ds0;                // [N, D] or null
};
// A span of steps acts on the value before it as x -> A x + S.
struct ScanSpan {
  float A, S;
};
// Scratch of sequences cut into segments: for each CTA (two an SM) its span and the spans before
// each of its (at most 8) warps, of 64 channels each.
constexpr size_t scan_span_count(int num_sms) { return static_cast<size_t>(2 * num_sms) * 9 * 64; }
struct ScanLaunch {
  ScanSpan* spans;
  int num_sms;
  int* launches;      // host: kernels launched (added to)
  SmemOptIn* opt_in;  // host: the context's
  // set by the launch
  int64_t blocks;  // of 32 lanes
  int W;           // warps that walk a block together
  int segs, seg;   // segments a block, and their length in places
  uint32_t div_mul;  // q / D
  int div_shift;
  bool wide;       // rows start on 16-byte boundaries
};
cudaError_t launch_rnn_scan(const RnnScanArgs& a, const ScanLaunch& c, cudaStream_t stream);
cudaError_t launch_rnn_scan_grad(const RnnScanGradArgs& a, const ScanLaunch& c,
                                 cudaStream_t stream);

}  // namespace dspark
