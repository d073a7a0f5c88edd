// internal.h -- host/device interface between the C ABI (api.cu) and the
// kernels.  Not part of the public boundary.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "dspark.h"
#include "smem_optin.h"

namespace dspark {

constexpr int kMaxK = 64;           // block positions per call
constexpr int kMaxRank = 256;       // Markov rank
constexpr int kBatchChunk = 128;    // requests per draft launch (MMA M)
constexpr int kDraftTileN = 128;    // vocabulary entries per draft MMA tile (MMA N)
constexpr int kDraftBoxV = 64;      // W2 TMA box width: one 128-byte swizzled row of bf16
constexpr int kDraftSliceRows = 128;  // W2 rows (the contraction dimension) per ring slot
// rows of one W2 box (and ring slot): the whole rank when it fits, else 128
inline int draft_slice_rows(int r) { return r < kDraftSliceRows ? r : kDraftSliceRows; }
constexpr int kMaxTopk = 32;
constexpr int kTopkPartUnits = 4096;  // per-piece top-k lists the context can hold
constexpr int kTraceSlots = 8;      // timestamps per (CTA, step) in the draft trace
constexpr uint64_t kDefaultTimeoutNs = 2000ull * 1000ull * 1000ull;  // 2 s per wait

// Per-(step, request, CTA) record of the draft kernel's cross-CTA reduction.
struct DraftPartial {
  unsigned long long key;  // (epoch, race score, token) packed, see draft.cu
  float m2;                // running max of l * log2(e) / T'
  float sum;               // sum of 2^(y - m2)
  float lbest;             // calibrated logit of this CTA's best token
  float pad;
};

// Per-request inputs of the draft kernel's residual mode (the verification draw).
struct ResRow {
  float offq2;  // log2 q(v) = l(v) * log2(e) / Td + offq2; -inf: no draft mass subtracted
  float offp2;  // log2 p(v) = P(v) * log2(e) / Tt + offp2
  int pos;      // draw position (noise counter)
  int excl;     // token whose weight is zero (a greedy draft's rejected token), or -1
};

struct DraftParams {
  const uint16_t* W1;       // [V, r]
  const int32_t* anchors;   // [B] (chunk)
  const int32_t* prev;      // teacher-forced predecessors [B, K] (chunk), or null
  const uint16_t* H;        // gated: [B, K, r] (chunk) bf16, or null (RNN head: input gate)
  const uint16_t* A;        // RNN head: decay gate [B, K, r] (chunk) bf16, or null
  int B, K, V, r;
  int b_global0;            // index of the chunk's first request in the call (noise key)
  int n_tiles;              // ceil(V / 128)
  int box_rows;             // rows of the U TMA box (multiple of 8, >= B)
  // U boxes of row pairs: the map views U as [B][K][V / 32][32] and a box holds 64 tokens
  // (two 32-token chunks) of up to 64 rows, each row's 256 bytes read contiguously (needs
  // V % 32 == 0); otherwise boxes of 32 tokens of every row
  int u_rowpair;
  float inv_t;              // 1 / T' (T' = T, or 1 when greedy)
  uint32_t seed_lo, seed_hi;
  uint32_t round_key0[10];  // Philox key schedule (seed_lo + i * Weyl0), host-computed
  uint32_t round_key1[10];  // (seed_hi + i * Weyl1)
  int32_t* tokens;          // [B, K] (chunk)
  float* logprobs;          // [B, K] (chunk)
  float* logits;            // teacher-forced: [B, K, V] (chunk)
  float* lse;               // teacher-forced: [B, K] (chunk)
  // fused confidence head (conf == null: off)
  const uint16_t* conf_h;   // [B, K, d] (chunk)
  const uint16_t* conf_w;   // [d (+ r)]
  float conf_bias;
  int conf_d;
  int conf_with_markov;
  float conf_threshold;
  const float* conf_tau;    // [K] STS temperatures, or null (all 1)
  float* conf;              // [B, K] (chunk)
  float* cumprod;           // [B, K] (chunk)
  int32_t* verify_len;      // [B] (chunk)
  // context scratch
  unsigned long long* keys; // [kMaxK][128]
  DraftPartial* partials;   // [kMaxK][128][grid]
  uint32_t* bar;            // grid-barrier counter
  int* status;              // device status word
  uint32_t bar_base;        // counter value at launch
  uint32_t epoch;           // key epoch of this launch (1 .. 16383)
  int debug_skip_cta;       // fault injection: CTA skipping its step-0 arrival (-1: none)
  unsigned long long* trace;  // optional phase timestamps [grid][K][kTraceSlots] (null: off)
  uint64_t timeout_ns;      // per-wait limit
  // acceptance-label mode (null otherwise)
  const float* target;      // [B, K+1, V] (chunk) target logits (read through tm_p)
  const float* lse_t;       // [B, K+1] (chunk) log sum_v exp(target / Tt)
  const float* offq2;       // [B, K] (chunk) log2 q(v) = l(v) * log2(e) / Td + offq2
  float* label;             // [B, K] (chunk) 1 - TV(q, p)
  float target_scale2;      // log2(e) / Tt
  // residual mode (verification draw, K = 1): per-row constants; the draw rows of the
  // caller's U [B, res_K, V] and P [B, res_K + 1, V] gathered in place through tm_u, tm_p
  const ResRow* rows;       // [B] (chunk), or null
  int res_K;
};

struct DraftArgs {
  CUtensorMap tm_w2;  // W2 [r, V] bf16, box {64, min(r, 128)}, 128B swizzle
  CUtensorMap tm_u;   // U chunk [B, K, V] fp32, box {32, 1, box_rows}, 128B swizzle (or
                      // row-pair boxes); residual mode: U as rows [B K, V], box {32, 1}
                      // (gathered by four)
  CUtensorMap tm_p;   // label mode: target chunk [B, K+1, V] fp32, box {32, 1, box_rows},
                      // 128B swizzle (or row-pair boxes); residual mode: P as rows
                      // [B (K + 1), V], box {32, 1}
  DraftParams p;
};

enum DraftMode {
  kModeSample = 0,
  kModeGreedy = 1,
  kModeTeacherForced = 2,
  kModeLabel = 3,
  kModeResidual = 4,  // one position: block race over max(0, p - q) (the verification draw)
};

int draft_smem_bytes();
int draft_threads(int mode, bool copies);
// extra_smem > 0 asks for that much more dynamic shared memory than the kernel allows, which
// the runtime refuses (the refused-launch test); the refusal's error is cleared before return
// dependent: launched as a programmatic dependent of the preceding kernel of the stream (which
// may then overlap the prologue; the kernel waits for it before reading any input), falling
// back to a plain cooperative launch where the runtime refuses the combination
cudaError_t launch_draft(const DraftArgs& args, int mode, int grid, cudaStream_t stream,
                         uint32_t extra_smem = 0, bool dependent = false);

// Gate GEMM: partial[split][m][n] = sum_{j in split} h[m, j] * Wg[j, n].
struct GateArgs {
  CUtensorMap tm_h;   // h [M, d] bf16, box {64, 128}
  CUtensorMap tm_wg;  // Wg [d, r] bf16, box {64, 64}
  float* partial;     // [splits][M][r]
  int M, d, r, splits, chunks_per_split;
  int* status;
  uint64_t timeout_ns;
};
cudaError_t launch_gate_gemm(const GateArgs& args, cudaStream_t stream);
cudaError_t launch_gate_finalize(const float* partial, int splits, int64_t n, float* H,
                                 uint16_t* Hb, cudaStream_t stream);

// Top-k of each row of U [rows][V] (V a multiple of 4).  part_i / part_v: scratch
// for up to part_units per-piece lists of kMaxTopk entries (null: whole rows
// only).  *launches receives the number of kernels launched.
cudaError_t launch_topk(const float* U, int rows, int V, int topk, int32_t* cand, float* cval,
                        int32_t* part_i, float* part_v, int part_units, int* status,
                        uint64_t timeout_ns, int* launches, cudaStream_t stream);
cudaError_t launch_pair_scores(const int32_t* cand, const float* cval, const uint16_t* A,
                               const uint16_t* Bt, const int32_t* anchors, const float* H,
                               int B, int K, int V, int r, int topk, float* S, int* status,
                               uint64_t timeout_ns, cudaStream_t stream);
cudaError_t launch_walk(const int32_t* cand, const float* S, const int32_t* anchors,
                        const uint16_t* A, int B, int K, int V, int r, int topk, float inv_t,
                        int sample, uint32_t seed_lo, uint32_t seed_hi, int32_t* tokens,
                        float* logprobs, const dspark_conf_args* conf, int* status,
                        cudaStream_t stream);
// ---- speculative verification (verify.cu)
struct VerifyArgs {
  const float* P;             // [B, K+1, V] target logits
  const float* U;             // [B, K, V] base logits of the draft
  const uint16_t* W1;         // [V, r]
  const uint16_t* W2;         // [r, V]
  const float* H;             // [B, K, r] gate (null: ungated)
  const int32_t* tokens;      // [B, K] drafted tokens
  const float* logq;          // [B, K] the draft's log-probabilities of them (draft T > 0)
  const int32_t* anchors;     // [B]
  const int32_t* ell;         // [B] verified positions (null: K)
  int B, K, V, r;
  float draft_temperature, target_temperature;
  uint32_t seed_lo, seed_hi;
  int32_t* n_acc;             // [B]
  int32_t* next_token;        // [B]
  float* accept_prob;         // [B, K] or null
  int* status;
  // context scratch
  float* lse_t;               // [B, K+1]
  int32_t* argmax_t;          // [B, K+1]
  // the draw (sampled target): the residual mode's per-row constants, predecessors and
  // gate rows at the draw position; rows null: no draw (a greedy target's token is its
  // argmax)
  uint16_t* H_sel;            // [B, r] bf16
  int32_t* prev_sel;          // [B]
  ResRow* rows;               // [B]
  // per-request scratch, zero between calls (the request's last CTA clears it)
  unsigned long long* fail_mask;  // [B] bit k: the test of position k failed
  int* count;                     // [B] CTAs of the request done
};
// One kernel: the target-row scan with the acceptance tests and the draw's per-row
// constants (the draft kernel's residual mode then reads the draw rows of U and P in place).
cudaError_t launch_verify(const VerifyArgs& v, cudaStream_t stream, int* launches);

// ---- acceptance label (label.cu)
// One warp per drafted position: its predecessor, the offset that turns the
// draft head's logits into log2 q (draft T > 0), and the label itself where one
// side is greedy (the other cases are summed by the draft kernel's label mode).
struct LabelPrepArgs {
  const float* P;             // [B, K+1, V]
  const float* U;             // [B, K, V]
  const uint16_t* W1;         // [V, r]
  const uint16_t* W2;         // [r, V]
  const float* H;             // [B, K, r] or null
  const int32_t* anchors;     // [B]
  const int32_t* tokens;      // [B, K]
  const float* logq;          // [B, K] (draft T > 0)
  float* lse_t;               // [B, K+1] out, rows k < K (target T > 0)
  int32_t* argmax_t;          // [B, K+1] out, rows k < K (target T = 0)
  int B, K, V, r;
  float inv_td, inv_tt;       // 0: greedy
  int32_t* prev;              // [B, K] out
  float* offq2;               // [B, K] out (draft T > 0)
  float* label;               // [B, K] out where one side is greedy
  int* status;
};
// One kernel: the scan of each drafted position's target row, then that row's
// preparation (predecessor, log2 q offset, the label where one side is greedy).
cudaError_t launch_label_prep(const LabelPrepArgs& a, cudaStream_t stream);

// ---- load-aware prefix scheduler (schedule.cu)
constexpr int kScheduleMaxCandidates = 16384;  // R * K
cudaError_t launch_schedule(const float* a, int R, int K, const float* sps, int32_t* ell,
                            float* theta, cudaStream_t stream);

cudaError_t launch_confidence(const uint16_t* h, const uint16_t* W1, const int32_t* anchors,
                              const int32_t* tokens, const uint16_t* w, float bias,
                              int with_markov, int B, int K, int d, int r, int V,
                              float threshold, const float* tau, float* conf, float* cumprod,
                              int32_t* verify_len, int* status, cudaStream_t stream);

// ---- sequential temperature scaling (calibrate.cu)
cudaError_t launch_sts_fit(const float* conf, const float* label, int N, int K, float tau_lo,
                           float tau_hi, float* tau, float* loss, cudaStream_t stream);

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
