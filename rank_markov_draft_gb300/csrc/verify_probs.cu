// verify_probs.cu -- verification of a drafted block against the target's probabilities,
// from random numbers the caller gives.
//
// Source: "DSpark: Repair the Joint, Meter the Verify", "Watch the Mass Land Wrong" (accept a
// drafted token with probability min(1, p/q), on a rejection the target resamples from what
// the draft left over); DSpark explainer, "Confidence-scheduled verification".
//
// Position k of the window survives while u_k q_k(x_k) < p_k(x_k), a product of two 24-bit
// numbers compared in 64 bits, so exactly.  At the first rejection j the weights are
// r_v = max(0, p_j(v) - q_j(v)), after a full window r = p_ell, and the token is the first v
// whose running sum of r passes u R, R the whole sum.  A vocabulary's sum in 32 bits is off by
// more than a rare token's probability, so a neighbour would be drawn; each difference is kept
// with its rounding error and summed as a pair of floats (hi + lo, about 2^-48 of the sum),
// partial sums are joined in 64 bits.

#include <cfloat>
#include <cstdint>

#include "internal.h"
#include "sm103.cuh"

namespace dspark {
namespace {

constexpr int kVpThreads = 256;
constexpr int kVpWarps = kVpThreads / 32;

// s + e = a + b exactly (Knuth's two-sum)
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = a + b;
  const float bb = s - a;
  e = (a - (s - bb)) + (b - bb);
}

struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(Pair x) {
    float s, e;
    two_sum(hi, x.hi, s, e);
    hi = s;
    lo += e + x.lo;
  }
  __device__ __forceinline__ double value() const {
    return static_cast<double>(hi) + static_cast<double>(lo);
  }
};

// max(0, p - q) with its rounding error; entries that are not finite have no mass
__device__ __forceinline__ Pair residual(float p, float q) {
  Pair r;
  two_sum(p, -q, r.hi, r.lo);
  if (!(r.hi > 0.f && r.hi <= FLT_MAX)) r = Pair{};
  return r;
}

// q of one token among m candidates (the first of equal ids counts, negative ids are empty)
__device__ __forceinline__ float candidate_q(const int32_t* ids, const float* q, int m, int v) {
  for (int i = 0; i < m; ++i)
    if (__ldg(ids + i) == v) return __ldg(q + i);
  return 0.f;
}

__global__ void __launch_bounds__(kVpThreads) verify_probs_kernel(const VerifyProbsArgs a) {
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int s_j, s_len;
  __shared__ double s_sum[kVpWarps];
  if (tid == 0) {
    s_len = a.ell == nullptr ? a.K : min(max(__ldg(a.ell + b), 0), a.K);
    s_j = s_len;
  }
  __syncthreads();
  const int len = s_len;
  if (tid < a.K) {
    const size_t o = static_cast<size_t>(b) * a.K + tid;
    float prob = -1.f;
    if (tid < len) {
      int x = __ldg(a.tokens + o);
      if (x < 0 || x >= a.V) {
        record_error(a.status, kStatusDeviceOob);
        x = 0;
      }
      const float p = __ldg(a.P + (static_cast<size_t>(b) * (a.K + 1) + tid) * a.V + x);
      const float q = a.m > 0 ? candidate_q(a.cand + o * a.m, a.cand_q + o * a.m, a.m, x)
                              : __ldg(a.Q + o * a.V + x);
      const bool ok = static_cast<double>(__ldg(a.u_accept + o)) * static_cast<double>(q) <
                      static_cast<double>(p);
      prob = q > 0.f ? fminf(1.f, p / q) : (p > 0.f ? 1.f : 0.f);
      if (!ok) atomicMin(&s_j, tid);
    }
    if (a.accept_prob != nullptr) a.accept_prob[o] = prob;
  }
  __syncthreads();
  const int j = s_j;
  const size_t o = static_cast<size_t>(b) * a.K + j;
  const float* prow = a.P + (static_cast<size_t>(b) * (a.K + 1) + j) * a.V;
  const float* qrow = a.m == 0 && j < len ? a.Q + o * a.V : nullptr;
  const int32_t* cid = a.m > 0 && j < len ? a.cand + o * a.m : nullptr;
  const int seg = ((a.V + kVpWarps - 1) / kVpWarps + 31) & ~31;
  const int v0 = min(a.V, warp * seg), v1 = min(a.V, v0 + seg);
  bool left = j < len;  // weights are what the draft left over (else the target's row)
  auto weight = [&](int v) {
    float q = 0.f;
    if (left) q = qrow != nullptr ? __ldg(qrow + v) : candidate_q(cid, a.cand_q + o * a.m, a.m, v);
    return residual(__ldg(prow + v), q);
  };
  double total;
  for (;;) {
    Pair acc;
    for (int v = v0 + lane; v < v1; v += 32) acc.add(weight(v));
    double s = acc.value();
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if (lane == 0) s_sum[warp] = s;
    __syncthreads();
    total = 0.0;
    for (int w = 0; w < kVpWarps; ++w) total += s_sum[w];
    if (total > 0.0 || !left) break;
    left = false;  // nothing left over: the target's own row
    __syncthreads();
  }
  if (tid == 0) a.n_acc[b] = j;
  if (!(total > 0.0)) {
    if (tid == 0) a.next_token[b] = -1;
    return;
  }
  const double want = static_cast<double>(__ldg(a.u_draw + b)) * total;
  int owner = -1;
  double before = 0.0, run = 0.0;
  for (int w = 0; w < kVpWarps; ++w) {
    if (s_sum[w] > 0.0 && (owner < 0 || run <= want)) {
      owner = w;
      before = run;
    }
    run += s_sum[w];
  }
  if (warp != owner) return;
  int found = -1;
  for (int v = v0; v < v1; v += 32) {
    double x = v + lane < v1 ? weight(v + lane).value() : 0.0;
    const bool mass = x > 0.0;
    for (int off = 1; off < 32; off <<= 1) {
      const double y = __shfl_up_sync(0xFFFFFFFFu, x, off);
      if (lane >= off) x += y;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, mass && before + x > want);
    const unsigned any = __ballot_sync(0xFFFFFFFFu, mass);
    if (hit) {
      found = v + __ffs(hit) - 1;
      break;
    }
    if (any) found = v + 31 - __clz(any);
    before += __shfl_sync(0xFFFFFFFFu, x, 31);
  }
  if (lane == 0) a.next_token[b] = found;
}

}  // namespace

cudaError_t launch_verify_probs(const VerifyProbsArgs& a, cudaStream_t stream) {
  verify_probs_kernel<<<a.B, kVpThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dspark
