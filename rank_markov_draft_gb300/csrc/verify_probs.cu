// verify_probs.cu -- verification of a drafted block against the target's probabilities,
// from random numbers the caller gives.
//
// Source: "DSpark: Repair the Joint, Meter the Verify", "Watch the Mass Land Wrong" (accept a
// drafted token with probability min(1, p/q), on a rejection the target resamples from what
// the draft left over); DSpark explainer, "Confidence-scheduled verification".
//
// Position k of the window survives while u_k q_k(x_k) < p_k(x_k), a product of two 24-bit
// numbers compared exactly.  At the first rejection j the weights are
// r_v = max(0, p_j(v) - q_j(v)), after a full window r = p_ell, and the token is the first v
// whose running sum of r passes u R, R the whole sum.  A negative p or q counts as zero, and so does
// a p that is not finite; a q that is infinite or NaN is above every p.  A vocabulary's sum in 32 bits is off by
// more than a rare token's probability, so a neighbour would be drawn; each difference is kept
// with its rounding error and summed as a pair of floats (hi + lo, about 2^-48 of the sum).
// (Pairs, not 64-bit arithmetic: this chip adds two doubles a clock and SM, and even the few
// sums of a warp's end in it took more of the kernel than its reads.)
//
// One small launch makes the tests of every position (where a request has one CTA, that CTA makes
// them: at one request of 4096 tokens the device then needs 8.2 us instead of 10.2 and the caller's
// thread 17.6 instead of 21).  The draw's reads one row (two with a dense draft) of the vocabulary
// once and starts while the tests are made.  A request's row is
// cut into segments, one a warp of its CTAs; a thread's next reads are always on their way to
// shared memory while it adds up the ones that have come.  The CTA of a request that ends last
// joins the segments' sums, in order, and reads the one segment where the sum passes u R again.
// 128 dense rows of 152k tokens (156 MB) take 39 us, 4.0 TB/s, 256 with lists (as many bytes) 50:
// beside the reads stand the tests' dependent loads, the last request's join, and the starts and ends
// of 1280 and 2560 CTAs in 2.1 and 4.2 waves, each with its row's position, its first reads, a fence
// and an atomic for eight and four slots of work a warp.
// Not kept: clusters, which could exchange the sums through shared memory, left SMs empty (the
// draw alone 41 us); warps that run on from segment to segment with a third launch that joins took
// 46 us, the bookkeeping and the third launch costing more than the starts that they saved.

#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "async_copy.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "sm103.cuh"
#include "training.h"

namespace dspark {
namespace {

constexpr int kVpThreads = 256;
constexpr int kVpWarps = kVpThreads / 32;
constexpr int kVpSegments = kVpWarps * kVpMaxCtas;  // of a request at most
constexpr int kVpGroup = 128;                       // tokens a warp adds up at a time
constexpr int kVpMaxGroups = 16;                    // of a segment (V <= 2^18)
constexpr int kVpSlot = 2 * kVpGroup;               // tokens of a ring's slot
constexpr int kVpRing = 3;                          // slots in shared memory, one worked on
static_assert(kVpSegments * kVpMaxGroups * kVpGroup >= 1 << 18 && kVpSegments == 128, "");

// s + e = a + b exactly (Knuth's two-sum), two at a time
__device__ __forceinline__ void two_sum(F2 a, F2 b, F2& s, F2& e) {
  const F2 neg(-1.f, -1.f);
  s = a + b;
  const F2 bb = fma2(a, neg, s);
  e = fma2(fma2(bb, neg, s), neg, a) + fma2(bb, neg, b);
}

__device__ __forceinline__ bool has_mass(float x) { return x > 0.f && x <= FLT_MAX; }
// A draft's probability: a negative one is zero, a NaN stays.
__device__ __forceinline__ float draft_mass(float q) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(q), "f"(0.f));
  return r;
}

// A number as hi + lo, |lo| at most half a step of hi.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float s = a.hi + b.hi, bb = s - a.hi;
  const float e = ((a.hi - (s - bb)) + (b.hi - bb)) + (a.lo + b.lo);
  const float hi = s + e;
  return {hi, e - (hi - s)};
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.hi, -b.lo}; }
__device__ __forceinline__ Pair operator*(float u, Pair a) {
  const float p = u * a.hi, e = fmaf(u, a.hi, -p) + u * a.lo, hi = p + e;
  return {hi, e - (hi - p)};
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
__device__ __forceinline__ Pair shfl_xor(Pair a, int off) {
  return {__shfl_xor_sync(0xFFFFFFFFu, a.hi, off), __shfl_xor_sync(0xFFFFFFFFu, a.lo, off)};
}
__device__ __forceinline__ Pair shfl(Pair a, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, a.hi, lane), __shfl_sync(0xFFFFFFFFu, a.lo, lane)};
}
// Running sums over a warp's lanes, in order.
__device__ __forceinline__ Pair warp_running(Pair x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Pair y{__shfl_up_sync(0xFFFFFFFFu, x.hi, off), __shfl_up_sync(0xFFFFFFFFu, x.lo, off)};
    if (lane >= off) x = y + x;
  }
  return x;
}

__device__ __forceinline__ Pair warp_sum(Pair x, int lane) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const Pair y = shfl_xor(x, off);
    x = lane & off ? y + x : x + y;  // (the same on both sides)
  }
  return x;
}
// The first lane with mass whose running sum passes `want`; where rounding leaves none, the last
// with mass (-1: none has).
__device__ __forceinline__ int first_past(Pair x, Pair run, Pair want) {
  const unsigned mass = __ballot_sync(0xFFFFFFFFu, x.hi > 0.f);
  const unsigned past = __ballot_sync(0xFFFFFFFFu, run > want) & mass;
  return past != 0u ? __ffs(past) - 1 : 31 - __clz(mass);
}

// Running sums of weights, two at a time.
struct Sum {
  F2 hi = F2(0.f, 0.f), lo = F2(0.f, 0.f);
  // max(0, p - q) as max(p, q) - q, with its rounding error (p - (p - q)) - q (exact where
  // p >= q >= 0).  An entry that is not finite ends in a sum that is not; kCareful gives such
  // entries no mass instead.
  template <bool kCareful>
  __device__ __forceinline__ void add_residual(float p0, float p1, float q0, float q1) {
    q0 = draft_mass(q0);
    q1 = draft_mass(q1);
    const F2 p(fmaxf(p0, q0), fmaxf(p1, q1)), q(q0, q1), neg(-1.f, -1.f);
    F2 d = fma2(q, neg, p), err = fma2(q, neg, fma2(d, neg, p)), s, e;
    if (kCareful) {
      float d0, d1, e0, e1;
      d.get(d0, d1);
      err.get(e0, e1);
      const bool m0 = has_mass(d0), m1 = has_mass(d1);
      d = F2(m0 ? d0 : 0.f, m1 ? d1 : 0.f);
      err = F2(m0 ? e0 : 0.f, m1 ? e1 : 0.f);
    }
    two_sum(hi, d, s, e);
    hi = s;
    lo = lo + (e + err);
  }
  template <bool kCareful>
  __device__ __forceinline__ void add_mass(float p0, float p1) {
    p0 = kCareful ? (has_mass(p0) ? p0 : 0.f) : fmaxf(p0, 0.f);
    p1 = kCareful ? (has_mass(p1) ? p1 : 0.f) : fmaxf(p1, 0.f);
    F2 s, e;
    two_sum(hi, F2(p0, p1), s, e);
    hi = s;
    lo = lo + e;
  }
  __device__ __forceinline__ Pair value() const {
    float a, b, c, d;
    hi.get(a, b);
    lo.get(c, d);
    return Pair{a, 0.f} + Pair{c, 0.f} + (Pair{b, 0.f} + Pair{d, 0.f});
  }
};

// One weight.
__device__ __forceinline__ Pair weight_of(float p, float q) {
  q = draft_mass(q);
  const float d = p - q;
  return has_mass(d) ? Pair{d, (p - d) - q} : Pair{0.f, 0.f};
}

// u q < p of the exact product (its low part is lost where the product is near the denormals)
__device__ __forceinline__ bool survives(float u, float q, float p) {
  const float hi = u * q;
  if (hi < 1e-30f) return static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);
  return hi < p || (hi == p && fmaf(u, q, -hi) < 0.f);
}

// The tests of a request's positions by a warp, a lane per position (K <= 64): the first that
// fails, or ell.
__device__ __forceinline__ int first_failure(const VerifyProbsArgs& a, int b, int lane) {
  const int len = a.ell == nullptr ? a.K : min(max(__ldg(a.ell + b), 0), a.K);
  int first = len;
  for (int k0 = 0; k0 < a.K; k0 += 32) {
    const int k = k0 + lane;
    bool fail = false;
    if (k < a.K) {
      const size_t o = static_cast<size_t>(b) * a.K + k;
      const float u = __ldg(a.u_accept + o);
      int x = __ldg(a.tokens + o);
      float prob = -1.f;
      if (k < len) {
        if (x < 0 || x >= a.V) {
          record_error(a.status, kStatusDeviceOob);
          x = 0;
        }
        const float target = __ldg(a.P + (static_cast<size_t>(b) * (a.K + 1) + k) * a.V + x);
        const float p = has_mass(target) ? target : 0.f;
        float q = 0.f;
        if (a.m == 0) {
          q = __ldg(a.Q + o * a.V + x);
        } else {
          bool found = false;
#pragma unroll 16
          for (int i = 0; i < a.m; ++i) {
            const int id = __ldg(a.cand + o * a.m + i);
            const float qi = __ldg(a.cand_q + o * a.m + i);
            if (id == x && !found) {
              q = qi;
              found = true;
            }
          }
        }
        q = draft_mass(q);
        fail = !survives(u, q, p);
        prob = q > 0.f ? fminf(1.f, p / q) : (p > 0.f && q == 0.f ? 1.f : 0.f);
      }
      if (a.accept_prob != nullptr) a.accept_prob[o] = prob;
    }
    const unsigned fails = __ballot_sync(0xFFFFFFFFu, fail);
    if (fails != 0u) first = min(first, k0 + __ffs(fails) - 1);
  }
  if (lane == 0) a.n_acc[b] = first;
  return first;
}

__global__ void __launch_bounds__(128) verify_tests_kernel(const VerifyProbsArgs a) {
  griddep_launch_dependents();
  const int b = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (b < a.B) first_failure(a, b, threadIdx.x & 31);
}

// kWide: rows start on 16-byte boundaries (V and the addresses a multiple of 4 tokens).
template <bool kWide>
__global__ void __launch_bounds__(kVpThreads, 4)
    verify_draw_kernel(const VerifyProbsArgs a, const int ctas, const int seg) {
  const int b = blockIdx.x / ctas, cta = blockIdx.x - b * ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = a.V, K = a.K, m = a.m;
  extern __shared__ float4 s_ring4[];  // [warp][kVpRing][p, q][kVpSlot]
  float* s_ring = reinterpret_cast<float*>(s_ring4);
  __shared__ int s_id[kMaxTeacher];
  __shared__ float s_q[kMaxTeacher];
  __shared__ Pair s_sum[kVpSegments];    // the last CTA's: of every segment
  __shared__ Pair s_group[kVpMaxGroups];  // and of the groups of the one it looks into
  __shared__ int s_done;

  const int len = a.ell == nullptr ? K : min(max(__ldg(a.ell + b), 0), K);
  int j;
  if (ctas == 1) {  // the only CTA makes the request's tests as well
    if (warp == 0) s_done = first_failure(a, b, lane);
    __syncthreads();
    j = s_done;
    __syncthreads();
  } else {
    griddep_wait();
    j = __ldcg(a.n_acc + b);
  }

  // ---- the row of the draw, and its segments
  const size_t o = static_cast<size_t>(b) * K + j;
  const float* prow = a.P + (static_cast<size_t>(b) * (K + 1) + j) * V;
  const float* qrow = m == 0 && j < len ? a.Q + o * V : nullptr;
  const bool sparse = m > 0 && j < len;
  const int segments = ctas * kVpWarps;
  const auto begin = [&](int s) { return min(V, s * seg); };
  const auto lists = [&]() {
    if (!sparse) return;
    for (int i = tid; i < m; i += kVpThreads) {
      s_id[i] = __ldg(a.cand + o * m + i);
      s_q[i] = __ldg(a.cand_q + o * m + i);
    }
    __syncthreads();
  };
  // q of the tokens v, v + step, ... among the candidates (from the last, so that the first of
  // equal ids stays)
  const auto candidates = [&](int v, int step, float (&q)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = 0.f;
#pragma unroll 4
    for (int i = m - 1; i >= 0; --i) {
      const int e = s_id[i] - v;
      const float x = s_q[i];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e == k * step) q[k] = x;
    }
  };

  // One pass over segment `s` by this warp; its sum.  Two rows or the target's alone.
  float* const ring = s_ring + warp * kVpRing * 2 * kVpSlot + (kWide ? 4 * lane : lane);
  const auto stream = [&](auto two, auto careful, bool listing, int s, auto meanwhile) {
    constexpr bool kTwo = decltype(two)::value, kCareful = decltype(careful)::value;
    const int v0 = begin(s), v1 = begin(s + 1);
    constexpr int kSlot = kTwo ? kVpSlot : 2 * kVpSlot;  // one row has a slot to itself
    const int slots = (v1 - v0 + kSlot - 1) / kSlot;
    const float* pp = prow + v0 + (kWide ? 4 * lane : lane);  // this lane's next copies
    const float* qq = kTwo ? qrow + v0 + (kWide ? 4 * lane : lane) : nullptr;
    int rest = v1 - v0 - (kWide ? 4 * lane : lane), to = 0, from = 0;
    // a lane copies the tokens it will read (zeros past the segment's end)
    const auto fetch = [&](int k) {
      if (k < slots) {
        float* dst = ring + to * 2 * kVpSlot;
        constexpr int kStep = kWide ? kVpGroup : 32, kPieces = kSlot / kStep;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int n = rest - i * kStep;  // tokens left from this piece on
          if (kWide) {
            const int bytes = n >= 4 ? 16 : (n > 0 ? 4 * n : 0);
            cp_async_16_zfill(dst + i * kStep, n > 0 ? pp + i * kStep : prow, bytes);
            if (kTwo) cp_async_16_zfill(dst + kVpSlot + i * kStep, n > 0 ? qq + i * kStep : qrow, bytes);
          } else {
            cp_async_4_zfill(dst + i * kStep, n > 0 ? pp + i * kStep : prow, n > 0 ? 4 : 0);
            if (kTwo)
              cp_async_4_zfill(dst + kVpSlot + i * kStep, n > 0 ? qq + i * kStep : qrow, n > 0 ? 4 : 0);
          }
        }
        pp += kSlot;
        if (kTwo) qq += kSlot;
        rest -= kSlot;
        to = to == kVpRing - 1 ? 0 : to + 1;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kVpRing - 1; ++k) fetch(k);
    meanwhile();
    uint32_t listed = 0u;  // groups of the segment that hold a candidate
    if (!kTwo && listing) {
      for (int i = lane; i < m; i += 32) {
        const int id = s_id[i];
        if (id >= v0 && id < v1) listed |= 1u << ((id - v0) / kVpGroup);
      }
      listed = __reduce_or_sync(0xFFFFFFFFu, listed);
    }
    Sum sum;
    for (int k = 0; k < slots; ++k) {
      fetch(k + kVpRing - 1);
      cp_async_wait_group<kVpRing - 1>();
      const float* src = ring + from * 2 * kVpSlot;
      from = from == kVpRing - 1 ? 0 : from + 1;
#pragma unroll
      for (int h = 0; h < kSlot / kVpGroup; ++h) {
        float p[4], q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = h * kVpGroup + (kWide ? i : 32 * i);
          p[i] = src[at];
          if (kTwo) q[i] = src[kVpSlot + at];
        }
        const int g = kSlot / kVpGroup * k + h;
        if (kTwo) {
          sum.add_residual<kCareful>(p[0], p[1], q[0], q[1]);
          sum.add_residual<kCareful>(p[2], p[3], q[2], q[3]);
        } else if (listed >> g & 1u) {
          candidates(v0 + g * kVpGroup + (kWide ? 4 * lane : lane), kWide ? 1 : 32, q);
          sum.add_residual<true>(p[0], p[1], q[0], q[1]);
          sum.add_residual<true>(p[2], p[3], q[2], q[3]);
        } else {
          sum.add_mass<kCareful>(p[0], p[1]);
          sum.add_mass<kCareful>(p[2], p[3]);
        }
      }
    }
    return warp_sum(sum.value(), lane);
  };
  using No = std::false_type;
  using Yes = std::true_type;

  bool left = j < len;  // weights are what the draft left over, else the target's row
  {
    const int s = cta * kVpWarps + warp;
    const Pair mine = left && qrow != nullptr ? stream(Yes{}, No{}, false, s, lists)
                                              : stream(No{}, No{}, left, s, lists);
    if (lane == 0) reinterpret_cast<float2*>(a.sums)[b * kVpSegments + s] = make_float2(mine.hi, mine.lo);
  }
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_done = atomicAdd(a.count + b, 1);
  }
  __syncthreads();
  if (s_done != ctas - 1) return;

  // ---- the request's last CTA: the total, the segment where the running sum passes u total
  __threadfence();
  if (tid == 0) a.count[b] = 0;  // as it was found
  if (tid < segments) {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(a.sums) + b * kVpSegments + tid);
    s_sum[tid] = Pair{x.x, x.y};
  }
  const Pair none{0.f, 0.f};
  Pair want = none;
  int owner = -1;
  for (bool careful = false;;) {
    __syncthreads();
    // (each warp for itself: lane's four segments, then the lanes)
    Pair x[4], of_lane = none;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = 4 * lane + i < segments ? s_sum[4 * lane + i] : none;
      of_lane = of_lane + x[i];
    }
    const Pair run = warp_running(of_lane, lane), total = shfl(run, 31);
    if (total.hi > 0.f && total.hi <= FLT_MAX) {
      want = __ldg(a.u_draw + b) * total;
      const int at = first_past(of_lane, run, want);
      if (at > 0) want = want - shfl(run, at - 1);
      Pair acc = none;
      int found = -1, last = -1;
      for (int i = 0; i < 4; ++i) {
        const Pair y = shfl(x[i], at);
        if (y.hi > 0.f) {
          last = i;
          if (found < 0 && acc + y > want) found = i;
          if (found < 0) acc = acc + y;
        }
      }
      if (found < 0) {  // (rounding) the last with mass: what is before it goes off again
        found = last;
        acc = none;
        for (int i = 0; i < found; ++i) acc = acc + shfl(x[i], at);
      }
      want = want - acc;
      owner = 4 * at + found;
      break;
    }
    // rare: an infinity or NaN among the probabilities (they get no mass), or nothing left over
    // (then the target's own row); this CTA reads the row once more by itself
    if (total.hi == 0.f) {
      if (!left) break;
      left = false;
    } else if (careful) {
      break;
    }
    careful = true;
    __syncthreads();
    for (int s = warp; s < segments; s += kVpWarps) {
      const Pair sum = left && qrow != nullptr ? stream(Yes{}, Yes{}, false, s, [] {})
                                               : stream(No{}, Yes{}, left, s, [] {});
      if (lane == 0) s_sum[s] = sum;
    }
  }
  if (owner < 0) {
    if (tid == 0) a.next_token[b] = -1;
    return;
  }

  // ---- that segment: the sums of its groups (two a warp), the group's token
  const int w0 = begin(owner), w1 = begin(owner + 1);
  const bool two = left && qrow != nullptr;
  constexpr int kEach = kVpMaxGroups / kVpWarps;
  Pair x[kEach][4], each[kEach];  // this lane's four tokens of a group, in order
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int t = w0 + (warp + k * kVpWarps) * kVpGroup + 4 * lane;
    float p[4], q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = t + i < w1 ? __ldg(prow + t + i) : 0.f;
      q[i] = two && t + i < w1 ? __ldg(qrow + t + i) : 0.f;
    }
    if (left && sparse && t < w1) candidates(t, 1, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[k][i] = weight_of(p[i], q[i]);
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    each[k] = (x[k][0] + x[k][1]) + (x[k][2] + x[k][3]);
    const Pair y = warp_sum(each[k], lane);
    if (lane == 0) s_group[warp + k * kVpWarps] = y;
  }
  __syncthreads();
  const Pair of_group = lane < kVpMaxGroups ? s_group[lane] : none;
  Pair run = warp_running(of_group, lane);
  const int g = first_past(of_group, run, want);
  if (g % kVpWarps != warp) return;
  if (g > 0) want = want - shfl(run, g - 1);
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (g / kVpWarps == k) {
      run = warp_running(each[k], lane);
      const int chosen = first_past(each[k], run, want);
      Pair acc = shfl(run, max(chosen - 1, 0));
      if (lane != chosen) return;
      if (chosen == 0) acc = none;
      int found = -1, last = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc = acc + x[k][i];
        if (!(x[k][i].hi > 0.f)) continue;
        last = i;
        if (found < 0 && acc > want) found = i;
      }
      a.next_token[b] = w0 + g * kVpGroup + 4 * lane + (found >= 0 ? found : last);
    }
}

}  // namespace

cudaError_t launch_verify_probs(const VerifyProbsArgs& all, SmemOptIn& opt_in, int* launches,
                                cudaStream_t stream) {
  // A CTA per 15,360 tokens, 16 at most; every segment a multiple of 4 tokens.  (Of 152k tokens, in
  // 5 / 6 / 8 / 10 / 16 CTAs: 128 dense rows 43.4 / 42.6 / 43.2 / 39.0 / 39.1 us, 256 rows with lists
  // 54.0 / 51.4 / 52.6 / 49.2 / 55.5 us.  Measured at these two batches alone: the rule does not look
  // at B, and one request of 152k tokens has 10 CTAs.)
  const int ctas = std::min(kVpMaxCtas, (all.V + 15359) / 15360), segments = ctas * kVpWarps;
  const int seg = ((all.V + segments - 1) / segments + 3) & ~3;
  const bool wide = all.V % 4 == 0 && reinterpret_cast<uintptr_t>(all.P) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(all.Q) % 16 == 0;
  const auto fn = wide ? verify_draw_kernel<true> : verify_draw_kernel<false>;
  constexpr int kSmem = kVpWarps * kVpRing * 2 * kVpSlot * 4;
  cudaError_t e = opt_in(fn, kSmem);
  if (e != cudaSuccess) return e;
  for (int b0 = 0; b0 < all.B; b0 += kVpMaxRequests) {  // as many as there is scratch for
    VerifyProbsArgs a = all;
    const size_t rows = static_cast<size_t>(b0) * a.K;
    a.B = std::min(kVpMaxRequests, all.B - b0);
    a.P += (rows + b0) * a.V;
    if (a.m == 0) a.Q += rows * a.V;
    if (a.m > 0) a.cand += rows * a.m;
    if (a.m > 0) a.cand_q += rows * a.m;
    a.tokens += rows;
    a.u_accept += rows;
    a.u_draw += b0;
    if (a.ell != nullptr) a.ell += b0;
    a.n_acc += b0;
    a.next_token += b0;
    if (a.accept_prob != nullptr) a.accept_prob += rows;
    if (ctas > 1) {
      verify_tests_kernel<<<(a.B + 3) / 4, 128, 0, stream>>>(a);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
    cfg.blockDim = dim3(kVpThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, fn, a, ctas, seg);
    if (e != cudaSuccess) return e;
    *launches += ctas > 1 ? 2 : 1;
  }
  return cudaSuccess;
}

}  // namespace dspark
