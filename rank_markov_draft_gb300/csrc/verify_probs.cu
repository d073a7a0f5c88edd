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
// whose running sum of r passes u R, R the whole sum.  A vocabulary's sum in 32 bits is off by
// more than a rare token's probability, so a neighbour would be drawn; each difference is kept
// with its rounding error and summed as a pair of floats (hi + lo, about 2^-48 of the sum).
// (Pairs, not 64-bit arithmetic: this chip adds two doubles a clock and SM, and even the few
// sums of a warp's end in it took more of the kernel than its reads.)
//
// One small launch makes the tests of every position.  The draw's reads one row (two with a
// dense draft) of the vocabulary once and starts while the tests are made.  A request is a
// cluster of CTAs whose warps take consecutive segments of the row, each read as it comes; the
// segments' sums go to every CTA of the cluster, the CTA that holds the segment where the sum
// passes u R reads that one segment (16 KB at most, still in L2) again, in order.

#include <cfloat>
#include <cstdint>

#include "cluster.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "sm103.cuh"

namespace dspark {
namespace {

constexpr int kVpThreads = 256;
constexpr int kVpWarps = kVpThreads / 32;
constexpr int kVpGroup = 128;              // tokens a warp reads at a time
constexpr int kVpSegment = 32 * kVpGroup;  // of a warp at most
constexpr int kVpMaxCtas = 8;

// s + e = a + b exactly (Knuth's two-sum), two at a time
__device__ __forceinline__ void two_sum(F2 a, F2 b, F2& s, F2& e) {
  const F2 neg(-1.f, -1.f);
  s = a + b;
  const F2 bb = fma2(a, neg, s);
  e = fma2(fma2(bb, neg, s), neg, a) + fma2(bb, neg, b);
}

__device__ __forceinline__ bool has_mass(float x) { return x > 0.f && x <= FLT_MAX; }

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

// Running sums of weights, two at a time.
struct Sum {
  F2 hi = F2(0.f, 0.f), lo = F2(0.f, 0.f);
  __device__ __forceinline__ void add(F2 x, F2 err) {
    F2 s, e;
    two_sum(hi, x, s, e);
    hi = s;
    lo = lo + (e + err);
  }
  // max(0, p - q) with its rounding error; entries that are not finite have no mass
  __device__ __forceinline__ void add_residual(float p0, float p1, float q0, float q1) {
    F2 d, e;
    two_sum(F2(p0, p1), F2(-q0, -q1), d, e);
    float d0, d1, e0, e1;
    d.get(d0, d1);
    e.get(e0, e1);
    const bool m0 = has_mass(d0), m1 = has_mass(d1);
    add(F2(m0 ? d0 : 0.f, m1 ? d1 : 0.f), F2(m0 ? e0 : 0.f, m1 ? e1 : 0.f));
  }
  __device__ __forceinline__ void add_mass(float p0, float p1) {
    add(F2(has_mass(p0) ? p0 : 0.f, has_mass(p1) ? p1 : 0.f), F2(0.f, 0.f));
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
  const float d = p - q, bb = d - p;
  return has_mass(d) ? Pair{d, (p - (d - bb)) - (q + bb)} : Pair{0.f, 0.f};
}

// u q < p of the exact product (its low part is lost where the product is near the denormals)
__device__ __forceinline__ bool survives(float u, float q, float p) {
  const float hi = u * q;
  if (hi < 1e-30f) return static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);
  return hi < p || (hi == p && fmaf(u, q, -hi) < 0.f);
}

// A warp per request, a lane per position (K <= 64): n_acc is the first that fails, or ell.
__global__ void __launch_bounds__(128) verify_tests_kernel(const VerifyProbsArgs a) {
  griddep_launch_dependents();
  const int b = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= a.B) return;
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
        const float p = __ldg(a.P + (static_cast<size_t>(b) * (a.K + 1) + k) * a.V + x);
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
        fail = !survives(u, q, p);
        prob = q > 0.f ? fminf(1.f, p / q) : (p > 0.f ? 1.f : 0.f);
      }
      if (a.accept_prob != nullptr) a.accept_prob[o] = prob;
    }
    const unsigned fails = __ballot_sync(0xFFFFFFFFu, fail);
    if (fails != 0u) first = min(first, k0 + __ffs(fails) - 1);
  }
  if (lane == 0) a.n_acc[b] = first;
}

// kWide: rows start on 16-byte boundaries (V and the addresses a multiple of 4 tokens).
template <bool kWide>
__global__ void __launch_bounds__(kVpThreads, 5) verify_draw_kernel(const VerifyProbsArgs a) {
  const uint32_t rank = cluster_cta_rank(), ctas = cluster_cta_count();
  const int b = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = a.V, K = a.K, m = a.m;
  __shared__ int s_id[kMaxTeacher];
  __shared__ float s_q[kMaxTeacher];
  __shared__ alignas(8) Pair s_sum[2][kVpMaxCtas * kVpWarps];  // of the cluster's segments
  __shared__ Pair s_warp[kVpWarps];
  __shared__ int s_last[kVpWarps], s_hit[kVpWarps];

  const int len = a.ell == nullptr ? K : min(max(__ldg(a.ell + b), 0), K);
  griddep_wait();
  const int j = __ldcg(a.n_acc + b);

  // ---- the row of the draw, and this warp's segment of it
  const size_t o = static_cast<size_t>(b) * K + j;
  const float* prow = a.P + (static_cast<size_t>(b) * (K + 1) + j) * V;
  const float* qrow = m == 0 && j < len ? a.Q + o * V : nullptr;
  const bool sparse = m > 0 && j < len;
  const int segments = static_cast<int>(ctas) * kVpWarps;
  const int seg = ((V + segments - 1) / segments + 3) & ~3;
  const auto begin = [&](int s) { return min(V, s * seg); };
  const int v0 = begin(rank * kVpWarps + warp), v1 = begin(rank * kVpWarps + warp + 1);
  uint32_t listed = 0u;  // groups of this warp's segment that hold a candidate
  if (sparse) {
    for (int i = tid; i < m; i += kVpThreads) {
      s_id[i] = __ldg(a.cand + o * m + i);
      s_q[i] = __ldg(a.cand_q + o * m + i);
    }
    __syncthreads();
    for (int i = lane; i < m; i += 32) {
      const int id = s_id[i];
      if (id >= v0 && id < v1) listed |= 1u << ((id - v0) / kVpGroup);
    }
    listed = __reduce_or_sync(0xFFFFFFFFu, listed);
  }
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

  bool left = j < len;  // weights are what the draft left over, else the target's row
  int owner = -1, pass = 0;
  Pair want{0.f, 0.f};
  for (;; ++pass) {
    Sum sum;
    const auto group = [&](int v, int g, const float (&p)[4], float (&q)[4]) {
      if (left && qrow == nullptr && (listed >> g & 1u)) candidates(v, kWide ? 1 : 32, q);
      if (left && (qrow != nullptr || (listed >> g & 1u))) {
        sum.add_residual(p[0], p[1], q[0], q[1]);
        sum.add_residual(p[2], p[3], q[2], q[3]);
      } else {
        sum.add_mass(p[0], p[1]);
        sum.add_mass(p[2], p[3]);
      }
    };
    const auto load = [&](const float* row, int v, float (&x)[4]) {
      if (kWide) {
        const float4 f = __ldcs(reinterpret_cast<const float4*>(row + v));
        x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __ldcs(row + v + 32 * i);
      }
    };
    const int lane0 = kWide ? 4 * lane : lane;
    const bool two = left && qrow != nullptr;
    int v = v0, g = 0;
    // two groups at a time (four loads of a lane in flight); the row's last group by itself
    for (; v + 2 * kVpGroup <= v1; v += 2 * kVpGroup, g += 2) {
      float p0[4], p1[4], q0[4], q1[4];
      load(prow, v + lane0, p0);
      load(prow, v + kVpGroup + lane0, p1);
      if (two) {
        load(qrow, v + lane0, q0);
        load(qrow, v + kVpGroup + lane0, q1);
      }
      group(v + lane0, g, p0, q0);
      group(v + kVpGroup + lane0, g + 1, p1, q1);
    }
    for (; v < v1; v += kVpGroup, ++g) {
      float p[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = v + lane0 + (kWide ? i : 32 * i);
        p[i] = t < v1 ? __ldcs(prow + t) : 0.f;
        q[i] = t < v1 && two ? __ldcs(qrow + t) : 0.f;
      }
      group(v + lane0, g, p, q);
    }
    // every CTA of the cluster gets every segment's sum
    Pair mine = sum.value();
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const Pair other = shfl_xor(mine, off);
      mine = lane & off ? other + mine : mine + other;  // (the same on both sides)
    }
    if (lane < static_cast<int>(ctas))
      st_cluster_f32x2(&s_sum[pass][rank * kVpWarps + warp], lane, mine.hi, mine.lo);
    if (ctas > 1)
      cluster_barrier();
    else
      __syncthreads();
    // total, and the segment where the running sum passes u total (each warp for itself)
    const Pair none{0.f, 0.f};
    const Pair lo = lane < segments ? s_sum[pass][lane] : none;
    const Pair run_lo = warp_running(lo, lane);
    Pair total = shfl(run_lo, 31), hi = none, run_hi = none;
    if (segments > 32) {
      hi = lane + 32 < segments ? s_sum[pass][lane + 32] : none;
      run_hi = total + warp_running(hi, lane);
      total = shfl(run_hi, 31);
    }
    if (total.hi > 0.f) {
      want = __ldg(a.u_draw + b) * total;
      const unsigned m_lo = __ballot_sync(0xFFFFFFFFu, lo.hi > 0.f);
      const unsigned m_hi = __ballot_sync(0xFFFFFFFFu, hi.hi > 0.f);
      const unsigned p_lo = __ballot_sync(0xFFFFFFFFu, run_lo > want) & m_lo;
      const unsigned p_hi = __ballot_sync(0xFFFFFFFFu, run_hi > want) & m_hi;
      // (rounding may leave no segment past it: then the last with mass)
      owner = p_lo != 0u ? __ffs(p_lo) - 1
              : p_hi != 0u ? 31 + __ffs(p_hi)
              : m_hi != 0u ? 63 - __clz(m_hi) : 31 - __clz(m_lo);
      if (owner > 0) {  // what the owner's own sum has to pass: less the sum before it
        const Pair before = owner <= 32 ? shfl(run_lo, owner - 1) : shfl(run_hi, owner - 33);
        want = want - before;
      }
      break;
    }
    if (!left) break;
    left = false;  // nothing left over: the target's own row
  }
  if (owner < 0) {
    if (rank == 0 && tid == 0) a.next_token[b] = -1;
    return;
  }
  if (owner / kVpWarps != static_cast<int>(rank)) return;

  // ---- the owner's segment in order: 16 tokens a thread, then the thread that passes `want`
  constexpr int kPer = kVpSegment / kVpThreads;
  const int t0 = begin(owner) + tid * kPer, t1 = min(t0 + kPer, begin(owner + 1));
  uint32_t of_list = 0u;  // which of them are candidates
  if (left && sparse)
    for (int i = 0; i < m; ++i) {
      const int e = s_id[i] - t0;
      if (e >= 0 && e < kPer) of_list |= 1u << e;
    }
  const auto weight = [&](int e) {
    if (t0 + e >= t1) return Pair{0.f, 0.f};
    float q = 0.f;
    if (left && qrow != nullptr) q = __ldg(qrow + t0 + e);
    if (of_list >> e & 1u)
      for (int i = m - 1; i >= 0; --i)
        if (s_id[i] == t0 + e) q = s_q[i];
    return weight_of(__ldg(prow + t0 + e), q);
  };
  Pair sum{0.f, 0.f};
  int last = -1;
#pragma unroll 8
  for (int e = 0; e < kPer; ++e) {
    const Pair x = weight(e);
    if (x.hi > 0.f) last = t0 + e;
    sum = sum + x;
  }
  const Pair run = warp_running(sum, lane);
  last = __reduce_max_sync(0xFFFFFFFFu, last);
  if (lane == 31) s_warp[warp] = run;
  if (lane == 0) s_last[warp] = last;
  __syncthreads();
  Pair base{0.f, 0.f};
  int end = -1;
  for (int k = 0; k < kVpWarps; ++k) {
    if (k < warp) base = base + s_warp[k];
    end = max(end, s_last[k]);
  }
  const unsigned hits = __ballot_sync(0xFFFFFFFFu, sum.hi > 0.f && base + run > want);
  if (lane == 0) s_hit[warp] = hits != 0u ? 1 : 0;
  __syncthreads();
  int first = -1;
  for (int k = kVpWarps - 1; k >= 0; --k)
    if (s_hit[k] != 0) first = k;
  if (first < 0) {  // rounding: the segment's last token with mass
    if (tid == 0) a.next_token[b] = end;
    return;
  }
  if (warp != first) return;
  const int chosen = __ffs(hits) - 1;
  const Pair before = base + shfl(run, max(chosen - 1, 0));
  if (lane != chosen) return;
  Pair acc = chosen > 0 ? before : base;
  int found = -1;
  for (int e = 0; e < kPer && found < 0; ++e) {
    const Pair x = weight(e);
    if (!(x.hi > 0.f)) continue;
    acc = acc + x;
    last = t0 + e;  // (of this thread's: the one if rounding leaves none past it)
    if (acc > want) found = t0 + e;
  }
  a.next_token[b] = found >= 0 ? found : last;
}

}  // namespace

cudaError_t launch_verify_probs(const VerifyProbsArgs& a, cudaStream_t stream) {
  // One CTA per 32768 tokens at least (a warp's segment fits its 32 group bits); more CTAs than
  // that while rows are long, so that a request's reads are spread: a CTA per 16384 tokens.
  int ctas = 1;
  while (ctas < kVpMaxCtas && a.V > ctas * 16384) ctas *= 2;
  const bool wide = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.P) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.Q) % 16 == 0;
  verify_tests_kernel<<<(a.B + 3) / 4, 128, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
  cfg.blockDim = dim3(kVpThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, wide ? verify_draw_kernel<true> : verify_draw_kernel<false>, a);
}

}  // namespace dspark
