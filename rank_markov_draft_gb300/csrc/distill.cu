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
//
// The gradient needs the row's sum, so a kernel that streams reads every logit twice.  Here a
// row is spread over the registers of a cluster of CTAs (about 40 KB a CTA): one read of the
// logits, all loads of a thread in flight at once, one exchange of (maximum, sum) through the
// cluster's shared memory, one write.  Clusters walk over the rows.  In each CTA one warp holds
// no part of the row: it prepares the next row's teacher slots (which count, the student's
// logits there, a bit map of their tokens) while the others stream the current one, so the
// dependent loads of the slots hide behind the row's.  The map tells the streaming warps which
// registers to overwrite with -inf, so neither pass tests for the teacher's tokens; their own
// gradients are written last, over the zeros.

#include <algorithm>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>
#include <cuda_bf16.h>

#include "cluster.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "rowscan.cuh"
#include "sm103.cuh"

namespace dspark {
namespace {

constexpr float kLn2 = kScanLn2;

// The larger of two values, NaN if either is (so that a row of NaN is not taken for a masked one).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = max_nan(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
  return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}

// 2^((m - top) c), 0 where m is -inf (an empty part, whatever top is)
__device__ __forceinline__ float part_scale(float m, float top, float c) {
  return m == -INFINITY ? 0.f : ex2_approx((m - top) * c);
}

// 16 bytes of a row: 4 fp32 or 8 bf16 logits.
template <typename T>
struct Row16;

template <>
struct Row16<float> {
  static constexpr int kVec = 4, kPairs = 2;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float x) { *p = x; }
  static __device__ __forceinline__ float max4(const uint4& w) {
    return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                   max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  static __device__ __forceinline__ F2 pair(const uint4& w, int i) {
    return i == 0 ? F2(__uint_as_float(w.x), __uint_as_float(w.y))
                  : F2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  static __device__ __forceinline__ F2 pair_again(const uint4& w, int i, uint2) {
    return pair(w, i);
  }
  static __device__ __forceinline__ void set_pair(uint4& w, int i, float a, float b) {
    (i == 0 ? w.x : w.z) = __float_as_uint(a);
    (i == 0 ? w.y : w.w) = __float_as_uint(b);
  }
  static __device__ __forceinline__ float get(const uint4& w, int e) {
    return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w);
  }
  static __device__ __forceinline__ void mask(uint4& w, uint32_t bits) {
    if (bits & 1u) w.x = kNegInf;
    if (bits & 2u) w.y = kNegInf;
    if (bits & 4u) w.z = kNegInf;
    if (bits & 8u) w.w = kNegInf;
  }
};

template <>
struct Row16<uint16_t> {
  static constexpr int kVec = 8, kPairs = 4;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static __device__ __forceinline__ float one(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
  }
  static __device__ __forceinline__ void put(uint16_t* p, float x) {
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(x));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float max4(const uint4& w) {
    const uint32_t m = max2(max2(w.x, w.y), max2(w.z, w.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t word(const uint4& w, int i) {
    return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
  }
  static __device__ __forceinline__ F2 pair(const uint4& w, int i) {
    const uint32_t x = word(w, i);
    return F2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  }
  // The same by two byte selections that only the launch knows: the compiler would otherwise
  // keep the unpacked logits of the first pass, twice the registers, for the second.
  static __device__ __forceinline__ F2 pair_again(const uint4& w, int i, uint2 sel) {
    const uint32_t x = word(w, i);
    return F2(__uint_as_float(__byte_perm(x, 0u, sel.x)), __uint_as_float(__byte_perm(x, 0u, sel.y)));
  }
  static __device__ __forceinline__ void set_pair(uint4& w, int i, float a, float b) {
    uint32_t x;  // one rounding to bf16, to nearest even, of each gradient
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(b), "f"(a));
    (i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w) = x;
  }
  static __device__ __forceinline__ uint16_t get(const uint4& w, int e) {
    return static_cast<uint16_t>(word(w, e >> 1) >> (16 * (e & 1)));
  }
  static __device__ __forceinline__ void half(uint32_t& w, uint32_t bits, uint32_t x) {
    if (bits & 1u) w = (w & 0xFFFF0000u) | (x & 0xFFFFu);
    if (bits & 2u) w = (w & 0xFFFFu) | (x << 16);
  }
  static __device__ __forceinline__ void mask(uint4& w, uint32_t bits) {
    half(w.x, bits, 0xFF80u);
    half(w.y, bits >> 2, 0xFF80u);
    half(w.z, bits >> 4, 0xFF80u);
    half(w.w, bits >> 6, 0xFF80u);
  }
};

// The sign of q - p where 32 bits cannot tell: TV's derivative jumps there, so the two sides
// are compared in 64 bits (rare: one slot in 1e5).
__device__ __noinline__ float sign64(float s, float top, float total, float t, float t_top,
                                     float sum_t, float rho, float T) {
  const double q = exp((static_cast<double>(s) - top) / T) / total;
  const double p = exp((static_cast<double>(t) - t_top) / T) / sum_t * (1.0 - rho);
  return q > p ? 1.f : (q < p ? -1.f : 0.f);
}

__device__ __forceinline__ float sign_of(float a, float b) {
  return a > b ? 1.f : (a < b ? -1.f : 0.f);
}

// Named barriers: the streaming warps hand their sums to the slot warp (they only arrive), the
// slot warp hands back the gradient's coefficients, and tells that a row's slots are ready (one
// barrier for even and one for odd rows, since it runs a row ahead).
constexpr int kBarSums = 1, kBarCoef = 2, kBarSlots = 3;
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

struct SlotSmem {  // double-buffered by the row's turn
  int next_id[kMaxTeacher];   // the row after the next, as it arrives
  float next_t[kMaxTeacher];
  int id[2][kMaxTeacher];     // the slots that count, or -1
  int pos[2][kMaxTeacher];    // map position of every slot with a token, or -1
  float t[2][kMaxTeacher], s[2][kMaxTeacher];  // the teacher's and the student's logits
  int out_id[2][kMaxTeacher];                  // the last row's slots, for their gradients
  float out_g[2][kMaxTeacher];
  float2 part[2][32];                          // (maximum, sum) of each streaming warp
  alignas(8) float2 cta[2][8];                 // of each CTA of the cluster
  alignas(8) uint64_t bar[2];                  // counts the bytes of cta[]
  float coef[3];                               // outside coefficient, any of it at all, maximum
};

// Where a row lies: `off` elements past a 16-byte boundary, so `head` elements before the first
// aligned vector, `body` vectors, `tail` elements after the last.
template <typename T>
struct RowSpan {
  int off, head, body, tail;
  __device__ __forceinline__ RowSpan(const T* row, int V) {
    constexpr int kVec = Row16<T>::kVec;
    off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    head = off > 0 ? min(V, kVec - off) : 0;
    body = (V - head) / kVec;
    tail = V - head - body * kVec;
  }
};

template <typename T>
struct SlotWarp {
  const DistillArgs& a;
  const float c;
  SlotSmem& sm;
  uint32_t* map[2];
  int lane;
  bool first;  // rank 0 of the cluster

  struct Row {
    int64_t n;
    float w;
    float t_top, s_top, sum_t, sum_s;
  };

  __device__ __forceinline__ float weight(int64_t n) const {
    return a.row_weight != nullptr ? __ldg(a.row_weight + n) : 1.f;
  }
  // The first row from n on, in steps of `step`, that has a weight (N: none).
  __device__ __forceinline__ Row next_live(int64_t n, int64_t step) const {
    Row r;
    for (r.n = n; r.n < a.N; r.n += step)
      if ((r.w = weight(r.n)) != 0.f) return r;
    r.n = a.N;
    return r;
  }
  // Start copying a row's slots to shared memory (each lane copies the slots it reads).
  __device__ __forceinline__ void fetch(const Row& r) const {
    if (r.n < a.N)
      for (int j = lane; j < a.k; j += 32) {
        cp_async_4(&sm.next_id[j], a.teacher_ids + r.n * a.k + j);
        cp_async_4(&sm.next_t[j], a.teacher_logits + r.n * a.k + j);
      }
    cp_async_commit();
  }
  // Buffer b: the map's bits of two rows ago out, this row's in; the slots that count and the
  // logits there; their maxima and sums.
  __device__ __forceinline__ void prepare(Row& r, int b) {
    const T* row = static_cast<const T*>(a.logits) + r.n * a.ld;
    const int off = RowSpan<T>(row, a.V).off;
    for (int j = lane; j < a.k; j += 32)
      if (sm.pos[b][j] >= 0) map[b][sm.pos[b][j] >> 5] = 0u;
    cp_async_wait_all();
    __syncwarp();
    bool again = false;
    for (int j = lane; j < a.k; j += 32) {
      int id = sm.next_id[j];
      if (id >= a.V) {
        if (first) record_error(a.status, kStatusDeviceOob);
        id = -1;
      }
      const int pos = id < 0 ? -1 : id + off;
      sm.pos[b][j] = pos;
      sm.id[b][j] = id;
      if (pos >= 0) again |= (atomicOr(&map[b][pos >> 5], 1u << (pos & 31)) >> (pos & 31)) & 1u;
    }
    if (__any_sync(0xFFFFFFFFu, again)) {  // a token more than once: its first slot counts
      __syncwarp();
      uint32_t drop = 0u;
      for (int i = 0; lane + 32 * i < a.k; ++i) {
        const int id = sm.id[b][lane + 32 * i];
        for (int j = 0; j < lane + 32 * i; ++j)
          if (id >= 0 && sm.id[b][j] == id) drop |= 1u << i;
      }
      __syncwarp();
      for (int i = 0; lane + 32 * i < a.k; ++i)
        if (drop >> i & 1u) sm.id[b][lane + 32 * i] = -1;
    }
    r.t_top = r.s_top = -INFINITY;
#pragma unroll 4
    for (int j = lane; j < a.k; j += 32) {
      const int id = sm.id[b][j];
      const float t = id >= 0 ? sm.next_t[j] : -INFINITY;
      const float s = id >= 0 ? Row16<T>::one(row + id) : -INFINITY;
      sm.t[b][j] = t;
      sm.s[b][j] = s;
      r.t_top = max_nan(r.t_top, t);
      r.s_top = max_nan(r.s_top, s);
    }
    r.t_top = warp_max(r.t_top);
    r.s_top = warp_max(r.s_top);
    r.sum_t = r.sum_s = 0.f;
    for (int j = lane; j < a.k; j += 32) {
      r.sum_t += part_scale(sm.t[b][j], r.t_top, c);
      r.sum_s += part_scale(sm.s[b][j], r.s_top, c);
    }
    r.sum_t = warp_sum(r.sum_t);
    r.sum_s = warp_sum(r.sum_s);
    __syncwarp();
  }
  // Loss and coefficients from the outside's (maximum, sum).
  __device__ __forceinline__ void finish(const Row& r, int b, float m_out, float sum_out,
                                         int threads) {
    const bool grads = a.grad != nullptr;
    const float rho = a.teacher_rest != nullptr
                          ? fminf(fmaxf(__ldg(a.teacher_rest + r.n), 0.f), 1.f)
                          : 0.f;
    const float top = max_nan(m_out, r.s_top);
    const bool any = !(r.t_top == -INFINITY || top == -INFINITY);
    const float out_part = sum_out * part_scale(m_out, top, c);
    const float total = r.sum_s * part_scale(r.s_top, top, c) + out_part;
    const float inv = 1.f / total, p_scale = (1.f - rho) / r.sum_t;
    const float ratio = log2f(total) - log2f(r.sum_t) + log2f(1.f - rho);
    const float q_rest = out_part * inv, sgn_r = sign_of(q_rest, rho);
    float S = 0.f, kl = 0.f, tv = 0.f;
    for (int j = lane; j < a.k; j += 32) {
      const float tj = sm.t[b][j], sj = sm.s[b][j];
      // an empty slot has neither side (a teacher's logit of -inf keeps its student's)
      const float xj = (tj - r.t_top) * c, yj = (sj - top) * c;
      const float p = tj == -INFINITY ? 0.f : exp2f(xj) * p_scale;
      const float q = sj == -INFINITY ? 0.f : exp2f(yj) * inv;
      float sg = sign_of(q, p);
      if (fabsf(q - p) < 1e-5f * p)
        sg = sign64(sj, top, total, tj, r.t_top, r.sum_t, rho, a.temperature);
      S += sg * q;
      tv += fabsf(p - q);
      if (p > 0.f) kl += p * (xj - yj + ratio);
      sm.t[b][j] = p;
      sm.s[b][j] = q;
      sm.out_g[b][j] = sg;
    }
    if (grads) {
      S = warp_sum(S) + sgn_r * q_rest;
      const float wt = r.w / a.temperature;
      if (lane == 0) {
        sm.coef[0] = wt *
                     (a.alpha_kl * (q_rest - rho) + 0.5f * a.alpha_tv * (sgn_r - S) * q_rest) /
                     sum_out;
        sm.coef[1] = any && sum_out != 0.f ? 1.f : 0.f;
        sm.coef[2] = m_out;
      }
      __syncwarp();
      bar_arrive(kBarCoef, threads);
      for (int j = lane; j < a.k; j += 32) {
        const float p = sm.t[b][j], q = sm.s[b][j], sg = sm.out_g[b][j];
        sm.out_g[b][j] =
            any ? wt * (a.alpha_kl * (q - p) + 0.5f * a.alpha_tv * (sg - S) * q) : 0.f;
        sm.out_id[b][j] = sm.id[b][j];
      }
    }
    if (!first) return;
    kl = warp_sum(kl);
    tv = 0.5f * (warp_sum(tv) + fabsf(rho - q_rest));
    if (rho > 0.f)
      kl += rho * (log2f(rho) - log2f(sum_out) - (m_out - top) * c + log2f(total));
    if (lane == 0) {
      a.loss[r.n] =
          any ? r.w * ((a.alpha_kl != 0.f ? a.alpha_kl * kl * kLn2 : 0.f) + a.alpha_tv * tv) : 0.f;
      if (a.tv != nullptr) a.tv[r.n] = any ? tv : 0.f;
    }
  }
  // The gradients of a finished row's slots whose tokens this CTA holds, over the zeros that
  // its streaming warps wrote there before they arrived at a barrier this warp has passed.
  __device__ __forceinline__ void patch(int64_t n, int b, int v0, int cnt, bool edges,
                                        const RowSpan<T>& sp) const {
    T* grad = static_cast<T*>(a.grad) + n * a.ld_grad;
    for (int j = lane; j < a.k; j += 32) {
      const int id = sm.out_id[b][j];
      if (id < 0) continue;
      const int e = id - sp.head;
      const bool inner = e >= 0 && e < sp.body * Row16<T>::kVec;
      const int v = e / Row16<T>::kVec - v0;
      if (inner ? v >= 0 && v < cnt : edges) Row16<T>::put(grad + id, sm.out_g[b][j]);
    }
  }
};

// A cluster walks over rows g, g + clusters, ...; CTA `rank` holds body vectors [v0, v0 + cnt)
// of a row, vector i of a streaming thread at tid + i * (threads - 32); all but the last i are
// full (the host picks the threads so).  The up to 14 elements outside the body are single elements of warp
// 0's lanes in rank 0.
template <typename T, int NV, int kMaxThreads, int kPerSm>
__global__ void __launch_bounds__(kMaxThreads, kPerSm)
    distill_kernel(const DistillArgs a, const float c, const int map_words, const uint2 sel) {
  using R = Row16<T>;
  constexpr int kVec = R::kVec;
  const int nt = blockDim.x, row_threads = nt - 32, row_warps = row_threads / 32;
  __shared__ SlotSmem sm;
  extern __shared__ uint32_t maps[];  // 2 x map_words

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_cta_rank(), ctas = cluster_cta_count();
  const int64_t step = gridDim.x / ctas, n0 = blockIdx.x / ctas;
  const bool grads = a.grad != nullptr;
  const auto v_begin = [&](int body, int r) {
    return static_cast<int>(static_cast<int64_t>(body) * r / static_cast<int>(ctas));
  };
  for (int i = tid; i < 2 * map_words; i += nt) maps[i] = 0u;
  for (int i = tid; i < 2 * kMaxTeacher; i += nt) (&sm.pos[0][0])[i] = -1;
  if (tid == 0) {
    mbar_init(&sm.bar[0], 1);
    mbar_init(&sm.bar[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (ctas > 1) cluster_barrier();  // every CTA's mbarriers exist

  if (warp == row_warps) {  // ---------------------------------------------- the slot warp
    SlotWarp<T> sw{a, c, sm, {maps, maps + map_words}, lane, rank == 0};
    using Row = typename SlotWarp<T>::Row;
    Row cur = sw.next_live(n0, step), last;
    last.n = a.N;
    if (cur.n < a.N) {
      sw.fetch(cur);
      sw.prepare(cur, 0);
      bar_arrive(kBarSlots, nt);
    }
    Row nxt = cur.n < a.N ? sw.next_live(cur.n + step, step) : cur;
    sw.fetch(nxt);
    for (int turn = 0; cur.n < a.N; ++turn) {
      const int b = turn & 1;
      Row after = nxt;
      if (nxt.n < a.N) {
        sw.prepare(nxt, b ^ 1);
        bar_arrive(kBarSlots + (b ^ 1), nt);
        after = sw.next_live(nxt.n + step, step);
        sw.fetch(after);
      }
      bar_sync(kBarSums, nt);
      const float2 o = lane < row_warps ? sm.part[b][lane] : make_float2(-INFINITY, 0.f);
      if (!grads) {  // the streaming warps go on at once
        __syncwarp();
        bar_arrive(kBarCoef, nt);
      }
      float m = warp_max(o.x);
      float sum = warp_sum(o.y * part_scale(o.x, m, c));
      if (ctas > 1) {
        if (lane == 0) mbar_arrive_expect_tx(&sm.bar[b], 8u * ctas);
        if (lane < static_cast<int>(ctas)) st_async_f32x2(&sm.cta[b][rank], &sm.bar[b], lane, m, sum);
        if (!mbar_wait_cluster(&sm.bar[b], (turn >> 1) & 1, a.timeout_ns) && lane == 0)
          record_error(a.status, kStatusTimeout);
        __syncwarp();
        const float2 p = lane < static_cast<int>(ctas) ? sm.cta[b][lane] : make_float2(-INFINITY, 0.f);
        m = warp_max(p.x);
        sum = warp_sum(p.y * part_scale(p.x, m, c));
      }
      if (grads || rank == 0) sw.finish(cur, b, m, sum, nt);
      if (grads && last.n < a.N) {  // (the streaming warps were done with it at kBarSums)
        const RowSpan<T> sp(static_cast<const T*>(a.logits) + last.n * a.ld, a.V);
        const int v0 = v_begin(sp.body, rank);
        sw.patch(last.n, b ^ 1, v0, v_begin(sp.body, rank + 1) - v0, rank == 0, sp);
      }
      last = cur;
      cur = nxt;
      nxt = after;
      if (grads && cur.n >= a.N) {
        bar_sync(kBarSums, nt);  // the streaming warps have written the last row
        const RowSpan<T> sp(static_cast<const T*>(a.logits) + last.n * a.ld, a.V);
        const int v0 = v_begin(sp.body, rank);
        __syncwarp();
        sw.patch(last.n, b, v0, v_begin(sp.body, rank + 1) - v0, rank == 0, sp);
      }
    }
    if (ctas > 1) cluster_barrier();  // no CTA leaves while another may still store into it
    return;
  }

  // ------------------------------------------------------------- the warps that hold the row
  const F2 scale(c, c);
  int turn = 0;
  float w_next = n0 < a.N ? (a.row_weight != nullptr ? __ldg(a.row_weight + n0) : 1.f) : 0.f;
  for (int64_t n = n0; n < a.N; n += step) {
    const float w = w_next;
    w_next = n + step < a.N && a.row_weight != nullptr ? __ldg(a.row_weight + n + step) : 1.f;
    const T* row = static_cast<const T*>(a.logits) + n * a.ld;
    T* grad = grads ? static_cast<T*>(a.grad) + n * a.ld_grad : nullptr;
    const RowSpan<T> sp(row, a.V);
    const int v0 = v_begin(sp.body, rank), cnt = v_begin(sp.body, rank + 1) - v0;
    const uint4* src = reinterpret_cast<const uint4*>(row + sp.head) + v0 + tid;
    T* dst = grad + sp.head + static_cast<int64_t>(v0 + tid) * kVec;
    const bool aligned = (reinterpret_cast<uintptr_t>(grad + sp.head) & 15u) == 0;
    // this thread's single element, if it has one
    int edge = -1;
    if (rank == 0 && tid < 16) {
      if (tid < sp.head) edge = tid;
      if (tid >= 8 && tid - 8 < sp.tail) edge = a.V - sp.tail + tid - 8;
    }
    const auto has = [&](int i) { return i < NV - 1 || tid + i * row_threads < cnt; };
    const auto store = [&](int i, const uint4& g) {
      if (aligned) {
        __stcs(reinterpret_cast<uint4*>(dst) + i * row_threads, g);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) dst[i * row_threads * kVec + e] = R::get(g, e);
      }
    };
    if (w == 0.f) {  // neither read nor looked at
      if (rank == 0 && tid == 0) {
        a.loss[n] = 0.f;
        if (a.tv != nullptr) a.tv[n] = 0.f;
      }
      if (grads) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (has(i)) store(i, make_uint4(0u, 0u, 0u, 0u));
        if (edge >= 0) R::put(grad + edge, 0.f);
      }
      continue;
    }
    uint4 x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (has(i))
        x[i] = __ldcs(src + i * row_threads);
      else
        x[i] = make_uint4(R::kNegInf, R::kNegInf, R::kNegInf, R::kNegInf);
    }
    float xe = edge >= 0 ? R::one(row + edge) : -INFINITY;
    const int b = turn & 1;
    ++turn;
    const uint32_t* map = maps + b * map_words;
    bar_sync(kBarSlots + b, nt);
    // the teacher's tokens out
    {
      const int p0 = v0 + tid + (sp.off > 0 ? 1 : 0);
      const uint8_t* bytes = reinterpret_cast<const uint8_t*>(map);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int p = p0 + i * row_threads;
        if (!has(i)) continue;
        const uint32_t bits = kVec == 8 ? bytes[p] : (bytes[p >> 1] >> (4 * (p & 1))) & 15u;
        if (bits != 0u) R::mask(x[i], bits);
      }
      if (edge >= 0 && (map[(edge + sp.off) >> 5] >> ((edge + sp.off) & 31) & 1u)) xe = -INFINITY;
    }
    {
      float m = max_nan(xe, R::max4(x[0]));
#pragma unroll
      for (int i = 1; i < NV; ++i) m = max_nan(m, R::max4(x[i]));
      m = warp_max(m);
      const float ref = m == -INFINITY ? 0.f : m;
      const F2 minus(-ref, -ref);
      F2 acc(ex2_approx((xe - ref) * c), 0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int p = 0; p < R::kPairs; ++p) {
          float y0, y1;
          ((R::pair(x[i], p) + minus) * scale).get(y0, y1);
          acc = acc + F2(ex2_approx(y0), ex2_approx(y1));
        }
      float sa, sb;
      acc.get(sa, sb);
      const float sum = warp_sum(sa + sb);
      if (lane == 0) sm.part[b][warp] = make_float2(m, sum);
      __syncwarp();
      bar_arrive(kBarSums, nt);
    }
    bar_sync(kBarCoef, nt);
    if (!grads) continue;
    const bool zero = sm.coef[1] == 0.f;
    const float coef = sm.coef[0], m_out = sm.coef[2];
    const float ref = m_out == -INFINITY ? 0.f : m_out;
    const F2 minus(-ref, -ref), mul(coef, coef);
    const auto write = [&](auto exp2_of) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        uint4 g;
#pragma unroll
        for (int p = 0; p < R::kPairs; ++p) {
          float y0, y1;
          ((R::pair_again(x[i], p, sel) + minus) * scale).get(y0, y1);
          (F2(exp2_of(y0), exp2_of(y1)) * mul).get(y0, y1);
          R::set_pair(g, p, y0, y1);
        }
        if (has(i)) store(i, g);
      }
      if (edge >= 0) R::put(grad + edge, exp2_of((xe - ref) * c) * coef);
    };
    if (zero) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (has(i)) store(i, make_uint4(0u, 0u, 0u, 0u));
      if (edge >= 0) R::put(grad + edge, 0.f);
    } else if (fabsf(coef) <= 1.f) {
      write([](float y) { return ex2_approx(y); });
    } else {
      // the fast exponential drops results below 2^-126, which a coefficient above one brings
      // back into range
      write([](float y) { return exp2f(y); });
    }
  }
  if (grads && turn > 0) {
    __syncwarp();
    bar_arrive(kBarSums, nt);
  }
  if (ctas > 1) cluster_barrier();
}

// Clusters of this launch that the device holds at once (an SM takes kPerSm CTAs, but a cluster
// has to fit one GPC); asked once for each shape a kernel is launched with.
int resident_clusters(const void* fn, const cudaLaunchConfig_t& cfg, int ctas) {
  static std::mutex lock;
  static std::map<std::tuple<const void*, int, unsigned, size_t>, int> known;
  const auto key = std::make_tuple(fn, ctas, cfg.blockDim.x, cfg.dynamicSmemBytes);
  std::lock_guard<std::mutex> hold(lock);
  const auto it = known.find(key);
  if (it != known.end()) return it->second;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = 1;
  }
  if (known.size() < 4096) known[key] = n;
  return n;
}

template <typename T, int NV, int kMaxThreads, int kPerSm>
cudaError_t launch(const DistillArgs& a, int row_threads, int ctas, int num_sms,
                   cudaStream_t stream) {
  const auto fn = distill_kernel<T, NV, kMaxThreads, kPerSm>;
  const int map_words = (a.V + 2 * Row16<T>::kVec + 31) / 32;
  // (the largest maps are above the default limit of dynamic shared memory)
  static const cudaError_t once =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * 4 * 8200);
  if (once != cudaSuccess) return once;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms / ctas * ctas));
  cfg.blockDim = dim3(row_threads + 32);
  cfg.dynamicSmemBytes = 2 * 4 * map_words;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int64_t clusters =
      std::min<int64_t>(a.N, resident_clusters(reinterpret_cast<const void*>(fn), cfg, ctas));
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * ctas));
  const float c = static_cast<float>(1.4426950408889634 / static_cast<double>(a.temperature));
  return cudaLaunchKernelEx(&cfg, fn, a, c, map_words, make_uint2(0x1044u, 0x3244u));
}

// Streaming threads that hold `most` vectors in NV each with all but the last NV full for a CTA
// of `least` (0: none below `limit` do).
int threads_for(int nv, int most, int least, int limit) {
  const int t = (((most + nv - 1) / nv + 31) / 32) * 32;
  return t <= limit && (nv - 1) * t <= least ? std::max(t, 32) : 0;
}

template <typename T>
cudaError_t dispatch(const DistillArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kVec = Row16<T>::kVec;
  // 16-byte vectors of a row: a row that starts off a boundary has one less
  const int body = a.V / kVec, body_least = std::max(0, (a.V - kVec + 1) / kVec);
  // The smallest cluster whose CTAs hold the row in 288 threads x 9 vectors (three CTAs an SM),
  // up to 8 CTAs; more CTAs a row while the SMs would otherwise be empty.
  int ctas = 1;
  while (ctas < 8 && ((body + ctas - 1) / ctas > 288 * 9 ||
                      (a.N * ctas * 2 <= num_sms && (body + ctas - 1) / ctas > 288)))
    ctas *= 2;
  const int most = std::max(1, (body + ctas - 1) / ctas), least = body_least / ctas;
  int t;
  if ((t = threads_for(1, most, least, 96))) return launch<T, 1, 128, 6>(a, t, ctas, num_sms, stream);
  if ((t = threads_for(2, most, least, 96))) return launch<T, 2, 128, 6>(a, t, ctas, num_sms, stream);
  if ((t = threads_for(3, most, least, 96))) return launch<T, 3, 128, 6>(a, t, ctas, num_sms, stream);
  if ((t = threads_for(4, most, least, 288)))
    return launch<T, 4, 320, 3>(a, t, ctas, num_sms, stream);
  if ((t = threads_for(6, most, least, 288)))
    return launch<T, 6, 320, 3>(a, t, ctas, num_sms, stream);
  if ((t = threads_for(9, most, least, 288)))
    return launch<T, 9, 320, 3>(a, t, ctas, num_sms, stream);
  if ((t = threads_for(10, most, least, 480)))
    return launch<T, 10, 512, 2>(a, t, ctas, num_sms, stream);
  // (fp32 rows of more than 153600 logits)
  t = threads_for(10, most, least, 992);
  return launch<T, 10, 1024, 1>(a, t, ctas, num_sms, stream);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int num_sms, cudaStream_t stream) {
  return a.dtype == DSPARK_F32 ? dispatch<float>(a, num_sms, stream)
                               : dispatch<uint16_t>(a, num_sms, stream);
}

}  // namespace dspark
