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
// The gradient needs the row's sum, so every logit is wanted twice, and is to come from memory
// once.  Two kernels:
//   Short rows (152 KB at most) lie in the registers of one CTA between the passes.  CTAs walk
//   over the rows; one warp of each holds no part of the row and prepares the next row's teacher
//   slots (which count, the student's logits there, a bit map of their tokens) while the others
//   stream the current one, so the dependent loads of the slots hide behind the row's.
//   Long rows are cut into segments of 7 to 22 KB (fewer rows into shorter ones, from 2 KB), one a
//   warp.  A warp sums its segment of one round, then writes the gradient of its segment of the
//   round before, which it reads again: the two readings are one round (18 to 55 MB over the chip)
//   apart, so that the second may come from L2.  In fp32 it does, but for 7%, since the copies say
//   what is read for the last time; in bf16 83% of it comes from DRAM.  Each
//   segment's (maximum, sum) goes through memory to the row's service warp (one in each CTA),
//   which joins them, finishes the row and publishes the coefficients; a round of work lies
//   between, so nobody waits for long.  The launch is cooperative: all of its CTAs run.
//   2048 x 151936 with gradient: fp32 450 us (5.5 TB/s, 83% of a copy's rate, the 10% of the rows
//   that have no weight counted as read), bf16 272 us (4.6 TB/s; what it moves, the second reading
//   with it, is 84% of a copy's rate and bounds it: 47% of the issue slots are used), 1024 bf16 rows
//   without 68 us (4.6 TB/s): neither DRAM nor the issue slots (59%) bound that one, but its eight
//   units a warp, dealt out with the rows of no weight among them, and a short launch's start and end.
// In both the teacher's tokens are left out of the outside sum by overwriting them with -inf on
// chip, and their own gradients are written last, over what the stream wrote there.

#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>

#include "async_copy.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "rowscan.cuh"
#include "sm103.cuh"
#include "training.h"

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
  static __device__ __forceinline__ float max8(const uint4& v, const uint4& w) {
    return max_nan(max4(v), max4(w));
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
  static __device__ __forceinline__ float max8(const uint4& v, const uint4& w) {
    const uint32_t m = max2(max2(max2(v.x, v.y), max2(v.z, v.w)), max2(max2(w.x, w.y), max2(w.z, w.w)));
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

// The sign of q - p, where TV's derivative jumps.  Where the slot's own exponentials and products in
// 32 bits could hide it (rare: one slot in 1e5) they are taken in 64; the row's sums stay those of 32
// bits, a few 1e-7 off, so a nearer tie falls either way, all slots of a row alike.  (So it does by
// the roundings of the logits and of the teacher's rest themselves.  Sums in 64 bits as well cost
// short rows of 128 slots 4 to 10%.)
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
  float coef[3];                               // outside coefficient, any of it at all, maximum
};

// (From 96 * 16 vectors on; up to 288 * 9 three CTAs share an SM, up to 288 * 16 two, then there is one.)
// 4096 rows of 10000 / 16400 fp32 logits took 90 / 131 us, cut in segments as the longer ones 129 / 156;
// of 20000 / 36800 bf16 88 / 135 against 137 / 174; 2048 of 30400 fp32 125 against 135, of 76800 bf16
// 148 against 152; and 128 rows of 50257 bf16 16.4 against 30.7.
constexpr int kShortVectors = 608 * 16;  // of the longest row that lies in one CTA's registers

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

// The sides of a row's teacher slots: maxima and sums of the logits that count, and the
// teacher's rest.
struct SlotStats {
  float t_top, s_top, sum_t, sum_s, rho;
};
__device__ __forceinline__ float teacher_rest(const DistillArgs& a, int64_t n) {
  const float rho = a.teacher_rest != nullptr ? __ldg(a.teacher_rest + n) : 0.f;
  return rho < 0.f ? 0.f : (rho > 1.f ? 1.f : rho);  // (a NaN stays, and makes its row NaN)
}

// A row's events (one warp).  t, s, g: the slots' teacher and student logits, their gradients on
// return (t and s are overwritten with p and q).
struct RowEvents {
  float rho, m_out, sum_out, top, total, q_rest, sgn_r, S, kl, tv, wt;
  bool any;  // both sides have a distribution

  __device__ __forceinline__ RowEvents(const DistillArgs& a, float c, float w,
                                       const SlotStats& r, float m, float sum, float* t, float* s,
                                       float* g, int lane)
      : rho(r.rho), m_out(m), sum_out(sum) {
    top = max_nan(m_out, r.s_top);
    any = !(r.t_top == -INFINITY || top == -INFINITY);
    const float out_part = sum_out * part_scale(m_out, top, c);
    total = r.sum_s * part_scale(r.s_top, top, c) + out_part;
    const float inv = 1.f / total, p_scale = (1.f - rho) / r.sum_t;
    const float ratio = log2f(total) - log2f(r.sum_t) + log2f(1.f - rho);
    q_rest = out_part * inv;
    sgn_r = sign_of(q_rest, rho);  // (all it is made of are the sums)
    S = kl = tv = 0.f;
    for (int j = lane; j < a.k; j += 32) {
      const float tj = t[j], sj = s[j];
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
      t[j] = p;
      s[j] = q;
      g[j] = sg;
    }
    S = warp_sum(S) + sgn_r * q_rest;
    wt = w / a.temperature;
  }
  // of any other token v: coefficient * 2^((x_v - m_out) c), where there is one
  __device__ __forceinline__ float coefficient(const DistillArgs& a) const {
    return wt * (a.alpha_kl * (q_rest - rho) + 0.5f * a.alpha_tv * (sgn_r - S) * q_rest) / sum_out;
  }
  __device__ __forceinline__ bool outside() const { return any && sum_out != 0.f; }
  __device__ __forceinline__ float slot(const DistillArgs& a, float p, float q, float sg) const {
    return any ? wt * (a.alpha_kl * (q - p) + 0.5f * a.alpha_tv * (sg - S) * q) : 0.f;
  }
  __device__ __forceinline__ void write_loss(const DistillArgs& a, float c, int64_t n, float w,
                                             int lane) {
    kl = warp_sum(kl);
    tv = 0.5f * (warp_sum(tv) + fabsf(rho - q_rest));
    if (rho > 0.f)
      kl += rho * (log2f(rho) - log2f(sum_out) - (m_out - top) * c + log2f(total));
    if (lane == 0) {
      a.loss[n] = any ? w * ((a.alpha_kl != 0.f ? a.alpha_kl * kl * kLn2 : 0.f) + a.alpha_tv * tv)
                      : 0.f;
      if (a.tv != nullptr) a.tv[n] = any ? tv : 0.f;
    }
  }
};

template <typename T>
struct SlotWarp {
  const DistillArgs& a;
  const float c;
  SlotSmem& sm;
  uint32_t* map[2];
  int lane;

  struct Row : SlotStats {
    int64_t n;
    float w;
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
        record_error(a.status, kStatusDeviceOob);
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
    r.rho = teacher_rest(a, r.n);
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
  // Coefficients and loss from the outside's (maximum, sum).
  __device__ __forceinline__ void finish(const Row& r, int b, float m_out, float sum_out,
                                         int threads) {
    RowEvents ev(a, c, r.w, r, m_out, sum_out, sm.t[b], sm.s[b], sm.out_g[b], lane);
    if (a.grad != nullptr) {
      if (lane == 0) {
        sm.coef[0] = ev.coefficient(a);
        sm.coef[1] = ev.outside() ? 1.f : 0.f;
        sm.coef[2] = m_out;
      }
      __syncwarp();
      bar_arrive(kBarCoef, threads);
      for (int j = lane; j < a.k; j += 32) {
        sm.out_g[b][j] = ev.slot(a, sm.t[b][j], sm.s[b][j], sm.out_g[b][j]);
        sm.out_id[b][j] = sm.id[b][j];
      }
    }
    ev.write_loss(a, c, r.n, r.w, lane);
  }
  // The gradients of a finished row's slots, over what the streaming warps wrote there before
  // they arrived at a barrier that this warp has passed.
  __device__ __forceinline__ void patch(int64_t n, int b) const {
    T* grad = static_cast<T*>(a.grad) + n * a.ld_grad;
    for (int j = lane; j < a.k; j += 32) {
      const int id = sm.out_id[b][j];
      if (id >= 0) Row16<T>::put(grad + id, sm.out_g[b][j]);
    }
  }
};

// Short rows.  A CTA walks over rows; vector i of a streaming thread is the row's body vector
// tid + i * (threads - 32); all but the last kPartial of them are full (the host picks the threads
// so).  The up to 14 elements outside the body are single elements of warp 0's lanes.
template <typename T, int NV, int kPartial, int kMaxThreads, int kPerSm>
__global__ void __launch_bounds__(kMaxThreads, kPerSm)
    distill_short_kernel(const DistillArgs a, const float c, const int map_words, const uint2 sel) {
  using R = Row16<T>;
  constexpr int kVec = R::kVec;
  const int nt = blockDim.x, row_threads = nt - 32, row_warps = row_threads / 32;
  __shared__ SlotSmem sm;
  extern __shared__ uint32_t maps[];  // 2 x map_words

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t step = gridDim.x, n0 = blockIdx.x;
  const bool grads = a.grad != nullptr;
  for (int i = tid; i < 2 * map_words; i += nt) maps[i] = 0u;
  for (int i = tid; i < 2 * kMaxTeacher; i += nt) (&sm.pos[0][0])[i] = -1;
  __syncthreads();

  if (warp == row_warps) {  // ---------------------------------------------- the slot warp
    SlotWarp<T> sw{a, c, sm, {maps, maps + map_words}, lane};
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
      sw.finish(cur, b, m, sum, nt);
      if (grads && last.n < a.N)  // (the streaming warps were done with it at kBarSums)
        sw.patch(last.n, b ^ 1);
      last = cur;
      cur = nxt;
      nxt = after;
      if (grads && cur.n >= a.N) {
        bar_sync(kBarSums, nt);  // the streaming warps have written the last row
        sw.patch(last.n, b);
      }
    }
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
    const int cnt = sp.body;
    const uint4* src = reinterpret_cast<const uint4*>(row + sp.head) + tid;
    T* dst = grad + sp.head + static_cast<int64_t>(tid) * kVec;
    const bool aligned = (reinterpret_cast<uintptr_t>(grad + sp.head) & 15u) == 0;
    // this thread's single element, if it has one
    int edge = -1;
    if (tid < 16) {
      if (tid < sp.head) edge = tid;
      if (tid >= 8 && tid - 8 < sp.tail) edge = a.V - sp.tail + tid - 8;
    }
    const auto has = [&](int i) { return i < NV - kPartial || tid + i * row_threads < cnt; };
    const auto store = [&](int i, const uint4& g) {
      if (aligned) {
        __stcs(reinterpret_cast<uint4*>(dst) + i * row_threads, g);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) dst[i * row_threads * kVec + e] = R::get(g, e);
      }
    };
    if (w == 0.f) {  // neither read nor looked at
      if (tid == 0) {
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
      const int p0 = tid + (sp.off > 0 ? 1 : 0);
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
}

// ---- long rows
constexpr int kLongWarps = 8;               // that stream, and one more for the service
constexpr int kLongThreads = kLongWarps * 32 + 32;
constexpr int kLongEach = 4;                // vectors of a lane in a ring's slot
constexpr int kLongSlot = 32 * kLongEach;   // vectors of a slot
constexpr int kLongRing = 4;                // slots in shared memory, one worked on
// Vectors of a segment that the rows' cut starts from; the count that divides the warps may then leave
// up to 784 fp32 and 1408 bf16, and few rows are cut down to a slot's 128 (see the dispatch).  A
// segment costs a warp some 500 instructions beside its logits,
// but what is summed in a round has to be in L2 when the gradient reads it: 2048 x 151936 rows
// took, cut in 32 / 38 / 64 segments, fp32 517 / 460 / 446 us and, in 16 / 19 / 24 / 32, bf16
// 283 / 272 / 286 / 290 us (loss alone 70 / 68 / - / 73 us).
template <typename T>
constexpr int kLongSegment = sizeof(T) == 4 ? 608 : 1024;
constexpr int kHash = 2 * kMaxTeacher;

// Values that pass between CTAs carry the launch's tag beside them in one 8-byte word, so a reader
// that sees the tag sees the value.
__device__ __forceinline__ void publish(unsigned long long* p, uint32_t tag, float x) {
  *reinterpret_cast<volatile unsigned long long*>(p) =
      static_cast<unsigned long long>(tag) << 32 | __float_as_uint(x);
}
// Wait for kN consecutive words of this launch, read together; false after `timeout_ns` or once
// *abort is set.  Orders nothing that follows (see `acquire`).
template <int kN>
__device__ __forceinline__ bool await(const unsigned long long* p, uint32_t tag, float (&x)[kN],
                                      uint64_t timeout_ns, volatile int* abort) {
  uint64_t deadline = 0;
  for (uint32_t spins = 1;; ++spins) {
    unsigned long long v[kN];
    bool there = true;
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = *const_cast<const volatile unsigned long long*>(p + i);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      there = there && static_cast<uint32_t>(v[i] >> 32) == tag;
      x[i] = __uint_as_float(static_cast<uint32_t>(v[i]));
    }
    if (there) return true;
    if ((spins & 31u) != 0u) continue;
    if (*abort != 0) return false;
    const uint64_t now = globaltimer_ns();
    if (deadline == 0) {
      deadline = now + timeout_ns;
    } else if (now > deadline) {
      *abort = 1;
      return false;
    }
  }
}
// What the writer of a word seen by `await` wrote before it is visible after this.
__device__ __forceinline__ void acquire(const unsigned long long* p) {
  asm volatile("{\n\t.reg .b64 v;\n\tld.acquire.gpu.global.u64 v, [%0];\n\t}" ::"l"(p) : "memory");
}

struct LongSmem {
  uint4 ring[kLongWarps][kLongRing][kLongSlot];
  int2 list[kLongWarps][kMaxTeacher];  // a warp's segment's teacher tokens, and their gradients
  // the service warp's row
  int id[kMaxTeacher];
  float t[kMaxTeacher], s[kMaxTeacher], g[kMaxTeacher];
  int key[kHash], slot[kHash];  // tokens seen, and their first slots
  int abort;
};

// How rows are cut: S segments of `vecs` vectors (the last of a row has fewer); unit / S is the
// high word of unit * magic (unit * S is far below 2^32).
struct Split {
  int S, vecs;
  uint32_t magic;
};

// One of the row's segments: body vectors [v0, v0 + cnt) in `slots` slots; the first segment's
// warp has the elements outside the body as well.
template <typename T>
struct Segment {
  int64_t n;
  int index, v0, cnt, slots;
  const T* row;
  RowSpan<T> sp;
  __device__ __forceinline__ Segment(const DistillArgs& a, int unit, const Split& d)
      : n(static_cast<int64_t>(static_cast<uint64_t>(unit) * d.magic >> 32)),
        index(unit - static_cast<int>(n) * d.S),
        v0(index * d.vecs),
        row(static_cast<const T*>(a.logits) + n * a.ld),
        sp(row, a.V) {
    cnt = min(max(sp.body - v0, 0), d.vecs);
    slots = (cnt + kLongSlot - 1) / kLongSlot;
  }
  // this lane's single element, -1: none
  __device__ __forceinline__ int edge(int V, int lane) const {
    if (index != 0) return -1;
    if (lane < sp.head) return lane;
    return lane >= 8 && lane - 8 < sp.tail ? V - sp.tail + lane - 8 : -1;
  }
  // whether token `id` lies in this segment, edges among them
  __device__ __forceinline__ bool holds(int id) const {
    const int e = id - sp.head - v0 * Row16<T>::kVec;
    const bool body = id >= sp.head && id < sp.head + sp.body * Row16<T>::kVec;
    return body ? e >= 0 && e < cnt * Row16<T>::kVec : index == 0;
  }
};

template <typename T>
__global__ void __launch_bounds__(kLongThreads, 2)
    distill_long_kernel(const DistillArgs a, const float c, const Split split) {
  const int S = split.S;
  using R = Row16<T>;
  constexpr int kVec = R::kVec;
  extern __shared__ uint4 s_raw[];
  LongSmem& sm = *reinterpret_cast<LongSmem*>(s_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = a.k, V = a.V;
  const bool grads = a.grad != nullptr;
  const LongScratch& x = a.scratch;
  const uint32_t tag = __ldcg(x.epoch) + 1u;
  const auto weight = [&](int64_t n) { return a.row_weight != nullptr ? __ldg(a.row_weight + n) : 1.f; };
  if (threadIdx.x == 0) sm.abort = 0;
  __syncthreads();

  if (warp == kLongWarps) {  // ------------------------------------------- the service warp
    for (int i = lane; i < kHash; i += 32) {
      sm.key[i] = -1;
      sm.slot[i] = kMaxTeacher;
    }
    for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
      const float w = weight(n);
      if (w == 0.f) {
        if (lane == 0) {
          a.loss[n] = 0.f;
          if (a.tv != nullptr) a.tv[n] = 0.f;
        }
        continue;
      }
      const T* row = static_cast<const T*>(a.logits) + n * a.ld;
      // the slots that count: of equal tokens the first
      __syncwarp();
#pragma unroll 2
      for (int j = lane; j < k; j += 32) {
        int id = __ldg(a.teacher_ids + n * k + j);
        const float t = __ldg(a.teacher_logits + n * k + j);
        if (id >= V) {
          record_error(a.status, kStatusDeviceOob);
          id = -1;
        }
        sm.t[j] = t;
        sm.id[j] = id;
        sm.g[j] = id >= 0 ? R::one(row + id) : 0.f;
        if (id >= 0) {
          uint32_t h = (static_cast<uint32_t>(id) * 2654435761u) >> 23;
          for (;;) {
            const int old = atomicCAS(&sm.key[h], -1, id);
            if (old == -1 || old == id) break;
            h = (h + 1u) & (kHash - 1);
          }
          atomicMin(&sm.slot[h], j);
          sm.s[j] = __uint_as_float(h);
        }
      }
      __syncwarp();
      SlotStats st{-INFINITY, -INFINITY, 0.f, 0.f, teacher_rest(a, n)};
      uint32_t counts = 0u;
      for (int i = 0, j = lane; j < k; ++i, j += 32)
        if (sm.id[j] >= 0 && sm.slot[__float_as_uint(sm.s[j])] == j) counts |= 1u << i;
      __syncwarp();
      for (int i = 0, j = lane; j < k; ++i, j += 32) {
        if (sm.id[j] >= 0) {  // the table as it was
          const uint32_t h = __float_as_uint(sm.s[j]);
          sm.key[h] = -1;
          sm.slot[h] = kMaxTeacher;
        }
        const bool in = counts >> i & 1u;
        if (!in) sm.id[j] = -1;
        sm.t[j] = in ? sm.t[j] : -INFINITY;
        sm.s[j] = in ? sm.g[j] : -INFINITY;
        st.t_top = max_nan(st.t_top, sm.t[j]);
        st.s_top = max_nan(st.s_top, sm.s[j]);
      }
      st.t_top = warp_max(st.t_top);
      st.s_top = warp_max(st.s_top);
      for (int j = lane; j < k; j += 32) {
        st.sum_t += part_scale(sm.t[j], st.t_top, c);
        st.sum_s += part_scale(sm.s[j], st.s_top, c);
      }
      st.sum_t = warp_sum(st.sum_t);
      st.sum_s = warp_sum(st.sum_s);
      // the segments' sums
      float m = -INFINITY, sum = 0.f;
      bool ok = true;
      for (int i = lane; i < S; i += 32) {
        float part[2] = {-INFINITY, 0.f};
        const unsigned long long* p = x.part + (n * kLongMaxSegments + i) * 2;
        ok = ok && await(p, tag, part, a.timeout_ns, &sm.abort);
        const float top = max_nan(m, part[0]);
        sum = sum * part_scale(m, top, c) + part[1] * part_scale(part[0], top, c);
        m = top;
      }
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        if (lane == 0) record_error(a.status, kStatusTimeout);
        break;
      }
      const float m_out = warp_max(m);
      const float sum_out = warp_sum(sum * part_scale(m, m_out, c));
      RowEvents ev(a, c, w, st, m_out, sum_out, sm.t, sm.s, sm.g, lane);
      if (grads) {
        for (int j = lane; j < k; j += 32)
          x.list[n * kMaxTeacher + j] =
              make_int2(sm.id[j], __float_as_int(ev.slot(a, sm.t[j], sm.s[j], sm.g[j])));
        __syncwarp();
        if (lane == 0) {
          __threadfence();
          unsigned long long* p = x.coef + n * 3;
          publish(p, tag, ev.coefficient(a));
          publish(p + 1, tag, m_out);
          publish(p + 2, tag, ev.outside() ? 1.f : 0.f);
        }
      }
      ev.write_loss(a, c, n, w, lane);
    }
  } else {  // -------------------------------------------------------- the streaming warps
    const int units = static_cast<int>(a.N) * S, step = gridDim.x * kLongWarps;
    const int u0 = warp * gridDim.x + blockIdx.x;
    const int own = u0 < units ? (units - u0 + step - 1) / step : 0;  // this warp's units
    // Tasks in turn: sum(0), -, sum(1), gradient(0), sum(2), gradient(1), ...; -1: none.  (Units
    // taken from a counter as warps get to them, which would even out rows of no weight, were no
    // faster: the waits for the counter and the bookkeeping cost what they gave.)
    const int tasks = grads ? 2 * (own + 1) : own;
    const auto is_sum = [&](int t) { return !grads || (t & 1) == 0; };
    const auto unit_of = [&](int t) {
      const int i = grads ? (t >> 1) - (t & 1) : t;
      return i < own ? i : -1;
    };
    const auto live = [&](int64_t n) { return weight(n) != 0.f; };
    const uint32_t ring = smem_addr(&sm.ring[warp][0][lane]);
    constexpr uint32_t kSlotBytes = kLongSlot * 16;
    // the copies run ahead of the work by kLongRing - 1 slots, over the tasks' ends
    // What is read for the last time leaves L2 first: 2048 x 151936 fp32 466 -> 446 us, 34 -> 7% of
    // the second reading from DRAM.  bf16 is faster without (271 against 291 us).
    constexpr bool kHint = sizeof(T) == 4;
    const uint64_t policy_again = l2_policy_evict_normal(), policy_last = l2_policy_evict_first();
    uint64_t f_policy = policy_last;
    int f_task = -1, f_left = 0, f_rest = 0;
    uint32_t f_to = 0;
    const uint4* f_src = nullptr;
    const auto advance = [&]() {  // to the next task that has something to copy
      while (f_left == 0 && f_task + 1 < tasks) {
        ++f_task;
        const int i = unit_of(f_task);
        if (i < 0) continue;
        const Segment<T> g(a, u0 + i * step, split);
        if (!live(g.n)) continue;
        f_left = g.slots;
        if (kHint) f_policy = grads && is_sum(f_task) ? policy_again : policy_last;
        f_rest = g.cnt - lane;
        f_src = reinterpret_cast<const uint4*>(g.row + g.sp.head) + g.v0 + lane;
      }
    };
    const auto fetch = [&]() {
      if (f_left == 0) advance();
      if (f_left > 0) {
#pragma unroll
        for (int e = 0; e < kLongEach; ++e)
          if (f_rest > 32 * e) {
            if (kHint)
              asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(
                               ring + f_to + 512 * e),
                           "l"(f_src + 32 * e), "l"(f_policy)
                           : "memory");
            else
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring + f_to + 512 * e),
                           "l"(f_src + 32 * e)
                           : "memory");
          }
        f_src += kLongSlot;
        f_rest -= kLongSlot;
        f_to = (f_to + kSlotBytes) & (kLongRing * kSlotBytes - 1);
        --f_left;
      }
      cp_async_commit();
    };
    uint32_t from = 0;
    const auto next_slot = [&](uint4 (&v)[kLongEach]) {
      fetch();
      cp_async_wait_group<kLongRing - 1>();
#pragma unroll
      for (int e = 0; e < kLongEach; ++e)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[e].x), "=r"(v[e].y), "=r"(v[e].z), "=r"(v[e].w)
                     : "r"(ring + from + 512 * e)
                     : "memory");
      from = (from + kSlotBytes) & (kLongRing * kSlotBytes - 1);
    };
#pragma unroll 1
    for (int i = 0; i < kLongRing - 1; ++i) fetch();

    const F2 scale(c, c);
    const uint4 nothing = make_uint4(R::kNegInf, R::kNegInf, R::kNegInf, R::kNegInf);
    for (int task = 0; task < tasks; ++task) {
      const int i = unit_of(task);
      if (i < 0) continue;
      const Segment<T> g(a, u0 + i * step, split);
      const int edge = g.edge(V, lane);
      const bool alive = live(g.n);
      if (is_sum(task)) {  // ---- the sum of a segment
        if (!alive) continue;
        // the teacher's tokens of this segment
        float xe = edge >= 0 ? R::one(g.row + edge) : -INFINITY;
        int listed_n = 0;
        uint32_t listed = 0u;  // slots with any
        for (int j0 = 0; j0 < k; j0 += 32) {
          const int j = j0 + lane;
          const int id = j < k ? __ldg(a.teacher_ids + g.n * k + j) : -1;
          const bool in = id >= 0 && id < V && g.holds(id);
          const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, in);
          if (in) {
            sm.list[warp][listed_n + __popc(lanes & ((1u << lane) - 1u))] = make_int2(id, 0);
            const int e = id - g.sp.head - g.v0 * kVec;
            if (e >= 0 && e < g.cnt * kVec) listed |= 1u << (e / (kLongSlot * kVec));
          }
          listed_n += __popc(lanes);
        }
        listed = __reduce_or_sync(0xFFFFFFFFu, listed);
        __syncwarp();
        if (g.index == 0 && g.sp.head + g.sp.tail > 0)
          for (int j = 0; j < listed_n; ++j)
            if (sm.list[warp][j].x == edge) xe = -INFINITY;
        float m = xe, sum = xe == -INFINITY ? 0.f : 1.f;
        if (!(xe == xe)) sum = xe;
        const auto add = [&](uint4 (&v)[kLongEach], int s) {
          if (listed >> s & 1u) {
            uint32_t bits[kLongEach] = {};
            for (int j = 0; j < listed_n; ++j) {
              const int e = sm.list[warp][j].x - g.sp.head - (g.v0 + s * kLongSlot + lane) * kVec;
#pragma unroll
              for (int h = 0; h < kLongEach; ++h)
                if (e >= 32 * h * kVec && e < (32 * h + 1) * kVec) bits[h] |= 1u << (e - 32 * h * kVec);
            }
#pragma unroll
            for (int h = 0; h < kLongEach; ++h)
              if (bits[h] != 0u) R::mask(v[h], bits[h]);
          }
          float top = max_nan(m, R::max8(v[0], v[1]));
#pragma unroll
          for (int h = 2; h < kLongEach; h += 2) top = max_nan(top, R::max8(v[h], v[h + 1]));
          if (__any_sync(0xFFFFFFFFu, !(top == m))) {
            sum *= part_scale(m, top, c);
            m = top;
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const F2 minus(-ref, -ref);
          F2 acc[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < kLongEach; ++h)
#pragma unroll
            for (int p = 0; p < R::kPairs; ++p) {
              float y0, y1;
              ((R::pair(v[h], p) + minus) * scale).get(y0, y1);
              acc[h & 1] = acc[h & 1] + F2(ex2_approx(y0), ex2_approx(y1));
            }
          float y0, y1;
          (acc[0] + acc[1]).get(y0, y1);
          sum += y0 + y1;
        };
        const int full = g.cnt / kLongSlot;
        for (int s = 0; s < full; ++s) {
          uint4 v[kLongEach];
          next_slot(v);
          add(v, s);
        }
        if (full < g.slots) {
          uint4 v[kLongEach];
          next_slot(v);
          const int left = g.cnt - full * kLongSlot - lane;
#pragma unroll
          for (int h = 0; h < kLongEach; ++h)
            if (left <= 32 * h) v[h] = nothing;
          add(v, full);
        }
        const float top = warp_max(m);
        sum = warp_sum(sum * part_scale(m, top, c));
        const bool skip = task == 0 && static_cast<int>(blockIdx.x) == a.debug_skip_cta;
        if (lane == 0 && !skip) {
          unsigned long long* p = x.part + (g.n * kLongMaxSegments + g.index) * 2;
          publish(p, tag, top);
          publish(p + 1, tag, sum);
        }
        __syncwarp();  // (the list is read before the next sum writes it)
        continue;
      }
      // ---- the gradient of a segment
      float of_row[3] = {0.f, 0.f, 0.f};  // its row's coefficient, maximum, any outside
      if (alive) {
        const bool ok = await(x.coef + g.n * 3, tag, of_row, a.timeout_ns, &sm.abort);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          if (lane == 0) record_error(a.status, kStatusTimeout);
          break;
        }
      }
      T* grad = static_cast<T*>(a.grad) + g.n * a.ld_grad;
      T* dst = grad + g.sp.head + static_cast<int64_t>(g.v0 + lane) * kVec;
      const bool aligned = (reinterpret_cast<uintptr_t>(grad + g.sp.head) & 15u) == 0;
      const auto store = [&](int vec, const uint4& y) {  // wherever the gradient's rows start
        if (aligned) {
          __stcs(reinterpret_cast<uint4*>(dst) + vec, y);
        } else {
#pragma unroll
          for (int e = 0; e < kVec; ++e) dst[vec * kVec + e] = R::get(y, e);
        }
      };
      const uint4 zeros = make_uint4(0u, 0u, 0u, 0u);
      if (!alive) {  // a row of no weight, neither read nor looked at
        for (int v = 0; v + lane < g.cnt; v += 32) store(v, zeros);
        if (edge >= 0) R::put(grad + edge, 0.f);
        continue;
      }
      const float coef = of_row[0], any = of_row[2];
      const float ref = of_row[1] == -INFINITY ? 0.f : of_row[1];
      const F2 minus(-ref, -ref), mul(coef, coef);
      const float xe = edge >= 0 ? R::one(g.row + edge) : 0.f;
      const auto gradient = [&](const uint4& v, auto exp2_of) {
        uint4 y;
#pragma unroll
        for (int p = 0; p < R::kPairs; ++p) {
          float y0, y1;
          ((R::pair(v, p) + minus) * scale).get(y0, y1);
          (F2(exp2_of(y0), exp2_of(y1)) * mul).get(y0, y1);
          R::set_pair(y, p, y0, y1);
        }
        return y;
      };
      // The common case first.  Apart from it, in little code: a gradient that starts elsewhere
      // in 16 bytes than the logits; a coefficient above one, which brings results below 2^-126,
      // dropped by the fast exponential, back into range; no token outside with any probability.
      const bool common = aligned && any != 0.f && fabsf(coef) <= 1.f;
      int s = 0;
      if (common)
        for (int left = g.cnt - lane; s < g.slots; ++s, left -= kLongSlot) {
          uint4 v[kLongEach];
          next_slot(v);
#pragma unroll
          for (int h = 0; h < kLongEach; ++h) {
            const uint4 y = gradient(v[h], [](float y) { return ex2_approx(y); });
            if (left > 32 * h)
              __stcs(reinterpret_cast<uint4*>(dst) + s * kLongSlot + 32 * h, y);
          }
        }
#pragma unroll 1
      for (; s < g.slots; ++s) {
        uint4 v[kLongEach];
        next_slot(v);
        const int left = g.cnt - s * kLongSlot - lane;
#pragma unroll 1
        for (int h = 0; h < kLongEach; ++h) {
          const uint4 w = h == 0 ? v[0] : h == 1 ? v[1] : h == 2 ? v[2] : v[3];
          uint4 y = zeros;
          if (any != 0.f) y = gradient(w, [](float y) { return exp2f(y); });
          if (left > 32 * h) store(s * kLongSlot + 32 * h, y);
        }
      }
      if (edge >= 0) R::put(grad + edge, any != 0.f ? exp2f((xe - ref) * c) * coef : 0.f);
      // the teacher's tokens of this segment, over what is there now
      acquire(x.coef + g.n * 3);
      __syncwarp();
      for (int j = lane; j < k; j += 32) {
        const int2 e = __ldcg(x.list + g.n * kMaxTeacher + j);
        if (e.x >= 0 && g.holds(e.x)) R::put(grad + e.x, __int_as_float(e.y));
      }
    }
    cp_async_wait_all();  // (copies are left under way only where a wait ran out)
  }
  __syncthreads();
  if (threadIdx.x == 0) {  // the launch's last CTA moves the tag on
    __threadfence();
    if (atomicAdd(x.done, 1u) == gridDim.x - 1) {
      *x.done = 0u;
      *x.epoch = tag;
    }
  }
}

template <typename T, int NV, int kPartial, int kMaxThreads, int kPerSm>
cudaError_t launch_short(const DistillArgs& a, int row_threads, int num_sms, cudaStream_t stream) {
  const auto fn = distill_short_kernel<T, NV, kPartial, kMaxThreads, kPerSm>;
  const int map_words = (a.V + 2 * Row16<T>::kVec + 31) / 32;
  const float c = static_cast<float>(1.4426950408889634 / static_cast<double>(a.temperature));
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>(a.N, static_cast<int64_t>(num_sms) * kPerSm));
  fn<<<grid, row_threads + 32, 2 * 4 * map_words, stream>>>(a, c, map_words,
                                                             make_uint2(0x1044u, 0x3244u));
  return cudaGetLastError();
}

// Streaming threads that hold `most` vectors in nv each with all but the last `partial` full
// where there are `least` (0: none up to `limit` do).
int threads_for(int nv, int partial, int most, int least, int limit) {
  const int t = (((most + nv - 1) / nv + 31) / 32) * 32;
  return t <= limit && (nv - partial) * t <= least ? std::max(t, 32) : 0;
}

template <typename T>
cudaError_t dispatch(const DistillArgs& all, int num_sms, uint32_t extra_smem, SmemOptIn& opt_in,
                     int* launches, cudaStream_t stream) {
  constexpr int kVec = Row16<T>::kVec;
  // 16-byte vectors of a row: a row that starts off a boundary has one less
  const int body = all.V / kVec, body_least = std::max(0, (all.V - kVec + 1) / kVec);
  const int most = std::max(1, body), least = body_least;
  int t;
  if (body <= kShortVectors) {
    *launches += 1;
    // Few threads with many vectors while they hold the row: a row is bound by its slot warp's
    // chain, and small CTAs bring more of those to an SM.  4096 rows, 128 slots, in three warps
    // against up to nine: 9120 bf16 logits 70 -> 61 us, 15400 78 -> 64, 24000 86 -> 76; 6000 fp32
    // 88 -> 74 (loss alone 70 -> 53).
    if ((t = threads_for(1, 1, most, least, 96)))
      return launch_short<T, 1, 1, 128, 6>(all, t, num_sms, stream);
    if ((t = threads_for(2, 1, most, least, 96)))
      return launch_short<T, 2, 1, 128, 6>(all, t, num_sms, stream);
    if ((t = threads_for(3, 1, most, least, 96)))
      return launch_short<T, 3, 1, 128, 6>(all, t, num_sms, stream);
    if ((t = threads_for(4, 1, most, least, 96)))
      return launch_short<T, 4, 1, 128, 6>(all, t, num_sms, stream);
    if ((t = threads_for(6, 2, most, least, 96)))
      return launch_short<T, 6, 2, 128, 6>(all, t, num_sms, stream);
    if ((t = threads_for(8, 2, most, least, 96)))
      return launch_short<T, 8, 2, 128, 6>(all, t, num_sms, stream);
    if ((t = threads_for(16, 6, most, least, 96)))
      return launch_short<T, 16, 6, 128, 4>(all, t, num_sms, stream);
    if ((t = threads_for(9, 2, most, least, 288)))
      return launch_short<T, 9, 2, 320, 3>(all, t, num_sms, stream);
    if ((t = threads_for(12, 2, most, least, 288)))
      return launch_short<T, 12, 2, 320, 2>(all, t, num_sms, stream);
    if ((t = threads_for(16, 2, most, least, 288)))
      return launch_short<T, 16, 2, 320, 2>(all, t, num_sms, stream);
    t = threads_for(16, 2, most, least, 608);
    return launch_short<T, 16, 2, 640, 1>(all, t, num_sms, stream);
  }
  const auto fn = distill_long_kernel<T>;
  cudaError_t e = opt_in(fn, static_cast<int>(sizeof(LongSmem)));
  if (e != cudaSuccess) return e;
  for (int64_t n0 = 0; n0 < all.N; n0 += kLongMaxRows) {  // as many rows as there is scratch for
    DistillArgs a = all;
    a.N = std::min<int64_t>(kLongMaxRows, all.N - n0);
    a.logits = static_cast<const T*>(a.logits) + n0 * a.ld;
    if (a.grad != nullptr) a.grad = static_cast<T*>(a.grad) + n0 * a.ld_grad;
    a.teacher_ids += n0 * a.k;
    a.teacher_logits += n0 * a.k;
    if (a.teacher_rest != nullptr) a.teacher_rest += n0;
    if (a.row_weight != nullptr) a.row_weight += n0;
    a.loss += n0;
    if (a.tv != nullptr) a.tv += n0;
    // shorter segments (a slot at least) while there are warps without any
    int S = std::min(kLongMaxSegments, (body + kLongSegment<T> - 1) / kLongSegment<T>);
    const int64_t warps = 2ll * num_sms * kLongWarps;
    while (S < kLongMaxSegments && a.N * S < warps && body / (2 * S) >= kLongSlot) S *= 2;
    S = std::min(S, kLongMaxSegments);
    // With more units than warps, a count that divides the warps: a round of units is then whole
    // rows, and no sum waits a round for the rest of its row (2048 x 151936, 63 against 64
    // segments fp32, without hints to L2: 536 and 472 us; 28 against 32 bf16: 309
    // and 284).  The nearest one.
    if (a.N * S > warps) {
      int near = 1;
      for (int d = 2; d <= kLongMaxSegments; ++d)
        if (warps % d == 0 && std::max(d, S) * std::min(near, S) < std::max(near, S) * std::min(d, S))
          near = d;
      S = near;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * num_sms);
    cfg.blockDim = dim3(kLongThreads);
    cfg.dynamicSmemBytes = sizeof(LongSmem) + extra_smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const float c = static_cast<float>(1.4426950408889634 / static_cast<double>(a.temperature));
    const Split split{S, (body + S - 1) / S, static_cast<uint32_t>((1ull << 32) / S + 1)};
    e = cudaLaunchKernelEx(&cfg, fn, a, c, split);
    if (e != cudaSuccess) return e;
    *launches += 1;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, int num_sms, uint32_t extra_smem,
                           SmemOptIn& opt_in, int* launches, cudaStream_t stream) {
  return a.dtype == DSPARK_F32
             ? dispatch<float>(a, num_sms, extra_smem, opt_in, launches, stream)
             : dispatch<uint16_t>(a, num_sms, extra_smem, opt_in, launches, stream);
}

}  // namespace dspark
