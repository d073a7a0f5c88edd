// rnn_scan.cu -- the RNN head's gated linear recurrence over given sequences, and its
// gradients.
//
// Source: DSpark explainer, "The RNN head"; the equations are this library's reading (as for
// the RNN draft):  a = sigmoid(za), g = sigmoid(zg) (1 where zg is absent),
//   s_t = a_t s_{t-1} + g_t e_t                         (channel by channel)
// and backwards, with ds the gradient of the states used outside the recurrence,
//   delta_t = ds_t + y_{t+1},  y_t = a_t delta_t,  y_L = ds_last,  ds0 = y_0
//   dza_t = delta_t s_{t-1} a_t (1 - a_t),  dzg_t = delta_t e_t g_t (1 - g_t),
//   de_t = delta_t g_t.
// A reset at t makes a_t zero and drops the earlier state, whatever it holds (an infinity or NaN
// before a reset stays before it).
//
// Both directions are a recurrence x_t = a_t x_{t-1} + b_t, so a span of steps acts on the
// value before it as x -> A x + S (A the product of its decays, S its end from zero).  A warp
// works on 8 steps of 32 lanes at a time (a lane is 4 bytes of channels: two bf16 or one fp32;
// lanes run over sequences and channels alike, so no channel count leaves lanes empty).  The
// steps arrive in shared memory by asynchronous copies, the next units' while this one is
// worked on, so loads are in flight all the time; a warp that does not start a sequence learns
// the value before its steps from the spans before them.  Three ways:
//   very many lanes: one warp walks a block of lanes alone, from s0 on.
//   many lanes:      a CTA's warps hold consecutive spans, exchange (A, S) through shared
//                    memory and walk over the sequence; the value after a tile stays with them.
//   few lanes, long: the walk alone would leave most SMs empty, so every sequence is cut into
//                    segments, one a warp.  One launch finds the segments' spans (forward from
//                    three, backward from two streams), walking each from its end, so that the
//                    steps the second launch starts with are the ones still in L2; the second
//                    folds the spans before its segment and walks it.
// The first two read every input once.  8192 x 16 x 256 bf16: forward 48 us (5.9 TB/s, 88% of a
// copy's rate), backward 93 us (6.0 TB/s); segments, 1 x 65536 x 256 fp32 with resets: forward 81 us
// (470 MB, 5.8 TB/s of what it moves), 4 x 16384 x 256 bf16: backward 63 us (335 MB, 5.3 TB/s).

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <cuda_bf16.h>

#include "async_copy.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "sm103.cuh"
#include "training.h"

namespace dspark {
namespace {

constexpr float kRsLog2e = 1.4426950408889634f;

// ---- lanes: kVec channels in one 32-bit word
template <typename T, int kVec>
__device__ __forceinline__ float channel(uint32_t w, int i) {
  if (sizeof(T) == 4) return __uint_as_float(w);
  return __uint_as_float(kVec == 2 && i == 1 ? w & 0xFFFF0000u : w << 16);
}
__device__ __forceinline__ void put_lane(float* p, const float (&x)[1]) { __stcs(p, x[0]); }
__device__ __forceinline__ void put_lane(uint16_t* p, const float (&x)[1]) {
  __stcs(p, __bfloat16_as_ushort(__float2bfloat16_rn(x[0])));
}
__device__ __forceinline__ void put_lane(uint16_t* p, const float (&x)[2]) {
  uint32_t r;  // one rounding to bf16, to nearest even, where a value leaves the recurrence
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x[1]), "f"(x[0]));
  __stcs(reinterpret_cast<uint32_t*>(p), r);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two gates: sigmoid(z), exact zero and one at the far ends.
__device__ __forceinline__ void gates(float z0, float z1, float& a0, float& a1) {
  float y0, y1;
  (F2(z0, z1) * F2(-kRsLog2e, -kRsLog2e)).get(y0, y1);
  (F2(1.f, 1.f) + F2(ex2_approx(y0), ex2_approx(y1))).get(y0, y1);
  a0 = rcp_approx(y0);
  a1 = rcp_approx(y1);
}
// and their derivatives to full relative precision: with t = e^-|z| and r = 1 / (1 + t) the two
// sides of a gate are r and t r, the derivative t r^2.  t is the square of e^(-|z| / 2), which
// keeps it down to the denormals that a product with a large gradient brings back into range.
__device__ __forceinline__ void gates(float z0, float z1, float& a0, float& a1, float& slope0,
                                      float& slope1) {
  float y0, y1, l0, l1;
  (F2(fabsf(z0), fabsf(z1)) * F2(-0.5f * kRsLog2e, -0.5f * kRsLog2e)).get(y0, y1);
  const F2 h(ex2_approx(y0), ex2_approx(y1)), t = h * h;
  fma2(h, h, F2(1.f, 1.f)).get(y0, y1);
  y0 = rcp_approx(y0);
  y1 = rcp_approx(y1);
  const F2 r(y0, y1), low = t * r;
  (low * r).get(slope0, slope1);
  low.get(l0, l1);
  a0 = z0 >= 0.f ? y0 : l0;
  a1 = z1 >= 0.f ? y1 : l1;
}

// Spans.  kDrops in A: a reset inside, so the value before is dropped (a product that has merely
// underflowed keeps an infinity or NaN).
constexpr float kDrops = -1.f;
using Span = ScanSpan;
__device__ __forceinline__ float apply(Span f, float x) {
  return f.A == kDrops ? f.S : fmaf(f.A, x, f.S);
}
__device__ __forceinline__ Span then(Span f, Span g) {  // f first
  return {f.A == kDrops || g.A == kDrops ? kDrops : f.A * g.A, apply(g, f.S)};
}

// What a launch does with the sequences (see above).
enum class Mode { kWalk, kSpans, kSegments };

// ---- the two directions: their streams, their step's (a, b), and what a step writes
struct Stream {
  const void* p;
  int64_t ld;  // elements between rows
  int shift;   // rows back (the state before a step)
};

// Values of kSteps steps of a lane's channels, [step][channel], are worked on two at a time: the
// two channels of a step, or one channel of two steps.
template <typename T, int kVec, int kSteps>
struct Values {
  float v[kSteps * kVec];
  __device__ __forceinline__ void read(const uint32_t* words) {
#pragma unroll
    for (int k = 0; k < kSteps * kVec; ++k) v[k] = channel<T, kVec>(words[k / kVec * 32], k % kVec);
  }
  __device__ __forceinline__ void to_gates() {
#pragma unroll
    for (int k = 0; k < kSteps * kVec; k += 2) gates(v[k], v[k + 1], v[k], v[k + 1]);
  }
  __device__ __forceinline__ void to_gates(Values& slope) {
#pragma unroll
    for (int k = 0; k < kSteps * kVec; k += 2)
      gates(v[k], v[k + 1], v[k], v[k + 1], slope.v[k], slope.v[k + 1]);
  }
  __device__ __forceinline__ void times(const Values& o) {
#pragma unroll
    for (int k = 0; k < kSteps * kVec; k += 2)
      (F2(v[k], v[k + 1]) * F2(o.v[k], o.v[k + 1])).get(v[k], v[k + 1]);
  }
};
// x <- a x + b and products over a step's channels (explicit fused steps: what the compiler would
// fuse by itself differs between instances)
__device__ __forceinline__ void step(const float* a, const float* b, float (&x)[1]) {
  x[0] = fmaf(a[0], x[0], b[0]);
}
__device__ __forceinline__ void step(const float* a, const float* b, float (&x)[2]) {
  fma2(F2(a[0], a[1]), F2(x[0], x[1]), F2(b[0], b[1])).get(x[0], x[1]);
}
__device__ __forceinline__ void mul(const float (&x)[1], const float* y, float (&r)[1]) {
  r[0] = __fmul_rn(x[0], y[0]);
}
__device__ __forceinline__ void mul(const float (&x)[2], const float* y, float (&r)[2]) {
  (F2(x[0], x[1]) * F2(y[0], y[1])).get(r[0], r[1]);
}

template <typename T, int kVec>
struct Forward {
  using Args = RnnScanArgs;
  static constexpr bool kReverse = false;
  static constexpr int kStreams = 3, kWarps = 8, kSteps = 8;
  // units in shared memory of a warp: the one worked on and the ones on their way
  static constexpr __host__ __device__ int stages(Mode) { return 4; }
  static __device__ __forceinline__ Stream stream(const Args& p, int i) {
    return i == 0 ? Stream{p.za, p.ld_za, 0} : i == 1 ? Stream{p.zg, p.ld_zg, 0}
                                                      : Stream{p.e, p.ld_e, 0};
  }
  // the place of a stream among those copied (spans may need fewer), -1: none
  static constexpr __host__ __device__ int streams(Mode) { return 3; }
  static constexpr __device__ int place(Mode, int i) { return i; }
  static __device__ __forceinline__ const float* first(const Args& p) { return p.s0; }

  // words: [stream][step][lane] of this warp, at this lane.  a < 0: a reset.
  Values<T, kVec, kSteps> a, b;
  template <Mode kMode, bool kReset>
  __device__ __forceinline__ void read(const Args& p, const uint32_t* words, uint32_t resets,
                                       int steps) {
    b.read(words + 2 * kSteps * 32);
    if (p.zg != nullptr) {
      a.read(words + kSteps * 32);
      a.to_gates();
      b.times(a);
    }
    a.read(words);
    a.to_gates();
    if (kReset && resets != 0u) {
#pragma unroll
      for (int k = 0; k < kSteps * kVec; ++k)
        if (resets >> (k / kVec) & 1u) a.v[k] = kDrops;
    }
    if (steps < kSteps) {  // a step past the end changes nothing
#pragma unroll
      for (int k = 0; k < kSteps * kVec; ++k)
        if (k / kVec >= steps) a.v[k] = 1.f, b.v[k] = 0.f;
    }
  }
  template <bool kReset>
  __device__ __forceinline__ void span(Span (&f)[kVec]) const {
    float A[kVec], S[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      A[i] = 1.f;
      S[i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (kReset) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const Span g = then(Span{A[i], S[i]}, Span{a.v[j * kVec + i], b.v[j * kVec + i]});
          A[i] = g.A;
          S[i] = g.S;
        }
      } else {
        mul(A, a.v + j * kVec, A);
        step(a.v + j * kVec, b.v + j * kVec, S);
      }
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = {A[i], S[i]};
  }
  template <bool kReset, bool kFull>
  __device__ __forceinline__ void run(const Args& p, const uint32_t*, uint32_t, int64_t n, int d,
                                      int64_t t0, int steps, float (&x)[kVec]) const {
    T* s = static_cast<T*>(p.s) + (n * p.L + t0) * p.D + d;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (!kFull && j >= steps) break;
      if (kReset) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = apply(Span{a.v[j * kVec + i], b.v[j * kVec + i]}, x[i]);
      } else {
        step(a.v + j * kVec, b.v + j * kVec, x);
      }
      put_lane(s + static_cast<int64_t>(j) * p.D, x);
    }
    if (p.s_last != nullptr && t0 + steps == p.L && (kFull || steps > 0))
#pragma unroll
      for (int i = 0; i < kVec; ++i) p.s_last[n * p.D + d + i] = x[i];
  }
};

template <typename T, int kVec>
struct Backward {
  using Args = RnnScanGradArgs;
  static constexpr bool kReverse = true;
  static constexpr int kStreams = 5, kWarps = 8, kSteps = 8;
  static constexpr __host__ __device__ int stages(Mode m) { return m == Mode::kSpans ? 5 : 2; }
  static __device__ __forceinline__ Stream stream(const Args& p, int i) {
    return i == 0   ? Stream{p.za, p.ld_za, 0}
           : i == 1 ? Stream{p.zg, p.ld_zg, 0}
           : i == 2 ? Stream{p.e, p.ld_e, 0}
           : i == 3 ? Stream{p.ds, p.D, 0}
                    : Stream{p.s, p.D, 1};
  }
  static constexpr __host__ __device__ int streams(Mode m) { return m == Mode::kSpans ? 2 : 5; }
  static constexpr __device__ int place(Mode m, int i) {
    return m != Mode::kSpans ? i : i == 0 ? 0 : i == 3 ? 1 : -1;
  }
  static __device__ __forceinline__ const float* first(const Args& p) { return p.ds_last; }

  Values<T, kVec, kSteps> a, slope, ds;
  uint32_t drop;
  int count;
  template <Mode kMode, bool kReset>
  __device__ __forceinline__ void read(const Args&, const uint32_t* words, uint32_t resets,
                                       int steps) {
    a.read(words);
    a.to_gates(slope);
    ds.read(words + place(kMode, 3) * kSteps * 32);
    drop = kReset ? resets : 0u;
    count = steps;
  }
  template <bool kReset>
  __device__ __forceinline__ void span(Span (&f)[kVec]) const {
    // y = a delta is kept as its two factors, so a step is one fused operation
    float A[kVec], an[kVec], delta[kVec], y[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      A[i] = an[i] = 1.f;
      delta[i] = 0.f;
    }
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      if (j >= count) continue;
      step(an, ds.v + j * kVec, delta);
      const bool reset = kReset && (drop >> j & 1u);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        an[i] = reset ? 0.f : a.v[j * kVec + i];
        if (reset) delta[i] = 0.f;
        if (kReset) A[i] = reset || A[i] == kDrops ? kDrops : A[i] * an[i];
      }
      if (!kReset) mul(A, an, A);
    }
    mul(delta, an, y);
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = {A[i], y[i]};
  }
  template <bool kReset, bool kFull>
  __device__ __forceinline__ void run(const Args& p, const uint32_t* words, uint32_t resets,
                                      int64_t n, int d, int64_t t0, int steps, float (&x)[kVec]) {
    const int64_t r = n * p.L + t0;
    T* pa = static_cast<T*>(p.dza) + r * p.ld_dza + d;
    T* pg = static_cast<T*>(p.dzg) + r * p.ld_dzg + d;
    T* pe = static_cast<T*>(p.de) + r * p.D + d;
    const int ld_a = static_cast<int>(p.ld_dza), ld_g = static_cast<int>(p.ld_dzg);
    // the state before each step, then delta
    Values<T, kVec, kSteps> o;
    o.read(words + 4 * kSteps * 32);
    if (t0 == 0)
#pragma unroll
      for (int i = 0; i < kVec; ++i) o.v[i] = p.s0 != nullptr ? p.s0[n * p.D + d + i] : 0.f;
    float an[kVec], delta[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      an[i] = 1.f;
      delta[i] = x[i];
    }
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      if (!kFull && j >= steps) continue;
      const int k = j * kVec;
      const bool reset = kReset && (resets >> j & 1u);
      float y[kVec];
      step(an, ds.v + k, delta);
      mul(delta, o.v + k, y);
      mul(y, slope.v + k, y);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        o.v[k + i] = delta[i];
        an[i] = reset ? 0.f : a.v[k + i];
        if (reset) y[i] = delta[i] = 0.f;
      }
      put_lane(pa + static_cast<int64_t>(j) * ld_a, y);
    }
    mul(delta, an, x);
    if (p.dzg != nullptr) {
      Values<T, kVec, kSteps> e;
      a.read(words + kSteps * 32);
      a.to_gates(slope);
      e.read(words + 2 * kSteps * 32);
      e.times(o);
      e.times(slope);
      o.times(a);
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
        if (kFull || j < steps) {
          float y[kVec];
#pragma unroll
          for (int i = 0; i < kVec; ++i) y[i] = e.v[j * kVec + i];
          put_lane(pg + static_cast<int64_t>(j) * ld_g, y);
        }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      if (kFull || j < steps) {
        float y[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[i] = o.v[j * kVec + i];
        put_lane(pe + static_cast<int64_t>(j) * p.D, y);
      }
    if (p.ds0 != nullptr && t0 == 0 && (kFull || steps > 0))
#pragma unroll
      for (int i = 0; i < kVec; ++i) p.ds0[n * p.D + d + i] = x[i];
  }
};

// A unit of work of a warp: kSteps steps at place `pos` (counted in such, in the recurrence's
// order)
// of a lane block; block < 0: none.  Walks: a CTA's kWarps / W groups of W warps take every
// gridDim.x-th kWarps / W blocks, W places at a time.  Segments: the CTA's warps are consecutive
// segments of c.seg places of one block.
template <template <typename, int> class Dir, typename T, int kVec, Mode kMode, bool kReset>
__global__ void __launch_bounds__((Dir<T, kVec>::kWarps * 32), 2)
    scan_kernel(const typename Dir<T, kVec>::Args p, const ScanLaunch c) {
  using D = Dir<T, kVec>;
  constexpr int kWarps = D::kWarps, kSteps = D::kSteps, kStages = D::stages(kMode);
  constexpr int kWords = D::streams(kMode) * kSteps * 32;
  constexpr int kWarpWords = kWords + 32 * kVec;
  constexpr bool kWalk = kMode == Mode::kWalk;
  extern __shared__ uint4 s_raw[];  // [stage][warp] x (kWords words, 32 kVec floats)
  __shared__ Span s_span[2][kWarps][32 * kVec];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = kWalk ? c.W : 1, groups = kWarps / W, group = warp / W, order = warp % W;
  const int64_t places = (p.L + kSteps - 1) / kSteps;
  const uint32_t lanes = static_cast<uint32_t>(p.N * p.D);  // channels of all sequences
  const auto words = [&](int stage) {
    return reinterpret_cast<uint32_t*>(s_raw) + (stage * kWarps + warp) * kWarpWords;
  };
  // units: (block, pos), pos in steps of W (walk), up or (spans) down to `pos_end`
  struct Unit {
    int64_t block, pos;
  };
  int64_t pos_begin = order, pos_end = 0;
  Unit cur;
  if (kWalk) {
    cur = Unit{static_cast<int64_t>(blockIdx.x) * groups + group, pos_begin};
    pos_end = (places + W - 1) / W * W + order;  // every warp of a group does every turn
    if (cur.block - group >= c.blocks) cur.block = -1;
  } else {
    const int per = c.segs / kWarps;  // CTAs a block
    const int64_t seg = static_cast<int64_t>(blockIdx.x % per) * kWarps + warp;
    pos_begin = seg * c.seg;
    pos_end = pos_begin + c.seg < places ? pos_begin + c.seg : places;
    cur = Unit{blockIdx.x / per, kMode == Mode::kSpans ? pos_end - 1 : pos_begin};
    if (pos_begin >= places) cur.block = -1;
  }
  const auto after = [&](Unit u) {
    if (u.block < 0) return u;
    if (kWalk) {
      u.pos += W;
      if (u.pos >= pos_end) {
        u.pos = pos_begin;
        u.block += static_cast<int64_t>(gridDim.x) * groups;
        if (u.block - group >= c.blocks) u.block = -1;
      }
    } else {
      u.pos += kMode == Mode::kSpans ? -1 : 1;
      if (u.pos < pos_begin || u.pos >= pos_end) u.block = -1;
    }
    return u;
  };
  const auto start = [&](const Unit& u) {  // first step
    return (D::kReverse ? places - 1 - u.pos : u.pos) * kSteps;
  };
  const auto sequence = [&](uint32_t q, int& n, int& d) {  // q / D by the launch's multiplier
    n = static_cast<int>((static_cast<uint64_t>(q) * c.div_mul) >> c.div_shift);
    d = static_cast<int>(q - static_cast<uint32_t>(n) * static_cast<uint32_t>(p.D));
  };
  // whether the 32 lanes of a block lie in one sequence (then one load brings all its flags)
  const bool one = kReset && p.D % (32 * kVec) == 0;

  // Start copying a unit's steps (and its flags, into a register).
  const auto fetch = [&](const Unit& u, int stage, uint32_t& flags) {
    const int64_t t0 = start(u);
    if (u.block < 0) {
      cp_async_commit();
      return;
    }
    uint32_t* dst = words(stage);
    const uint32_t q0 = static_cast<uint32_t>(u.block) * 32u * kVec, q = q0 + lane * kVec;
    const bool in = q < lanes;
    int n = 0, d = 0;
    if (in) sequence(q, n, d);
    const bool full = q0 + 32u * kVec <= lanes && t0 > 0 && t0 + kSteps <= p.L;
    if (c.wide) {  // 16-byte pieces: this lane's are 4 steps apart, in one sequence
      constexpr int kPiece = 16 / sizeof(T);
      const int sub = lane >> 3;
      const uint32_t qp = q0 + (lane & 7) * kPiece;
      const bool inp = qp < lanes;
      int np = 0, dp = 0;
      if (inp) sequence(qp, np, dp);
      const int row = np * static_cast<int>(p.L) + static_cast<int>(t0) + sub;
      uint32_t* to = dst + sub * 32 + (lane & 7) * 4;
#pragma unroll
      for (int i = 0; i < D::kStreams; ++i) {
        const Stream st = D::stream(p, i);
        const int at = D::place(kMode, i) * kSteps;
        if (st.p == nullptr || at < 0) continue;
        const int ld = static_cast<int>(st.ld);
        const T* src = static_cast<const T*>(st.p) + static_cast<int64_t>(row - st.shift) * ld + dp;
        if (full) {
#pragma unroll
          for (int j = 0; j < kSteps; j += 4)
            cp_async_16_zfill(to + (at + j) * 32, src + static_cast<int64_t>(j) * ld, 16);
        } else {
#pragma unroll
          for (int j = 0; j < kSteps; j += 4) {
            const int64_t t = t0 + j + sub;
            const bool on = inp && t0 >= 0 && t < p.L && (st.shift == 0 || t > 0);
            cp_async_16_zfill(to + (at + j) * 32,
                              on ? src + static_cast<int64_t>(j) * ld : static_cast<const T*>(st.p),
                              on ? 16 : 0);
          }
        }
      }
    } else {
      const int row = n * static_cast<int>(p.L) + static_cast<int>(t0);
#pragma unroll
      for (int i = 0; i < D::kStreams; ++i) {
        const Stream st = D::stream(p, i);
        const int at = D::place(kMode, i) * kSteps;
        if (st.p == nullptr || at < 0) continue;
        const int ld = static_cast<int>(st.ld);
        const T* src = static_cast<const T*>(st.p) + static_cast<int64_t>(row - st.shift) * ld + d;
        const auto on = [&](int j) {
          return in && t0 >= 0 && t0 + j < p.L && (st.shift == 0 || t0 + j > 0);
        };
        if (sizeof(T) * kVec == 4) {
#pragma unroll 4
          for (int j = 0; j < kSteps; ++j)
            cp_async_4_zfill(dst + (at + j) * 32 + lane,
                             on(j) ? src + static_cast<int64_t>(j) * ld : static_cast<const T*>(st.p),
                             on(j) ? 4 : 0);
        } else {  // single bf16 channels: no asynchronous copy is that small
          uint32_t v[kSteps];
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
            v[j] = on(j) ? static_cast<uint32_t>(__ldcs(src + static_cast<int64_t>(j) * ld)) : 0u;
#pragma unroll
          for (int j = 0; j < kSteps; ++j) dst[(at + j) * 32 + lane] = v[j];
        }
      }
    }
    if (kWalk && u.pos == pos_begin && D::first(p) != nullptr)
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        cp_async_4_zfill(dst + kWords + lane * kVec + i, D::first(p) + (in ? q + i : 0), in ? 4 : 0);
    cp_async_commit();
    if (kReset) {
      const uint8_t* src = p.reset + static_cast<int64_t>(n) * p.L + t0;
      flags = 0u;
      if (one) {
        if (in && lane < kSteps && t0 >= 0 && t0 + lane < p.L) flags = __ldg(src + lane);
      } else if (in && t0 >= 0) {
        for (int j = 0; j < kSteps && t0 + j < p.L; ++j)
          flags |= static_cast<uint32_t>(__ldg(src + j) != 0) << j;
      }
    }
  };

  // the first kStages - 1 units on their way
  uint32_t flags[kStages];  // of the units in turn
  Unit far = cur;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) {
    fetch(far, k, flags[k]);
    far = after(far);
  }
  float x[kVec];
  Span acc[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    x[i] = 0.f;
    acc[i] = {1.f, 0.f};
  }
  const size_t channel0 = static_cast<size_t>(lane) * kVec;
  if (kMode == Mode::kSpans) griddep_launch_dependents();
  if (kMode == Mode::kSegments) {
    griddep_wait();
    // the value before the segment: through the spans of the CTAs before this one and of the
    // warps before this one (the first of them drops what is before it for the sequence's first
    // value, which another CTA may by now have overwritten with the last)
    const int per = c.segs / kWarps, mine = blockIdx.x % per;
    const Span* sums = c.spans + (static_cast<size_t>(blockIdx.x) - mine) * (kWarps + 1) * 64;
    constexpr int kBatch = 16 / kVec;  // spans in flight
    for (int k0 = 0; k0 < mine; k0 += kBatch) {
      float2 f[kBatch][kVec];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (k0 + k < mine)
            f[k][i] = __ldcg(reinterpret_cast<const float2*>(
                sums + static_cast<size_t>(k0 + k) * (kWarps + 1) * 64 + channel0 + i));
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (k0 + k < mine) x[i] = apply(Span{f[k][i].x, f[k][i].y}, x[i]);
    }
    const Span* own = c.spans + (static_cast<size_t>(blockIdx.x) * (kWarps + 1) + 1 + warp) * 64;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float2 f = __ldcg(reinterpret_cast<const float2*>(own + channel0 + i));
      x[i] = apply(Span{f.x, f.y}, x[i]);
    }
  }
  int stage = 0;
  for (int turn = 0; cur.block >= 0; ++turn) {
    fetch(far, stage == 0 ? kStages - 1 : stage - 1, flags[kStages - 1]);
    far = after(far);
    cp_async_wait_group<kStages - 1>();
    __syncwarp();
    const uint32_t* in = words(stage) + lane;
    const int64_t t0 = start(cur), left = p.L - t0;
    const uint32_t q = static_cast<uint32_t>(cur.block) * 32u * kVec + lane * kVec;
    const bool valid = q < lanes && t0 >= 0;
    int n = 0, d = 0;
    if (valid) sequence(q, n, d);
    const int count = !valid || left <= 0 ? 0 : (left < kSteps ? static_cast<int>(left) : kSteps);
    uint32_t resets = 0u;
    if (kReset) resets = one ? __ballot_sync(0xFFFFFFFFu, flags[0] != 0u) : flags[0];
    if (kWalk && cur.pos == pos_begin) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        x[i] = D::first(p) != nullptr
                   ? __uint_as_float(words(stage)[kWords + lane * kVec + i])
                   : 0.f;
    }
    // (a unit without a reset, as most are, takes the shorter code)
    const bool any = kReset && __any_sync(0xFFFFFFFFu, resets != 0u);
    D dir;
    if (kReset && any)
      dir.template read<kMode, true>(p, in, resets, count);
    else
      dir.template read<kMode, false>(p, in, 0u, count);
    Span f[kVec];
    if (kMode == Mode::kSpans || W > 1) {
      if (kReset && any)
        dir.template span<true>(f);
      else
        dir.template span<false>(f);
    }
    if (kMode == Mode::kSpans) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = then(f[i], acc[i]);
    } else {
      float mine[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) mine[i] = x[i];
      if (W > 1) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) s_span[turn & 1][warp][lane * kVec + i] = f[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          for (int k = 0; k < W; ++k) {
            if (k == order) mine[i] = x[i];
            x[i] = apply(s_span[turn & 1][group * W + k][lane * kVec + i], x[i]);
          }
      }
      if (count == kSteps && !any)
        dir.template run<false, true>(p, in, 0u, n, d, t0, count, mine);
      else
        dir.template run<kReset, false>(p, in, resets, n, d, t0, count, mine);
      if (W == 1)
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = mine[i];
    }
    __syncwarp();  // this warp's steps are read before the next copies land on them
    cur = after(cur);
    stage = stage == kStages - 1 ? 0 : stage + 1;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) flags[k] = flags[k + 1];
  }
  if (kMode == Mode::kSpans) {
    // this CTA's span, and before each warp's segment the span of the warps before it
#pragma unroll
    for (int i = 0; i < kVec; ++i) s_span[0][warp][channel0 + i] = acc[i];
    __syncthreads();
    Span* out = c.spans + static_cast<size_t>(blockIdx.x) * (kWarps + 1) * 64;
    const int per = c.segs / kWarps;
    const uint32_t q = (blockIdx.x / per * 32u + lane) * kVec;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      Span f{1.f, 0.f};
      if (blockIdx.x % per == 0)
        f = {kDrops, q < lanes && D::first(p) != nullptr ? D::first(p)[q + i] : 0.f};
      for (int k = 0; k < warp; ++k) f = then(f, s_span[0][k][channel0 + i]);
      out[(1 + warp) * 64 + channel0 + i] = f;
      if (warp == kWarps - 1) out[channel0 + i] = then(f, acc[i]);
    }
  }
}

template <template <typename, int> class Dir, typename T, int kVec, Mode kMode, bool kReset>
cudaError_t scan_launch(const typename Dir<T, kVec>::Args& a, const ScanLaunch& c, int64_t grid,
                        cudaStream_t stream) {
  using D = Dir<T, kVec>;
  const auto fn = scan_kernel<Dir, T, kVec, kMode, kReset>;
  constexpr int kSmem =
      D::stages(kMode) * D::kWarps * (D::streams(kMode) * D::kSteps * 32 + 32 * kVec) * 4;
  cudaError_t e = (*c.opt_in)(fn, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(D::kWarps * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  // the walk of the segments starts while their spans are finished: its first copies read only
  // what the launch for the spans had to wait for as well
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kMode == Mode::kSegments ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, fn, a, c);
  if (e == cudaSuccess) *c.launches += 1;
  return e;
}

template <template <typename, int> class Dir, typename T, int kVec, bool kReset>
cudaError_t scan_as(const typename Dir<T, kVec>::Args& a, ScanLaunch c, cudaStream_t stream) {
  constexpr int kWarps = Dir<T, kVec>::kWarps, kSteps = Dir<T, kVec>::kSteps;
  const int64_t lanes = (a.N * a.D + kVec - 1) / kVec, places = (a.L + kSteps - 1) / kSteps;
  const int64_t room = 2 * c.num_sms;  // two CTAs fit an SM
  c.blocks = (lanes + 31) / 32;
  // q / D = q * div_mul >> div_shift for q < 2^31
  int bits = 0;
  while ((1ll << bits) < a.D) ++bits;
  c.div_shift = 31 + bits;
  c.div_mul = static_cast<uint32_t>(((1ull << c.div_shift) + a.D - 1) / a.D);
  // Segments where walking would leave most SMs without work and sequences are long enough to cut.
  // 16.8 M steps of fp32 channels in 8 / 38 / 76 / 152 / 304 blocks, forward and backward: segments
  // 82 and 95 us throughout, walking 1081 / 234 / 121 / 64 / 53 and 1504 / 325 / 166 / 86 / 70 us.
  if (8 * c.blocks <= 3 * room && places >= 4 * kWarps) {
    int64_t per = std::min(room / c.blocks, places / (2 * kWarps));  // CTAs a block
    c.segs = static_cast<int>(per * kWarps);
    c.seg = static_cast<int>((places + c.segs - 1) / c.segs);
    const cudaError_t e =
        scan_launch<Dir, T, kVec, Mode::kSpans, kReset>(a, c, c.blocks * per, stream);
    if (e != cudaSuccess) return e;
    return scan_launch<Dir, T, kVec, Mode::kSegments, kReset>(a, c, c.blocks * per, stream);
  }
  // More warps to a block while blocks are few, and none that would have a single turn (so 16 steps
  // give what 16 calls of one step give).  10 M steps of fp32 channels walked by 1 / 2 / 4 / 8 warps a
  // block, backward: 1216 blocks 47 / 45 / 45 / 43 us, 2432 and 4864 blocks 47 / 43 / 43 / 43 us, 9728
  // blocks 45 / 43 / 43 / 78 us; 5 M in 304 blocks 84 / 52 / 31 / 25 us.
  c.W = 1;
  while (c.W < kWarps && 2 * c.W < places && c.blocks * c.W < 8 * room * kWarps) c.W *= 2;
  const int64_t groups = kWarps / c.W;
  return scan_launch<Dir, T, kVec, Mode::kWalk, kReset>(
      a, c, std::min((c.blocks + groups - 1) / groups, room), stream);
}

template <template <typename, int> class Dir, typename T, int kVec>
cudaError_t scan_any(const typename Dir<T, kVec>::Args& a, const ScanLaunch& c,
                     cudaStream_t stream) {
  return a.reset != nullptr ? scan_as<Dir, T, kVec, true>(a, c, stream)
                            : scan_as<Dir, T, kVec, false>(a, c, stream);
}

// Whether every row of these tensors starts on a multiple of `bytes`.
struct Rows {
  const void* p;
  int64_t ld;
};
bool aligned(std::initializer_list<Rows> all, int D, size_t size, size_t bytes) {
  if (D * size % bytes != 0) return false;
  for (const Rows& r : all)
    if (r.p != nullptr && (reinterpret_cast<uintptr_t>(r.p) % bytes != 0 ||
                           static_cast<size_t>(r.ld) * size % bytes != 0))
      return false;
  return true;
}

}  // namespace

cudaError_t launch_rnn_scan(const RnnScanArgs& a, const ScanLaunch& launch, cudaStream_t stream) {
  const size_t size = a.dtype == DSPARK_F32 ? 4 : 2;
  const std::initializer_list<Rows> in = {{a.za, a.ld_za}, {a.zg, a.ld_zg}, {a.e, a.ld_e}};
  ScanLaunch c = launch;
  c.wide = aligned(in, a.D, size, 16);  // 16-byte copies, else 4-byte ones
  if (a.dtype == DSPARK_F32) return scan_any<Forward, float, 1>(a, c, stream);
  // pairs of bf16 channels where every row starts on a 4-byte boundary
  if (aligned(in, a.D, size, 4) && aligned({{a.s, a.D}}, a.D, size, 4))
    return scan_any<Forward, uint16_t, 2>(a, c, stream);
  c.wide = false;
  return scan_any<Forward, uint16_t, 1>(a, c, stream);
}

cudaError_t launch_rnn_scan_grad(const RnnScanGradArgs& a, const ScanLaunch& launch,
                                 cudaStream_t stream) {
  const size_t size = a.dtype == DSPARK_F32 ? 4 : 2;
  const std::initializer_list<Rows> in = {
      {a.za, a.ld_za}, {a.zg, a.ld_zg}, {a.e, a.ld_e}, {a.ds, a.D}, {a.s, a.D}};
  ScanLaunch c = launch;
  c.wide = aligned(in, a.D, size, 16);
  if (a.dtype == DSPARK_F32) return scan_any<Backward, float, 1>(a, c, stream);
  if (aligned(in, a.D, size, 4) &&
      aligned({{a.dza, a.ld_dza}, {a.dzg, a.ld_dzg}, {a.de, a.D}}, a.D, size, 4))
    return scan_any<Backward, uint16_t, 2>(a, c, stream);
  c.wide = false;
  return scan_any<Backward, uint16_t, 1>(a, c, stream);
}

}  // namespace dspark
