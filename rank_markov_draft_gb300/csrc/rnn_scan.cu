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
// A reset at t makes a_t zero.  A decay of exactly zero drops the earlier state, whatever it
// holds (an infinity or NaN before a reset stays before it).
//
// Both directions are a recurrence x_t = a_t x_{t-1} + b_t, so a span of steps acts on the
// value before it as x -> A x + S (A the product of its decays, S its end from zero).  A warp
// holds 16 steps of 32 lanes in registers (a lane is 4 bytes of channels: two bf16 or one fp32;
// lanes run over sequences and channels alike, so no channel count leaves lanes empty): it
// loads them once, reduces them to (A, S), learns the value before them from the warps before
// it, and runs them again from there.  Three ways to learn it:
//   L <= 16:         there is nothing before them but s0.
//   many lanes:      the CTA's W warps hold consecutive spans, exchange (A, S) through shared
//                    memory and walk over the sequence; the value after a tile stays with them.
//   few lanes, long: the walk alone would leave most SMs empty, so tiles of one sequence go to
//                    different CTAs in the order of a ticket.  A tile publishes its (A, S) as
//                    soon as it has them and its end value once that is known; a tile folds
//                    the (A, S) after the nearest known end value, strictly in order, so the
//                    result does not depend on which one that was.
// Every input is read once and every output written once in all three.

#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>

#include "internal.h"
#include "sm103.cuh"

namespace dspark {
namespace {

constexpr int kSteps = 16;      // of a warp
constexpr int kScanWarps = 8;   // of a CTA
constexpr float kRsLog2e = 1.4426950408889634f;

// ---- lanes: kVec channels of 4 bytes (2 for single bf16 channels), kept raw in one register
template <typename T, int kVec>
struct Lane;
template <>
struct Lane<float, 1> {
  static __device__ __forceinline__ uint32_t load(const float* p) {
    return __ldcs(reinterpret_cast<const uint32_t*>(p));
  }
  static __device__ __forceinline__ float get(uint32_t r, int) { return __uint_as_float(r); }
  static __device__ __forceinline__ void store(float* p, const float* x) { __stcs(p, x[0]); }
};
template <>
struct Lane<uint16_t, 1> {
  static __device__ __forceinline__ uint32_t load(const uint16_t* p) { return __ldcs(p); }
  static __device__ __forceinline__ float get(uint32_t r, int) { return __uint_as_float(r << 16); }
  static __device__ __forceinline__ void store(uint16_t* p, const float* x) {
    __stcs(p, __bfloat16_as_ushort(__float2bfloat16_rn(x[0])));
  }
};
template <>
struct Lane<uint16_t, 2> {
  static __device__ __forceinline__ uint32_t load(const uint16_t* p) {
    return __ldcs(reinterpret_cast<const uint32_t*>(p));
  }
  static __device__ __forceinline__ float get(uint32_t r, int i) {
    return __uint_as_float(i == 0 ? r << 16 : r & 0xFFFF0000u);
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float* x) {
    uint32_t r;  // one rounding to bf16, to nearest even, where a value leaves the recurrence
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x[1]), "f"(x[0]));
    __stcs(reinterpret_cast<uint32_t*>(p), r);
  }
};

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// sigmoid(z): exact zero and one at the far ends
__device__ __forceinline__ float gate(float z) {
  return rcp_approx(1.f + ex2_approx(-z * kRsLog2e));
}
// and 1 - sigmoid(z) to full relative precision, down to the denormals that a product with a
// large gradient brings back into range (so not the exponential that flushes them)
__device__ __forceinline__ float gate(float z, float& rest) {
  const float t = exp2f(-z * kRsLog2e);
  float a;
  asm("rcp.approx.f32 %0, %1;" : "=f"(a) : "f"(1.f + t));
  rest = t <= 1.f ? t * a : 1.f - a;
  return a;
}

// A span's effect x -> A x + S.  kDrops in A: a decay of exactly zero inside, so x is dropped
// (a product that has merely underflowed keeps an infinity or NaN).
constexpr float kDrops = -1.f;
struct Span {
  float A, S;
};
__device__ __forceinline__ float apply(Span f, float x) {
  return f.A == kDrops ? f.S : fmaf(f.A, x, f.S);
}
__device__ __forceinline__ Span then(Span f, Span g) {  // f first
  return {f.A == kDrops || g.A == kDrops ? kDrops : f.A * g.A, apply(g, f.S)};
}

// ---- the ticketed tiles' records (context scratch; flags and tickets zero between launches)
struct ChainView {
  Span* span;       // [slots][kChainLanes]
  float* end;       // [slots][kChainLanes]
  float* carry;     // [kChainBlocks][kChainLanes] the value after the launch before
  uint32_t* flag;   // [slots] 1: span known, 2: end known
  uint32_t* ticket; // [0] next ticket, [1] CTAs done
};
__device__ __forceinline__ ChainView chain_view(void* scratch) {
  ChainView v;
  v.span = static_cast<Span*>(scratch);
  v.end = reinterpret_cast<float*>(v.span + kChainSlots * kChainLanes);
  v.carry = v.end + kChainSlots * kChainLanes;
  v.flag = reinterpret_cast<uint32_t*>(v.carry + kChainBlocks * kChainLanes);
  v.ticket = v.flag + kChainSlots;
  return v;
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t r;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(r) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// One warp, tile `tile` of its chain, whose records start at slot `first`: publish the span,
// find the value before the tile, publish the value after it.  x: the value before tile 0 on
// entry, before this tile on return.
template <int kVec>
__device__ __forceinline__ void chain_step(const ChainView& v, int tile, int first, int lane,
                                           const Span (&span)[kVec], float (&x)[kVec], int* status,
                                           uint64_t timeout_ns) {
  const auto at = [&](int t, int i) {
    return static_cast<size_t>(first + t) * kChainLanes + lane * kVec + i;
  };
  uint32_t* flag = v.flag + first;
  if (tile > 0) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v.span[at(tile, i)] = span[i];
    __syncwarp();
    if (lane == 0) {
      __threadfence();
      st_release(flag + tile, 1u);
    }
    // the nearest earlier tile whose end is known, the spans of all after it being known too
    int from = -1;
    uint64_t deadline = 0;
    for (uint32_t spins = 0; from < 0; ++spins) {
      const int t = tile - 1 - lane;
      const uint32_t state = t >= 0 ? ld_acquire(flag + t) : 0u;
      const uint32_t ends = __ballot_sync(0xFFFFFFFFu, state == 2u);
      const uint32_t unknown = __ballot_sync(0xFFFFFFFFu, state == 0u);
      if (ends != 0u && (unknown & ((ends & (0u - ends)) - 1u)) == 0u) {
        from = tile - __ffs(ends);
      } else if (spins > 16u) {
        const uint64_t now = globaltimer_ns();
        if (deadline == 0) {
          deadline = now + timeout_ns;
        } else if (__shfl_sync(0xFFFFFFFFu, static_cast<int>(now > deadline), 0)) {
          if (lane == 0) record_error(status, kStatusTimeout);
          break;
        }
      }
    }
    __syncwarp();
    __threadfence();
    if (from >= 0) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[i] = __ldcg(v.end + at(from, i));
#pragma unroll 8
      for (int t = from + 1; t < tile; ++t)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(v.span + at(t, i)));
          x[i] = apply(Span{f.x, f.y}, x[i]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) v.end[at(tile, i)] = apply(span[i], x[i]);
  __syncwarp();
  if (lane == 0) {
    __threadfence();
    st_release(flag + tile, 2u);
  }
}

// The last CTA of the launch to finish leaves flags and tickets as it found them.
__device__ __forceinline__ void chain_leave(const ChainView& v, uint32_t* s_last) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    *s_last = atomicAdd(v.ticket + 1, 1u) == gridDim.x - 1 ? 1u : 0u;
  }
  __syncthreads();
  if (*s_last == 0u) return;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += blockDim.x) v.flag[i] = 0u;
  if (threadIdx.x < 2) v.ticket[threadIdx.x] = 0u;
}

// What a direction does with its 16 steps: load them, give their span, run them from a value.
template <typename T, int kVec>
struct Forward {
  using Args = RnnScanArgs;
  using Ln = Lane<T, kVec>;
  static constexpr bool kReverse = false;
  float a[kSteps][kVec], b[kSteps][kVec];

  __device__ __forceinline__ void load(const Args& p, int64_t n, int d, int64_t t0, int steps) {
    const int64_t r = n * p.L + t0;
    const T* za = static_cast<const T*>(p.za) + r * p.ld_za + d;
    const T* zg = static_cast<const T*>(p.zg) + r * p.ld_zg + d;
    const T* e = static_cast<const T*>(p.e) + r * p.ld_e + d;
    uint32_t ra[kSteps], rg[kSteps], re[kSteps], keep = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      ra[j] = rg[j] = re[j] = 0u;
      if (j < steps) {
        ra[j] = Ln::load(za + j * p.ld_za);
        if (p.zg != nullptr) rg[j] = Ln::load(zg + j * p.ld_zg);
        re[j] = Ln::load(e + j * p.ld_e);
        if (p.reset != nullptr && __ldg(p.reset + r + j) != 0) keep &= ~(1u << j);
      }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float g = p.zg != nullptr ? gate(Ln::get(rg[j], i)) : 1.f;
        a[j][i] = j >= steps ? 1.f : (keep >> j & 1u ? gate(Ln::get(ra[j], i)) : 0.f);
        b[j][i] = j < steps ? g * Ln::get(re[j], i) : 0.f;
      }
  }
  __device__ __forceinline__ void span(int, Span (&f)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      f[i] = {1.f, 0.f};
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
        f[i] = then(f[i], Span{a[j][i] == 0.f ? kDrops : a[j][i], b[j][i]});
    }
  }
  __device__ __forceinline__ void first_value(const Args& p, int64_t q, float (&x)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = p.s0 != nullptr ? p.s0[q + i] : 0.f;
  }
  __device__ __forceinline__ void run(const Args& p, int64_t n, int d, int64_t t0, int steps,
                                      float (&x)[kVec]) const {
    T* s = static_cast<T*>(p.s) + (n * p.L + t0) * p.D + d;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if (j >= steps) break;
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[i] = a[j][i] == 0.f ? b[j][i] : fmaf(a[j][i], x[i], b[j][i]);
      Ln::store(s + static_cast<int64_t>(j) * p.D, x);
    }
    if (p.s_last != nullptr && steps > 0 && t0 + steps == p.L)
#pragma unroll
      for (int i = 0; i < kVec; ++i) p.s_last[n * p.D + d + i] = x[i];
  }
};

template <typename T, int kVec>
struct Backward {
  using Args = RnnScanGradArgs;
  using Ln = Lane<T, kVec>;
  static constexpr bool kReverse = true;
  uint32_t za[kSteps], zg[kSteps], e[kSteps], ds[kSteps], s[kSteps], keep;

  __device__ __forceinline__ void load(const Args& p, int64_t n, int d, int64_t t0, int steps) {
    const int64_t r = n * p.L + t0;
    const T* pa = static_cast<const T*>(p.za) + r * p.ld_za + d;
    const T* pg = static_cast<const T*>(p.zg) + r * p.ld_zg + d;
    const T* pe = static_cast<const T*>(p.e) + r * p.ld_e + d;
    const T* pd = static_cast<const T*>(p.ds) + r * p.D + d;
    const T* ps = static_cast<const T*>(p.s) + (r - 1) * p.D + d;  // the state before
    keep = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      za[j] = zg[j] = e[j] = ds[j] = s[j] = 0u;
      if (j < steps) {
        za[j] = Ln::load(pa + j * p.ld_za);
        ds[j] = Ln::load(pd + static_cast<int64_t>(j) * p.D);
        if (p.reset != nullptr && __ldg(p.reset + r + j) != 0) keep &= ~(1u << j);
      }
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      if (j < steps) {
        if (p.zg != nullptr) zg[j] = Ln::load(pg + j * p.ld_zg);
        e[j] = Ln::load(pe + j * p.ld_e);
        if (t0 + j > 0) s[j] = Ln::load(ps + static_cast<int64_t>(j) * p.D);
      }
  }
  __device__ __forceinline__ void span(int steps, Span (&f)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      f[i] = {1.f, 0.f};
#pragma unroll
      for (int j = kSteps - 1; j >= 0; --j) {
        if (j >= steps) continue;
        const float a = keep >> j & 1u ? gate(Ln::get(za[j], i)) : 0.f;
        f[i] = then(f[i], Span{a == 0.f ? kDrops : a, a == 0.f ? 0.f : a * Ln::get(ds[j], i)});
      }
    }
  }
  __device__ __forceinline__ void first_value(const Args& p, int64_t q, float (&x)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = p.ds_last != nullptr ? p.ds_last[q + i] : 0.f;
  }
  __device__ __forceinline__ void run(const Args& p, int64_t n, int d, int64_t t0, int steps,
                                      float (&x)[kVec]) const {
    const int64_t r = n * p.L + t0;
    T* pa = static_cast<T*>(p.dza) + r * p.ld_dza + d;
    T* pg = static_cast<T*>(p.dzg) + r * p.ld_dzg + d;
    T* pe = static_cast<T*>(p.de) + r * p.D + d;
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      if (j >= steps) continue;
      float oa[kVec], og[kVec], oe[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        float na, ng = 0.f, g = 1.f;
        float a = gate(Ln::get(za[j], i), na);
        if (!(keep >> j & 1u)) a = 0.f;
        if (p.zg != nullptr) g = gate(Ln::get(zg[j], i), ng);
        float before = Ln::get(s[j], i);
        if (t0 + j == 0) before = p.s0 != nullptr ? p.s0[n * p.D + d + i] : 0.f;
        const float delta = Ln::get(ds[j], i) + x[i];
        oa[i] = a == 0.f ? 0.f : delta * before * a * na;
        og[i] = delta * Ln::get(e[j], i) * g * ng;
        oe[i] = delta * g;
        x[i] = a == 0.f ? 0.f : a * delta;
      }
      Ln::store(pa + j * p.ld_dza, oa);
      if (p.dzg != nullptr) Ln::store(pg + j * p.ld_dzg, og);
      Ln::store(pe + static_cast<int64_t>(j) * p.D, oe);
    }
    if (p.ds0 != nullptr && t0 == 0 && steps > 0)
#pragma unroll
      for (int i = 0; i < kVec; ++i) p.ds0[n * p.D + d + i] = x[i];
  }
};

// Walks: a CTA of kScanWarps warps is kScanWarps / W lane blocks of W consecutive spans (W = 1:
// no exchange).  Tickets: one lane block, tile c.first_tile + ticket / blocks of `tiles`.
template <template <typename, int> class Dir, typename T, int kVec, bool kTicket>
__global__ void __launch_bounds__(kScanWarps * 32, 2)
    scan_kernel(const typename Dir<T, kVec>::Args p, const int W, const int blocks,
                const ScanLaunch c) {
  using D = Dir<T, kVec>;
  __shared__ Span s_span[2][kScanWarps][32 * kVec];
  __shared__ float s_x[32 * kVec];
  __shared__ uint32_t s_ticket;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tiles = (p.L + W * kSteps - 1) / (W * kSteps);
  // `order`: this warp's place in the recurrence's order, `w` in the order of time
  const int group = warp / W, order = warp % W, w = D::kReverse ? W - 1 - order : order;
  int64_t block = static_cast<int64_t>(blockIdx.x) * (kScanWarps / W) + group;
  int64_t tile = 0, tile_end = tiles;
  ChainView chain{};
  if (kTicket) {
    chain = chain_view(c.chain);
    if (threadIdx.x == 0) s_ticket = atomicAdd(chain.ticket, 1u);
    __syncthreads();
    block = s_ticket % blocks;
    tile = c.first_tile + s_ticket / blocks;
    tile_end = tile + 1;
  }
  const int64_t q = (block * 32 + lane) * kVec;
  const bool valid = q < p.N * p.D;
  const int64_t n = valid ? q / p.D : 0;
  const int d = valid ? static_cast<int>(q - n * p.D) : 0;
  D steps;
  float x[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) x[i] = 0.f;
  if (valid && tile == 0) steps.first_value(p, q, x);
  if (kTicket && tile > 0 && tile == c.first_tile) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = chain.carry[block * kChainLanes + lane * kVec + i];
  }
  for (; tile < tile_end; ++tile) {
    const int64_t t0 = ((D::kReverse ? tiles - 1 - tile : tile) * W + w) * kSteps;
    const int64_t left = p.L - t0;
    const int count = !valid || left <= 0 ? 0 : (left < kSteps ? static_cast<int>(left) : kSteps);
    steps.load(p, n, d, t0, count);
    if (W > 1) {
      const int buf = static_cast<int>(tile & 1);
      Span f[kVec];
      steps.span(count, f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) s_span[buf][warp][lane * kVec + i] = f[i];
      __syncthreads();
      if (kTicket) {
        if (warp == 0) {
          Span all[kVec];
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            all[i] = {1.f, 0.f};
            for (int k = 0; k < W; ++k) all[i] = then(all[i], s_span[buf][k][lane * kVec + i]);
          }
          chain_step<kVec>(chain, static_cast<int>(tile - c.first_tile),
                           static_cast<int>(block) * c.launch_tiles, lane, all, x, c.status,
                           c.timeout_ns);
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            s_x[lane * kVec + i] = x[i];
            if (tile + 1 == c.first_tile + c.launch_tiles)
              chain.carry[block * kChainLanes + lane * kVec + i] = apply(all[i], x[i]);
          }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = s_x[lane * kVec + i];
      }
      float mine[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        mine[i] = x[i];
        for (int k = 0; k < W; ++k) {
          if (k == order) mine[i] = x[i];
          x[i] = apply(s_span[buf][group * W + k][lane * kVec + i], x[i]);
        }
      }
      steps.run(p, n, d, t0, count, mine);
    } else {
      steps.run(p, n, d, t0, count, x);
    }
  }
  if (kTicket) chain_leave(chain, &s_ticket);
}

template <template <typename, int> class Dir, typename T, int kVec>
cudaError_t scan_as(const typename Dir<T, kVec>::Args& a, ScanLaunch c, cudaStream_t stream) {
  const int64_t lanes = (a.N * a.D + kVec - 1) / kVec, blocks = (lanes + 31) / 32;
  int W = 1;
  while (W < kScanWarps && W * kSteps < a.L) W *= 2;
  const int64_t tiles = (a.L + W * kSteps - 1) / (W * kSteps);
  // Two CTAs fit an SM.  Where walking would leave SMs without and there are tiles to give
  // away, they go by tickets, as many to a launch as there are records (no record is used
  // twice in a launch, so a slow reader finds what it was told of).
  const int64_t most = kChainSlots / std::max<int64_t>(blocks, 1);
  if (W == kScanWarps && blocks < std::min(2 * c.num_sms, kChainBlocks) && tiles > 1) {
    for (int64_t t = 0; t < tiles; t += most) {
      c.first_tile = t;
      c.launch_tiles = static_cast<int>(std::min(most, tiles - t));
      scan_kernel<Dir, T, kVec, true>
          <<<static_cast<unsigned>(c.launch_tiles * blocks), kScanWarps * 32, 0, stream>>>(
              a, W, static_cast<int>(blocks), c);
      *c.launches += 1;
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const int64_t groups = kScanWarps / W;
  scan_kernel<Dir, T, kVec, false>
      <<<static_cast<unsigned>((blocks + groups - 1) / groups), kScanWarps * 32, 0, stream>>>(
          a, W, static_cast<int>(blocks), c);
  *c.launches += 1;
  return cudaGetLastError();
}

bool even(int64_t x) { return (x & 1) == 0; }
bool word_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

cudaError_t launch_rnn_scan(const RnnScanArgs& a, const ScanLaunch& c, cudaStream_t stream) {
  if (a.dtype == DSPARK_F32) return scan_as<Forward, float, 1>(a, c, stream);
  // pairs of bf16 channels where every row starts on a 4-byte boundary
  if (even(a.D) && even(a.ld_za) && even(a.ld_zg) && even(a.ld_e) && word_aligned(a.za) &&
      word_aligned(a.zg) && word_aligned(a.e) && word_aligned(a.s))
    return scan_as<Forward, uint16_t, 2>(a, c, stream);
  return scan_as<Forward, uint16_t, 1>(a, c, stream);
}

cudaError_t launch_rnn_scan_grad(const RnnScanGradArgs& a, const ScanLaunch& c,
                                 cudaStream_t stream) {
  if (a.dtype == DSPARK_F32) return scan_as<Backward, float, 1>(a, c, stream);
  if (even(a.D) && even(a.ld_za) && even(a.ld_zg) && even(a.ld_e) && even(a.ld_dza) &&
      even(a.ld_dzg) && word_aligned(a.za) && word_aligned(a.zg) && word_aligned(a.e) &&
      word_aligned(a.s) && word_aligned(a.ds) && word_aligned(a.dza) && word_aligned(a.dzg) &&
      word_aligned(a.de))
    return scan_as<Backward, uint16_t, 2>(a, c, stream);
  return scan_as<Backward, uint16_t, 1>(a, c, stream);
}

}  // namespace dspark
