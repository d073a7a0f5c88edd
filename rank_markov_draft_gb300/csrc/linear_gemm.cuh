// linear_gemm.cuh -- one matrix product on the tensor cores, with the linear layers' epilogue:
//   out(i, j) = act(sum_k A(i, k) B(k, j) + bias_j) + residual(i, j).
//
// A persistent block an SM walks over units (a tile of 128 x BN outputs, and a part of the
// contraction where the tiles alone would leave SMs idle).  One lane fills a ring of stages of 64
// terms by TMA (128-byte swizzle), one issues tcgen05.mma (M = 128, N = BN, accumulator in TMEM), and
// eight warps take finished accumulators through the epilogue while the next unit's products run into
// the other half of TMEM. Outputs whose rows TMA can write leave by it, a warp's 32 rows x 64 columns at
// a time through shared memory, and residuals arrive the same way, ahead of their products; others go
// element by element.  Either operand may lie with the contraction contiguous (K-major) or with
// its own index contiguous (MN-major), so x W, dz W^T and x^T dz read their matrices as they are.
//
// Where the products bound it, two blocks share tiles of 256 x 256 (PAIR): each loads half of A's rows and
// half of B's columns, so that an output costs two thirds of the reads from L2, which is what a block by
// itself waits for (0.52 us a stage of 48 KB; its products take 0.27).
//
// An operand may come in three parts, added up like further terms: A = A_0 + A_1 + A_2.
//
// The accumulator cuts what a sum of fp32 would round, so that a long sum of terms drifts (2e-6 of itself
// over 2048 terms, 2e-5 over 50000). So it starts again every 512 terms, and the epilogue's threads add up
// what it held, rounded, in registers: 5e-7 at any length, a sum of fp32 in order gives 4e-7 to 8e-7.
// (Every 256 terms gave 2.4e-7, but the logits' gradients then took 287 us instead of 221.)  bf16 outputs
// need it too: of the logits' dx, 17000 terms a block, 1.8% of the elements lay a step beside the nearest
// bf16 number without, 0.04% with it (0.11% where fp32 sums are taken in order).  It costs them 216 -> 221 us
// there, and 166 -> 184 where a tile's start waits for the one before (4096 x 8192 x 4096); every 1024 terms
// 175, and twice as many elements beside.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "activation.cuh"
#include "async_copy.cuh"
#include "cta_pair.cuh"
#include "sm103.cuh"
#include "typed.cuh"

namespace dspark {

struct GemmArgs {
  CUtensorMap a[3], b[3];
  CUtensorMap out_map, pre_map, res_map;  // (outputs by TMA) boxes of 32 rows x 128 bytes
  int a_parts, b_parts;     // 1, or 3 of one of them
  int64_t I;                // rows and columns of the output
  int J;
  int64_t tiles_i, units;
  int tiles_j, splits;
  int64_t steps, per_split; // stages of a tile (all parts), of a unit
  int64_t blocks_k;         // stages of a part
  int streams;              // columns of tiles are taken in turn from this many stretches of them
  // the epilogue
  const float* bias;
  const void* residual;
  int64_t ld_res, ld_out, ld_pre, split_stride;  // (elements of out between splits)
  int res_f32, out_f32, act;
  void *out, *pre;
  int* status;
  uint64_t timeout_ns;
  int out_first;            // L2 gives up the output's lines before others
  int skip_cta;             // testing: the block that loads nothing (-1: none)
};

constexpr int kGemmRestart = 8;  // stages of 64 terms after which the accumulator starts again
constexpr int kGemmEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kGemmEpiWarps;

// The epilogue: element by element; so with a residual, by asynchronous copies; by TMA; by TMA with
// a residual that arrives a chunk ahead (in two slots of 8 KB a warp instead of 4 KB, for which the
// operands' ring gives up half its stages: as good as none, since such outputs are bounded by their
// bytes).
enum GemmEpilogue { kEpiElements, kEpiElementsF32, kEpiElementsBf16, kEpiTma, kEpiResidual };

template <int BN, int EPI, bool PAIR = false>
struct GemmShape {
  static constexpr int kSlots = EPI == kEpiResidual ? 2 : 1;  // of a warp
  static constexpr uint32_t kResidual = 4096;  // 32 x 32 elements, bf16 rows in five pieces of 16 bytes
  static constexpr uint32_t kSlot = EPI == kEpiResidual ? 8192 : EPI == kEpiElementsF32 || EPI == kEpiElementsBf16 ? 4096 + 2 * kResidual : 4096;
  static constexpr uint32_t kA = 128 * 64 * 2, kB = (PAIR ? BN / 2 : BN) * 64 * 2;
  static constexpr uint32_t kEpi = kGemmEpiWarps * kSlots * kSlot;
  static constexpr int kStages = (226 * 1024 - 1024 - 512 - kEpi) / (kA + kB) < 8
                                     ? (226 * 1024 - 1024 - 512 - kEpi) / (kA + kB)
                                     : 8;
  static constexpr uint32_t kOffB = kStages * kA;
  static constexpr uint32_t kOffEpi = kOffB + kStages * kB;
  static constexpr uint32_t kOffBar = kOffEpi + kEpi;
  static constexpr uint32_t kSmem = kOffBar + 512 + 1024;
  static_assert(kStages >= 2 && kSmem <= 227 * 1024, "shared memory of a block");
  static_assert((2 * kStages + 8 + kGemmEpiWarps * kSlots) * 8 <= 512, "barriers");
  static_assert(2 * BN <= 512, "tensor memory columns");
};

// 16 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const float (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2, %3}], [%4], %5;" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(z), "r"(src), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// until this thread's stores have read their shared memory; until they are done
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void st_shared_v4(uint32_t p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared(uint32_t p) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(p) : "memory");
  return v;
}

__device__ __forceinline__ float ld_shared_bf16(uint32_t p) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(p) : "memory");
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// f with a pointer of the elements' type: one branch for many loads, which else would wait for one another.
template <typename F>
__device__ __forceinline__ void with_type(const void* p, int f32, F f) {
  if (f32)
    f(static_cast<const float*>(p));
  else
    f(static_cast<const __nv_bfloat16*>(p));
}
template <typename F>
__device__ __forceinline__ void with_type(void* p, int f32, F f) {
  if (f32)
    f(static_cast<float*>(p));
  else
    f(static_cast<__nv_bfloat16*>(p));
}

// 32 accumulators of this lane's row: the bias of their columns (lane j holds column j's) added, to and
// from 128 bytes of shared memory of the lane's own at `line` (16-byte units in place u ^ (lane & 7)), and
// the activation.
__device__ __forceinline__ void epi_bias(float (&v)[32], float bias) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xFFFFFFFFu, bias, j);
}
__device__ __forceinline__ void epi_put32(const float (&v)[32], uint32_t line) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    st_shared_v4(line ^ (u << 4), __float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]),
                 __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
}
// The activation in registers: 1825 x 256 x 35840 to bf16 takes 80 us with sigmoid and 90 with tanh against 59
// without (by a loop over the line some 25 more); to fp32, whose exponentials are exact, 105 against 71.  GELU, of
// many more instructions, is such a loop, for one copy of its code: 32 of them cost every kernel registers and
// gained nothing (182 to 192 us).
__device__ __forceinline__ void epi_act(int act, int out_f32, float (&v)[32]) {
  auto all = [&](auto a, auto quick) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = act_value<decltype(a)::value, decltype(quick)::value>(v[j]);
  };
  auto by_type = [&](auto a) {
    if (out_f32)
      all(a, std::false_type());
    else
      all(a, std::true_type());
  };
  if (act == DSPARK_ACT_SIGMOID) {
    by_type(std::integral_constant<int, DSPARK_ACT_SIGMOID>());
  } else if (act == DSPARK_ACT_TANH) {
    all(std::integral_constant<int, DSPARK_ACT_TANH>(), std::false_type());
  } else if (act == DSPARK_ACT_RELU) {
    all(std::integral_constant<int, DSPARK_ACT_RELU>(), std::false_type());
  } else if (act == DSPARK_ACT_SILU) {
    by_type(std::integral_constant<int, DSPARK_ACT_SILU>());
  }
}
__device__ __forceinline__ void epi_gelu(uint32_t line) {
#pragma unroll 2
  for (int u = 0; u < 8; ++u) {
    const uint4 w = ld_shared_v4(line ^ (u << 4));
    st_shared_v4(line ^ (u << 4), __float_as_uint(act_value<DSPARK_ACT_GELU, false>(__uint_as_float(w.x))),
                 __float_as_uint(act_value<DSPARK_ACT_GELU, false>(__uint_as_float(w.y))),
                 __float_as_uint(act_value<DSPARK_ACT_GELU, false>(__uint_as_float(w.z))),
                 __float_as_uint(act_value<DSPARK_ACT_GELU, false>(__uint_as_float(w.w))));
  }
}
__device__ __forceinline__ void epi_get32(float (&v)[32], uint32_t line) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint4 w = ld_shared_v4(line ^ (u << 4));
    v[4 * u] = __uint_as_float(w.x), v[4 * u + 1] = __uint_as_float(w.y);
    v[4 * u + 2] = __uint_as_float(w.z), v[4 * u + 3] = __uint_as_float(w.w);
  }
}

// Units first, first + stride, ... of a product.
template <int BN, bool A_MN, bool B_MN, int EPI, bool PAIR>
__device__ __forceinline__ void gemm_units(const GemmArgs& g, const int64_t first, const int64_t stride) {
  using S = GemmShape<BN, EPI, PAIR>;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* full = bars;                   // [kStages]
  uint64_t* empty = bars + kStages;        // [kStages]
  uint64_t* acc_full = bars + 2 * kStages; // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2]
  uint64_t* drain = acc_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(acc_full + 6);
  uint64_t* res_full = acc_full + 7;       // [warps][kSlots]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the pair's first block issues its products, on its own `full` and `acc_empty`
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  constexpr int kRows = PAIR ? 256 : 128;  // of a tile
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], (PAIR ? 2 : 1) * kGemmEpiWarps);
    }
    mbar_init(drain, 1);
    for (int s = 0; s < kGemmEpiWarps * S::kSlots; ++s) mbar_init(&res_full[s], 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.a[0]);
    tma_prefetch_desc(&g.b[0]);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, 2 * BN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * BN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {  // both blocks' barriers are ready
    __syncwarp();
    cluster_sync();
  }
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // what the call's kernels before this one made; and the scratch is read to its end

  // unit u: tile (u % tiles_i, u / tiles_i % tiles_j), part u / (tiles_i tiles_j) of its stages, so
  // that blocks working at one time share their B tiles in L2
  const int64_t tiles = g.tiles_i * g.tiles_j;
  auto column = [&](int64_t t) {  // of tile t
    const int n = static_cast<int>(t / g.tiles_i);
    if (g.streams == 1) return n * BN;
    const int each = g.tiles_j / g.streams, more = g.tiles_j % g.streams;
    const int r = n < each * g.streams ? n % g.streams : n - each * g.streams;
    return (r * each + min(r, more) + n / g.streams) * BN;
  };

  if (warp == 0) {
    if (lane == 0 && static_cast<int>(blockIdx.x) != g.skip_cta) {
      const uint64_t pol = l2_policy_evict_normal();
      bool ok = true;
      uint32_t n = 0;  // stages filled
      for (int64_t u = first; u < g.units && ok; u += stride) {
        const int64_t t = u % tiles, sp = u / tiles;
        const int i0 = static_cast<int>((t % g.tiles_i) * kRows + rank * 128);
        const int j0 = column(t) + static_cast<int>(rank) * (BN / 2);
        const int64_t end = min(g.steps, (sp + 1) * g.per_split);
        // MN-major boxes of 64 rows or columns of the output, those of the tile that lie within it (what the
        // others would hold counts for outputs only that are not stored; filling them with zeros takes as long
        // as two loads: dW of 64 x 50912 from 276 rows 83 us, without 30)
        constexpr int kBoxesB = PAIR ? BN / 128 : BN / 64;
        auto inside = [](int64_t extent, int64_t at, int most) {
          return static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(most), (extent - at + 63) / 64)));
        };
        const int boxes_a = A_MN ? inside(g.I, i0, 2) : 2, boxes_b = B_MN ? inside(g.J, j0, kBoxesB) : kBoxesB;
        uint32_t bytes = boxes_a * (S::kA / 2) + boxes_b * (S::kB / kBoxesB);
        if constexpr (PAIR)
          bytes += (A_MN ? inside(g.I, i0 + 128, 2) : 2) * (S::kA / 2) + (B_MN ? inside(g.J, j0 + BN / 2, kBoxesB) : kBoxesB) * (S::kB / kBoxesB);
        for (int64_t k = sp * g.per_split; k < end; ++k, ++n) {
          const uint32_t s = n % kStages;
          if (!mbar_wait(&empty[s], ((n / kStages) & 1) ^ 1, g.timeout_ns, abort_flag)) {
            ok = false;
            break;
          }
          const int part = k < g.blocks_k ? 0 : k < 2 * g.blocks_k ? 1 : 2;
          const int k0 = static_cast<int>(k - part * g.blocks_k) * 64;
          const CUtensorMap* const ma = &g.a[g.a_parts > 1 ? part : 0];
          const CUtensorMap* const mb = &g.b[g.b_parts > 1 ? part : 0];
          uint8_t* const sa = smem + s * S::kA;
          uint8_t* const sb = smem + S::kOffB + s * S::kB;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
          const uint32_t bar = PAIR ? cluster_addr(&full[s], 0) : 0;
          auto load = [&](uint8_t* to, const CUtensorMap* map, int x, int y) {
            if constexpr (PAIR)
              tma_load_2d_pair(to, map, x, y, bar, pol);
            else
              tma_load_2d(to, map, x, y, &full[s], pol);
          };
          if constexpr (A_MN) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (c < boxes_a) load(sa + c * 8192, ma, i0 + c * 64, k0);
          } else {
            load(sa, ma, k0, i0);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int c = 0; c < kBoxesB; ++c)
              if (c < boxes_b) load(sb + c * 8192, mb, j0 + c * 64, k0);
          } else {
            load(sb, mb, k0, j0);
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        record_error(g.status, kStatusTimeout);
        // copies under way end first (a pair's second block's are over when the first one's wait for
        // both is, or has run out; it meets the first at the end)
        for (uint32_t j = 0; rank == 0 && j < kStages && j < n; ++j) {
          const uint32_t m = n - 1 - j;
          if (!mbar_wait(&full[m % kStages], (m / kStages) & 1, g.timeout_ns, nullptr)) break;
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(kRows, BN, A_MN, B_MN);
      auto commit = [](uint64_t* bar) {
        if constexpr (PAIR)
          umma_commit_pair(bar);
        else
          umma_commit(bar);
      };
      bool ok = true, issued = false;
      uint32_t n = 0, i = 0;
      for (int64_t u = first; u < g.units && ok; u += stride) {
        const int64_t sp = u / tiles;
        const int64_t end = min(g.steps, (sp + 1) * g.per_split);
        for (int64_t k0 = sp * g.per_split; k0 < end && ok; k0 += kGemmRestart, ++i) {
          const uint32_t buf = i & 1;
          if (!(PAIR ? mbar_wait_cluster(&acc_empty[buf], ((i >> 1) & 1) ^ 1, g.timeout_ns, abort_flag)
                     : mbar_wait(&acc_empty[buf], ((i >> 1) & 1) ^ 1, g.timeout_ns, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + buf * BN;
          for (int64_t k = k0; k < min(end, k0 + kGemmRestart); ++k, ++n) {
            const uint32_t s = n % kStages;
            if (!mbar_wait(&full[s], (n / kStages) & 1, g.timeout_ns, abort_flag, 20u)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a0 = smem_addr(smem + s * S::kA), b0 = smem_addr(smem + S::kOffB + s * S::kB);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              // 16 terms: 32 bytes along K-major rows, two groups of eight rows of MN-major boxes
              const uint64_t da = A_MN ? smem_desc(a0 + kk * 2048, 8192, 1024) : smem_desc(a0 + kk * 32, 16, 1024);
              const uint64_t db = B_MN ? smem_desc(b0 + kk * 2048, 8192, 1024) : smem_desc(b0 + kk * 32, 16, 1024);
              const uint32_t add = k > k0 || kk > 0 ? 1u : 0u;
              if constexpr (PAIR)
                umma_bf16_pair(d, da, db, idesc, add);
              else
                umma_bf16(d, da, db, idesc, add);
            }
            issued = true;
            commit(&empty[s]);
          }
          if (ok) commit(&acc_full[buf]);
        }
      }
      if (!ok) {
        *abort_flag = 1;
        record_error(g.status, kStatusTimeout);
        if (issued) {  // products under way end before TMEM is freed
          commit(drain);
          mbar_wait(drain, 0, g.timeout_ns, nullptr);
        }
      }
    }
  } else {
    // warps of a TMEM quadrant take its rows; of two such warps each takes every other 64 columns
    const int q = warp & 3, e = warp - 2, group = e >> 2;
    constexpr int kChunks = BN / 64, kRound = kChunks < 2 ? 2 : kChunks;  // (of 64 columns the second group has none)
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint64_t pol_out = g.out_first ? l2_policy_evict_first() : l2_policy_evict_normal();
    const uint32_t slots = smem_addr(smem + S::kOffEpi + e * S::kSlots * S::kSlot);
    const uint32_t own = 128 * lane + ((lane & 7) << 4);  // this lane's line of a 4 KB box
    constexpr bool kCopied = EPI == kEpiElementsF32 || EPI == kEpiElementsBf16, kElements = EPI == kEpiElements || kCopied;
    auto place = [&](int64_t u, int64_t& row0, int& col0) {
      const int64_t t = u % tiles;
      row0 = (t % g.tiles_i) * kRows + rank * 128 + q * 32;
      col0 = column(t);
    };
    uint32_t phases = 0, pending = 0;  // bit a slot: of its barrier; a load is under way
    // the residual of chunk c of unit u on its way into a slot (fp32: both boxes; bf16: the second)
    auto load_residual = [&](int64_t u, int c, int slot) {
      if (EPI != kEpiResidual || u >= g.units) return;
      int64_t row0;
      int col0;
      place(u, row0, col0);
      const int col = col0 + 64 * c;
      if (row0 >= g.I || col >= g.J) return;
      pending |= 1u << slot;
      if (lane == 0) {
        uint64_t* const bar = &res_full[e * S::kSlots + slot];
        uint8_t* const to = smem + S::kOffEpi + (e * S::kSlots + slot) * S::kSlot;
        const uint64_t pol = l2_policy_evict_normal();
        mbar_arrive_expect_tx(bar, g.res_f32 ? 8192 : 4096);
        if (g.res_f32) {
          tma_load_2d(to, &g.res_map, col, static_cast<int>(row0), bar, pol);
          tma_load_2d(to + 4096, &g.res_map, col + 32, static_cast<int>(row0), bar, pol);
        } else {
          tma_load_2d(to + 4096, &g.res_map, col, static_cast<int>(row0), bar, pol);
        }
      }
    };
    // (position n + kSlots of the warp's chunks, from chunk c of unit u)
    auto load_later = [&](int64_t u, int c, int slot) {
      int k = c + 2 * S::kSlots;
      for (; k >= kRound; k -= kRound) u += stride;
      load_residual(u, k, slot);
    };
    // a residual whose rows TMA cannot take: the 32 x 32 elements of half h of chunk c, each row the pieces of
    // 16 bytes that hold it, copied asynchronously
    auto copy_residual = [&](int64_t u, int c, int h, int slot) {
      if constexpr (kCopied) {
        if (u < g.units && group < kChunks) {
          int64_t row0;
          int col0;
          place(u, row0, col0);
          const int cc = col0 + 64 * c + 32 * h, cols = min(32, g.J - cc);
          const int rows = cols > 0 ? static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(32), g.I - row0))) : 0;
          uint8_t* const to = smem + S::kOffEpi + e * S::kSlot + 4096 + S::kResidual * slot;
          if constexpr (EPI == kEpiElementsF32) {
            const float* p = static_cast<const float*>(g.residual) + row0 * g.ld_res + cc + lane;
            const int mine = lane < cols ? rows : 0;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (k < mine) cp_async_4(to + 128 * k + 4 * lane, p);
              p += g.ld_res;
            }
          } else {
            const auto start = reinterpret_cast<uintptr_t>(g.residual);
            const uintptr_t corner = start + 2 * (row0 * g.ld_res + cc);
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              const int k = (32 * i + lane) / 5, piece = (32 * i + lane) % 5;
              const uintptr_t row = corner + 2 * k * g.ld_res, end = row + 2 * cols;
              const uintptr_t from = (row & ~static_cast<uintptr_t>(15)) + 16 * piece;
              if (k >= rows || from >= end) continue;
              uint8_t* const at = to + 16 * (5 * k + piece);
              if (from >= start) {
                cp_async_16_zfill(at, reinterpret_cast<const void*>(from), static_cast<int>(min(end - from, static_cast<uintptr_t>(16))));
              } else {  // (nothing before the first element is touched)
                for (uintptr_t f = start; f < min(end, from + 16); f += 2)
                  *reinterpret_cast<__nv_bfloat16*>(at + (f - from)) = *reinterpret_cast<const __nv_bfloat16*>(f);
              }
            }
          }
        }
        cp_async_commit();
      }
    };
#pragma unroll 1
    for (int h = 0; h < 2; ++h) copy_residual(first, group, h, h);
    bool ok = true;
    uint32_t i = 0, n = 0;
    if (EPI == kEpiResidual && group < kChunks) {
      int64_t u = first;
      int c = group;
      for (int s = 0; s < S::kSlots; ++s) {
        for (; c >= kRound; c -= kRound) u += stride;
        load_residual(u, c, s);
        c += 2;
      }
    }
    auto accumulator_free = [&](uint32_t b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          mbar_arrive_cluster(cluster_addr(&acc_empty[b], 0));
        else
          mbar_arrive(&acc_empty[b]);
      }
    };
    for (int64_t u = first; u < g.units; u += stride, ++i) {
      int64_t row0;
      int col0;
      place(u, row0, col0);
      const int sp = static_cast<int>(u / tiles);
      // all accumulators of the unit but the last are added up in registers, and their sum joins that one
      const int64_t end = min(g.steps, (sp + 1) * g.per_split), stages = end - sp * g.per_split;
      constexpr int kMine = BN >= 128 ? BN / 32 : 4;  // 16-column pieces of a warp
      if (stages > kGemmRestart) {
        float sum[kMine][16];
#pragma unroll
        for (int p = 0; p < kMine; ++p)
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[p][j] = 0.f;
        auto piece = [&](uint32_t b, int p) { return lane_base + b * BN + 64 * (group + 2 * (p / 4)) + 16 * (p % 4); };
        for (int64_t left = stages;; left -= kGemmRestart) {
          const uint32_t b = i & 1;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[b], (i >> 1) & 1, g.timeout_ns, abort_flag));
          if (!ok) break;
          tc_fence_after();
          if (group < kChunks) {
#pragma unroll
            for (int p = 0; p < kMine; ++p) {
              uint32_t v[16];
              tmem_ld_x16(piece(b, p), v);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[p][j] += __uint_as_float(v[j]);
            }
          }
          if (left <= kGemmRestart) {
            if (group < kChunks) {
#pragma unroll
              for (int p = 0; p < kMine; ++p) tmem_st_x16(piece(b, p), sum[p]);
            }
            break;
          }
          accumulator_free(b);
          ++i;
        }
        if (!ok) break;
        tmem_wait_st();
      } else {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[i & 1], (i >> 1) & 1, g.timeout_ns, abort_flag));
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t b = i & 1;
#pragma unroll 1
      for (int c = group; c < kChunks; c += 2, ++n) {
        const int col = col0 + 64 * c, slot = n % S::kSlots;
        if (!kElements && (row0 >= g.I || col >= g.J)) {
          load_later(u, c, slot);
          continue;
        }
        const uint32_t box = slots + slot * S::kSlot, line = box + own;
        if constexpr (!kElements) {
          if (pending >> slot & 1) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&res_full[e * S::kSlots + slot], phases >> slot & 1, g.timeout_ns, abort_flag));
            if (!ok) break;
            phases ^= 1u << slot;
            pending &= ~(1u << slot);
          } else {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
          }
          // columns [col + shift, ...) of the slot's box at `from` on their way out
          auto store = [&](const CUtensorMap* map, uint32_t from, int shift) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (col + shift < g.J) tma_store_3d(map, from, col + shift, static_cast<int>(row0), sp, pol_out);
              bulk_commit();
            }
          };
          auto pass = [&](bool last, const CUtensorMap* map) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              float v[32], r[32];
              tmem_ld_x32(lane_base + b * BN + 64 * c + 32 * h, reinterpret_cast<uint32_t*>(v));
              const int cc = col + 32 * h;
              const float bias = g.bias != nullptr && cc + lane < g.J ? __ldg(g.bias + cc + lane) : 0.f;
              // an fp32 half is a box: its own beside a residual, else the slot's one, again
              const uint32_t half_box = EPI == kEpiResidual ? box + (h << 12) : box, half = half_box + own;
              if constexpr (EPI == kEpiResidual) {
                if (g.res_f32) {
                  epi_get32(r, half);
                } else {
#pragma unroll
                  for (int u8 = 0; u8 < 4; ++u8) {
                    const uint4 w = ld_shared_v4((line + 4096) ^ ((4 * h + u8) << 4));
                    widen2(w.x, r[8 * u8], r[8 * u8 + 1]);
                    widen2(w.y, r[8 * u8 + 2], r[8 * u8 + 3]);
                    widen2(w.z, r[8 * u8 + 4], r[8 * u8 + 5]);
                    widen2(w.w, r[8 * u8 + 6], r[8 * u8 + 7]);
                  }
                }
              }
              tmem_wait_ld();
              if (g.bias != nullptr) epi_bias(v, bias);
              if (last) epi_act(g.act, g.out_f32, v);
              if (last && g.act == DSPARK_ACT_GELU) {
                // (the slot's one box may hold the first half's bf16 outputs: they are kept meanwhile)
                uint4 keep[EPI == kEpiResidual ? 1 : 4];
                if constexpr (EPI != kEpiResidual) {
#pragma unroll
                  for (int u8 = 0; u8 < 4; ++u8) keep[u8] = ld_shared_v4(line ^ (u8 << 4));
                }
                epi_put32(v, half);
                epi_gelu(half);
                epi_get32(v, half);
                if constexpr (EPI != kEpiResidual) {
#pragma unroll
                  for (int u8 = 0; u8 < 4; ++u8) st_shared_v4(line ^ (u8 << 4), keep[u8].x, keep[u8].y, keep[u8].z, keep[u8].w);
                }
              }
              if constexpr (EPI == kEpiResidual) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] += r[j];
              }
              if (g.out_f32) {
                epi_put32(v, half);
                store(map, half_box, 32 * h);
                if (EPI != kEpiResidual && h == 0) {
                  if (lane == 0) bulk_wait_read();
                  __syncwarp();
                }
              } else {
#pragma unroll
                for (int u8 = 0; u8 < 4; ++u8)
                  st_shared_v4(line ^ ((4 * h + u8) << 4), narrow2(v[8 * u8], v[8 * u8 + 1]),
                               narrow2(v[8 * u8 + 2], v[8 * u8 + 3]), narrow2(v[8 * u8 + 4], v[8 * u8 + 5]),
                               narrow2(v[8 * u8 + 6], v[8 * u8 + 7]));
                if (h == 1) store(map, box, 0);
              }
            }
          };
          if (EPI == kEpiTma && g.pre != nullptr) {
            pass(false, &g.pre_map);
            if (lane == 0) bulk_wait_read();
            __syncwarp();
          }
          pass(true, &g.out_map);
          if constexpr (EPI == kEpiResidual) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
            load_later(u, c, slot);
          }
        } else {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int cc = col + 32 * h;
            const int rows = static_cast<int>(min(static_cast<int64_t>(32), g.I - row0));
            if (cc < g.J && rows > 0) {
              float v[32];
              tmem_ld_x32(lane_base + b * BN + 64 * c + 32 * h, reinterpret_cast<uint32_t*>(v));
              const float bias = g.bias != nullptr && cc + lane < g.J ? __ldg(g.bias + cc + lane) : 0.f;
              const bool in = cc + lane < g.J;
              tmem_wait_ld();
              if (g.bias != nullptr) epi_bias(v, bias);
              __syncwarp();
              epi_put32(v, line);
              // now by columns: element (k, lane)
              auto put = [&](void* to, int64_t ld, bool last) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = ld_shared(box + 128 * k + ((((lane >> 2) ^ (k & 7)) << 4) | ((lane & 3) << 2)));
                if (last) epi_act(g.act, g.out_f32, v);
                if constexpr (kCopied) {
                  if (last) {
                    cp_async_wait_group<1>();
                    __syncwarp();
                    const uint32_t from = box + 4096 + S::kResidual * h;
                    if constexpr (EPI == kEpiElementsF32) {
#pragma unroll
                      for (int k = 0; k < 32; ++k) v[k] += ld_shared(from + 128 * k + 4 * lane);
                    } else {
                      const auto row = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(g.residual) + 2 * (row0 * g.ld_res + cc));
                      const uint32_t pitch = 2 * static_cast<uint32_t>(g.ld_res);
#pragma unroll
                      for (int k = 0; k < 32; ++k) v[k] += ld_shared_bf16(from + 80 * k + (row + k * pitch & 15) + 2 * lane);
                    }
                  }
                }
                with_type(to, g.out_f32, [&](auto p) {
                  p += sp * g.split_stride + row0 * ld + cc + lane;
#pragma unroll
                  for (int k = 0; k < 32; ++k) {
                    if (in && k < rows) store1(p, v[k]);
                    p += ld;
                  }
                });
                __syncwarp();
              };
              if (g.pre != nullptr) put(g.pre, g.ld_pre, false);
              if (g.act == DSPARK_ACT_GELU) epi_gelu(line);
              put(g.out, g.ld_out, true);
            }
            // then on to the copies of the next chunk's same half
            const bool here = c + 2 < kRound;
            copy_residual(here ? u : u + stride, here ? c + 2 : group, h, h);
          }
        }
      }
      if (!ok) break;
      accumulator_free(b);
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      record_error(g.status, kStatusTimeout);
    }
    if constexpr (kCopied) cp_async_wait_all();
    if constexpr (!kElements) {
      // copies under way end before the block does
      for (int s = 0; s < S::kSlots; ++s)
        if (pending >> s & 1) mbar_wait(&res_full[e * S::kSlots + s], phases >> s & 1, g.timeout_ns, nullptr);
      if (lane == 0) bulk_wait();
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {  // neither block's shared memory is in use any more
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, 2 * BN);
    else
      tmem_dealloc(tmem, 2 * BN);
  }
}

template <int BN, bool A_MN, bool B_MN, int EPI, bool PAIR = false>
__global__ void __launch_bounds__(kGemmThreads, 1) linear_gemm_kernel(const __grid_constant__ GemmArgs g) {
  if constexpr (PAIR)
    gemm_units<BN, A_MN, B_MN, EPI, true>(g, blockIdx.x / 2, gridDim.x / 2);
  else
    gemm_units<BN, A_MN, B_MN, EPI, false>(g, blockIdx.x, gridDim.x);
}

// Both products of a gradient at once: pairs [0, dx_pairs) work on dz W^T, the others on x^T dz, and walk
// through the columns of dz side by side, so that what one has read of it the other finds in L2.
struct GemmBoth {
  GemmArgs dx, dw;
  int dx_pairs;
};
__global__ void __launch_bounds__(kGemmThreads, 1) linear_both_kernel(const __grid_constant__ GemmBoth b) {
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  if (pair < b.dx_pairs)
    gemm_units<256, false, false, kEpiTma, true>(b.dx, pair, b.dx_pairs);
  else
    gemm_units<256, true, true, kEpiTma, true>(b.dw, pair - b.dx_pairs, pairs - b.dx_pairs);
}

}  // namespace dspark
