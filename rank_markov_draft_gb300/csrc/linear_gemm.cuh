// linear_gemm.cuh -- one matrix product on the tensor cores, with the linear layers' epilogue:
//   out(i, j) = act(sum_k A(i, k) B(k, j) + bias_j) + residual(i, j).
//
// A persistent block an SM walks over units (a tile of 128 x BN outputs, and a part of the
// contraction where the tiles alone would leave SMs idle).  One lane fills a ring of stages of 64
// terms by TMA (128-byte swizzle), one issues tcgen05.mma (M = 128, N = BN, accumulator in TMEM), and
// eight warps take finished accumulators through the epilogue while the next unit's products run into
// the other half of TMEM.  Either operand may lie with the contraction contiguous (K-major) or with
// its own index contiguous (MN-major), so x W, dz W^T and x^T dz read their matrices as they are.
//
// An operand may come in two parts, added up in the accumulator: A = A_0 + A_1 doubles the terms.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "activation.cuh"
#include "async_copy.cuh"
#include "sm103.cuh"
#include "typed.cuh"

namespace dspark {

struct GemmArgs {
  CUtensorMap a[2], b[2];
  int a_parts, b_parts;     // 1, or 2 of one of them
  int64_t I;                // rows and columns of the output
  int J;
  int64_t tiles_i, units;
  int tiles_j, splits;
  int64_t steps, per_split; // stages of a tile (all parts), of a unit
  int64_t blocks_k;         // stages of a part
  // the epilogue
  const float* bias;
  const void* residual;
  int64_t ld_res, ld_out, ld_pre, split_stride;  // (elements of out between splits)
  int res_f32, out_f32, act;
  void *out, *pre;
  int* status;
  uint64_t timeout_ns;
  int skip_cta;             // testing: the block that loads nothing (-1: none)
};

constexpr int kGemmEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kGemmEpiWarps;
template <int BN>
struct GemmShape {
  static constexpr uint32_t kA = 128 * 64 * 2, kB = BN * 64 * 2;
  static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;  // 192 KB
  static constexpr uint32_t kOffB = kStages * kA;
  static constexpr uint32_t kOffEpi = kOffB + kStages * kB;
  static constexpr uint32_t kOffBar = kOffEpi + kGemmEpiWarps * 4096;
  static constexpr uint32_t kSmem = kOffBar + 256 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of a block");
  static_assert(2 * BN <= 512, "tensor memory columns");
};

// A warp's 32 x 32 outputs as coalesced pieces: four neighbours of a row a lane (VEC: rows allow
// 16-byte vectors of fp32 and 8-byte ones of bf16), or one.
template <bool VEC>
struct EpiMap {
  static constexpr int kIters = VEC ? 8 : 32;
  __device__ static __forceinline__ int row(int i, int lane) { return VEC ? 4 * i + lane / 8 : i; }
  __device__ static __forceinline__ int col(int lane) { return VEC ? 4 * (lane % 8) : lane; }
};

// The word of element (r, c) in a warp's 32 x 32 buffer: 16-byte units XORed with the row, so that
// both a lane writing its row and lanes reading along one meet no bank twice.
__device__ __forceinline__ int epi_word(int r, int c) { return 32 * r + (((c >> 2) ^ (r & 7)) << 2) + (c & 3); }

template <bool VEC>
__device__ __forceinline__ void epi_store(void* p, int f32, int64_t at, const float (&v)[4]) {
  if constexpr (VEC) {
    if (f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + at) =
          make_uint2(narrow2(v[0], v[1]), narrow2(v[2], v[3]));
  } else {
    if (f32)
      static_cast<float*>(p)[at] = v[0];
    else
      static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v[0]);
  }
}

// Residual elements as they lie in memory.
template <bool VEC>
struct EpiRaw {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, int f32, int64_t at) {
    if constexpr (VEC) {
      if (f32) {
        v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
      } else {
        const uint2 t = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at);
        v.x = t.x, v.y = t.y;
      }
    } else {
      v.x = f32 ? static_cast<const uint32_t*>(p)[at] : static_cast<const uint16_t*>(p)[at];
    }
  }
  __device__ __forceinline__ void add(int f32, float (&z)[4]) const {
    if constexpr (VEC) {
      if (f32) {
        z[0] += __uint_as_float(v.x), z[1] += __uint_as_float(v.y);
        z[2] += __uint_as_float(v.z), z[3] += __uint_as_float(v.w);
      } else {
        float a, b, c, d;
        widen2(v.x, a, b);
        widen2(v.y, c, d);
        z[0] += a, z[1] += b, z[2] += c, z[3] += d;
      }
    } else {
      z[0] += f32 ? __uint_as_float(v.x) : __uint_as_float(v.x << 16);
    }
  }
};

template <int BN, bool A_MN, bool B_MN, bool VEC>
__global__ void __launch_bounds__(kGemmThreads, 1) linear_gemm_kernel(const __grid_constant__ GemmArgs g) {
  using S = GemmShape<BN>;
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], kGemmEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&g.a[0]);
    tma_prefetch_desc(&g.b[0]);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // unit u: tile (u % tiles_i, u / tiles_i % tiles_j), part u / (tiles_i tiles_j) of its stages, so
  // that blocks working at one time share their B tiles in L2
  const int64_t tiles = g.tiles_i * g.tiles_j;

  if (warp == 0) {
    if (lane == 0 && static_cast<int>(blockIdx.x) != g.skip_cta) {
      const uint64_t pol = l2_policy_evict_normal();
      bool ok = true;
      uint32_t n = 0;  // stages filled
      for (int64_t u = blockIdx.x; u < g.units && ok; u += gridDim.x) {
        const int64_t t = u % tiles, sp = u / tiles;
        const int i0 = static_cast<int>(t % g.tiles_i) * 128, j0 = static_cast<int>(t / g.tiles_i) * BN;
        const int64_t end = min(g.steps, (sp + 1) * g.per_split);
        for (int64_t k = sp * g.per_split; k < end; ++k, ++n) {
          const uint32_t s = n % kStages;
          if (!mbar_wait(&empty[s], ((n / kStages) & 1) ^ 1, g.timeout_ns, abort_flag)) {
            ok = false;
            break;
          }
          const int part = k >= g.blocks_k ? 1 : 0;
          const int k0 = static_cast<int>(k - (part ? g.blocks_k : 0)) * 64;
          const CUtensorMap* const ma = &g.a[g.a_parts == 2 ? part : 0];
          const CUtensorMap* const mb = &g.b[g.b_parts == 2 ? part : 0];
          uint8_t* const sa = smem + s * S::kA;
          uint8_t* const sb = smem + S::kOffB + s * S::kB;
          mbar_arrive_expect_tx(&full[s], S::kA + S::kB);
          if constexpr (A_MN) {
            tma_load_2d(sa, ma, i0, k0, &full[s], pol);
            tma_load_2d(sa + 8192, ma, i0 + 64, k0, &full[s], pol);
          } else {
            tma_load_2d(sa, ma, k0, i0, &full[s], pol);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int c = 0; c < BN / 64; ++c)
              tma_load_2d(sb + c * 8192, mb, j0 + c * 64, k0, &full[s], pol);
          } else {
            tma_load_2d(sb, mb, k0, j0, &full[s], pol);
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        record_error(g.status, kStatusTimeout);
        for (uint32_t j = 0; j < kStages && j < n; ++j) {  // copies under way end first
          const uint32_t m = n - 1 - j;
          mbar_wait(&full[m % kStages], (m / kStages) & 1, g.timeout_ns, nullptr);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, BN, A_MN, B_MN);
      bool ok = true, issued = false;
      uint32_t n = 0, i = 0;
      for (int64_t u = blockIdx.x; u < g.units && ok; u += gridDim.x, ++i) {
        const int64_t sp = u / tiles;
        const int64_t k_begin = sp * g.per_split, end = min(g.steps, (sp + 1) * g.per_split);
        const uint32_t buf = i & 1;
        if (!mbar_wait(&acc_empty[buf], ((i >> 1) & 1) ^ 1, g.timeout_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * BN;
        for (int64_t k = k_begin; k < end; ++k, ++n) {
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
            umma_bf16(d, da, db, idesc, k > k_begin || kk > 0 ? 1u : 0u);
          }
          issued = true;
          umma_commit(&empty[s]);
        }
        if (ok) umma_commit(&acc_full[buf]);
      }
      if (!ok) {
        *abort_flag = 1;
        record_error(g.status, kStatusTimeout);
        if (issued) {  // products under way end before TMEM is freed
          umma_commit(drain);
          mbar_wait(drain, 0, g.timeout_ns, nullptr);
        }
      }
    }
  } else {
    using Map = EpiMap<VEC>;
    constexpr int kChunks = BN / 64;
    const int q = warp & 3, half = (warp - 2) >> 2;
    float* const buf32 = reinterpret_cast<float*>(smem + S::kOffEpi + (warp - 2) * 4096);
    const int col_l = Map::col(lane);
    uint32_t i = 0;
    for (int64_t u = blockIdx.x; u < g.units; u += gridDim.x, ++i) {
      const int64_t t = u % tiles, sp = u / tiles;
      const int64_t row0 = (t % g.tiles_i) * 128 + q * 32;
      const int col0 = static_cast<int>(t / g.tiles_i) * BN + half * (BN / 2);
      const int rows = static_cast<int>(min(static_cast<int64_t>(32), g.I - row0));  // (may be <= 0)
      const int64_t out0 = sp * g.split_stride;
      EpiRaw<VEC> res[Map::kIters];
      auto load_residual = [&](int c) {
        const int col = col0 + 32 * c + col_l;
#pragma unroll
        for (int k = 0; k < Map::kIters; ++k) {
          const int r = Map::row(k, lane);
          if (r < rows && col < g.J) res[k].load(g.residual, g.res_f32, (row0 + r) * g.ld_res + col);
        }
      };
      if (g.residual != nullptr) load_residual(0);
      const uint32_t b = i & 1;
      const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&acc_full[b], (i >> 1) & 1, g.timeout_ns, abort_flag));
      if (!ok) {
        if (lane == 0) {
          *abort_flag = 1;
          record_error(g.status, kStatusTimeout);
        }
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t v[32];
        tmem_ld_x32(tmem + b * BN + half * (BN / 2) + 32 * c + (static_cast<uint32_t>(q * 32) << 16), v);
        tmem_wait_ld();
        if (c == kChunks - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[b]);
        }
        const int cc = col0 + 32 * c;
        if (cc >= g.J || rows <= 0) continue;
        if (g.bias != nullptr) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (cc + j < g.J) v[j] = __float_as_uint(__uint_as_float(v[j]) + __ldg(g.bias + cc + j));
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(buf32 + epi_word(lane, 4 * j)) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        __syncwarp();
        const int col = cc + col_l;
        auto piece = [&](int k, float (&z)[4]) {
          const float* const p = buf32 + epi_word(Map::row(k, lane), col_l);
          if constexpr (VEC) {
            const float4 f = *reinterpret_cast<const float4*>(p);
            z[0] = f.x, z[1] = f.y, z[2] = f.z, z[3] = f.w;
          } else {
            z[0] = *p;
          }
        };
        if (g.pre != nullptr) {
#pragma unroll 4
          for (int k = 0; k < Map::kIters; ++k) {
            const int r = Map::row(k, lane);
            float z[4];
            piece(k, z);
            if (r < rows && col < g.J) epi_store<VEC>(g.pre, g.out_f32, (row0 + r) * g.ld_pre + col, z);
          }
        }
        if (g.act != DSPARK_ACT_NONE) {
          // in the buffer, each lane its row: one copy of the functions' code
          __syncwarp();
#pragma unroll 1
          for (int j = 0; j < 32; ++j) {
            float* const p = buf32 + 32 * lane + (j ^ lane);
            *p = act_value(g.act, *p);
          }
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < Map::kIters; ++k) {
          const int r = Map::row(k, lane);
          float z[4];
          piece(k, z);
          if (g.residual != nullptr) res[k].add(g.res_f32, z);
          if (r < rows && col < g.J) epi_store<VEC>(g.out, g.out_f32, out0 + (row0 + r) * g.ld_out + col, z);
        }
        if (c + 1 < kChunks && g.residual != nullptr) load_residual(c + 1);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 2 * BN);
  }
}

}  // namespace dspark
