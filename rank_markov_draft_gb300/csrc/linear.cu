// linear.cu -- y = act(x W + bias) + residual, and the gradients of x, W and the bias.
//
// The heads' projections (h Wa, h Wg; equivalence page, "What the two methods do") and calibrated
// logits (U + s W2), forward and backward.  The products are linear_gemm.cuh's; here are the choice of
// tiles and splits, the joining of splits, and what the operands need first: rows on 16-byte
// boundaries for TMA, and dz = dy act'(pre) as bf16 numbers.

#include <algorithm>
#include <type_traits>

#include "dependent.h"
#include "linear_gemm.cuh"
#include "split_jobs.h"
#include "step.h"
#include "tensor_map.h"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

constexpr int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// ------------------------------------------------------------------ joining of splits
// The epilogue over sums of `splits` partials [splits][I][ld_part], in their order; four columns a
// thread.
struct JoinArgs {
  const float* part;
  int64_t I, ld_part, stride;
  int J, splits;
  const float* bias;
  const void* residual;
  int64_t ld_res, ld_out, ld_pre;
  int res_f32, out_f32, act, vec;
  void *out, *pre;
};

__global__ void __launch_bounds__(256) linear_join_kernel(JoinArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int per_row = (a.J + 3) / 4;
  const int64_t n = a.I * per_row;
  for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < n; e += gridDim.x * 256ll) {
    const int64_t row = e / per_row;
    const int c = static_cast<int>(e - row * per_row) * 4;
    const float* p = a.part + row * a.ld_part + c;
    float z[4] = {};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float4 f = __ldcs(reinterpret_cast<const float4*>(p + s * a.stride));
      z[0] += f.x, z[1] += f.y, z[2] += f.z, z[3] += f.w;
    }
    const int m = min(4, a.J - c);
    float r[4] = {};
    if (a.residual != nullptr)
      with_type(a.residual, a.res_f32, [&](auto q) {
        q += row * a.ld_res + c;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < m) r[j] = load1(q + j);
      });
    if (a.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < m) z[j] += a.bias[c + j];
    }
    auto put = [&](void* dst, int64_t ld) {
      with_type(dst, a.out_f32, [&](auto q) {
        q += row * ld + c;
        if (a.vec) {
          if constexpr (sizeof(*q) == 4)
            *reinterpret_cast<float4*>(q) = make_float4(z[0], z[1], z[2], z[3]);
          else
            *reinterpret_cast<uint2*>(q) = make_uint2(narrow2(z[0], z[1]), narrow2(z[2], z[3]));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < m) store1(q + j, z[j]);
        }
      });
    };
    if (a.pre != nullptr) put(a.pre, a.ld_pre);
    with_act(a.act, [&](auto act) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        z[j] = a.out_f32 ? act_value<decltype(act)::value, false>(z[j]) : act_value<decltype(act)::value, true>(z[j]);
    });
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] += r[j];
    put(a.out, a.ld_out);
  }
}

// ------------------------------------------------------------------ dz, and rows for TMA
// src act'(pre) as the sum of one bf16 number or three (8 bits of it each), rows ld_dst apart, and the
// column sums of a block's rows.  Each of them may be left out.
struct SplitArgs {
  const void *src, *pre;
  int64_t rows, ld_src, ld_pre, ld_dst;
  int cols, src_f32, pre_f32, act, rows_per_block, vec;
  bf16* part[3];
  float* sums;  // [row blocks][cols]
};


// Eight neighbours from an address that allows no vectors, of a matrix that ends before `last`: the
// 16-byte pieces around them, of which the last is the next lane's first, moved into place. (Lanes that
// have no such pieces inside the matrix read element by element; all lanes of a warp call this.)
template <typename T>
__device__ __forceinline__ void load8_shifted(const T* p, const T* start, const T* last, bool use, float (&v)[8]) {
  constexpr int kOwn = sizeof(T) / 2;  // pieces of 16 bytes in eight elements
  const uintptr_t at = reinterpret_cast<uintptr_t>(p), piece = at & ~static_cast<uintptr_t>(15);
  const uint32_t off = static_cast<uint32_t>(at - piece) / sizeof(T);
  const bool whole = use && piece >= reinterpret_cast<uintptr_t>(start) &&
                     piece + 16 * (kOwn + 1) <= reinterpret_cast<uintptr_t>(last);
  uint32_t w[4 * kOwn + 4];
#pragma unroll
  for (int k = 0; k < kOwn + 1; ++k) {
    uint4 x = make_uint4(0, 0, 0, 0);
    // (a lane's first piece serves its neighbour too, so it is read whenever it lies inside)
    const bool inside = piece >= reinterpret_cast<uintptr_t>(start) && piece + 16 * (k + 1) <= reinterpret_cast<uintptr_t>(last);
    if (k < kOwn ? inside && (use || k == 0) : whole && (threadIdx.x & 31) == 31)
      x = reinterpret_cast<const uint4*>(piece)[k];
    w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w[j], 1);
    if ((threadIdx.x & 31) != 31) w[4 * kOwn + j] = next;
  }
  constexpr int kWords = 4 * kOwn + 4;
  const uint32_t words = sizeof(T) == 4 ? off : off / 2;
#pragma unroll
  for (int s = 2; s > 0; s /= 2)
    if (words & s) {
#pragma unroll
      for (int j = 0; j + s < kWords; ++j) w[j] = w[j + s];
    }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
  } else {
    if (off & 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) widen2(w[j], v[2 * j], v[2 * j + 1]);
  }
  if (!whole) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = use && p + j < last ? load1(p + j) : 0.f;
  }
}

// A warp takes 256 columns of a row, eight neighbours a lane; VEC: rows allow vectors of eight.  Bounded
// by the bytes of dy, the pre-activation and the parts: 3328 x 10000 with tanh or sigmoid in three parts
// takes 62 us (5.3 TB/s), fp32 dy without activation 48 (6.9 TB/s); with one row a thread the former took
// 68, rows that no vector can read 98.
template <bool VEC>
__device__ __forceinline__ void split_rows(const SplitArgs& a, const SplitBlocks::Place& here, float (&warps)[8][256]) {
  constexpr int kSplitRows = VEC ? 2 : 1;  // under way a thread, of dy and the pre-activation both
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = here.column * 256 + 8 * lane;
  const int64_t r0 = static_cast<int64_t>(here.row) * a.rows_per_block;
  const int64_t r1 = min(a.rows, r0 + a.rows_per_block);
  float sum[8] = {};
  // VEC: loads that no conversion waits for before the next are under way.
  auto words = [&](const void* p, int f32, int64_t ld, int64_t r, Raw8<float> (&raw)[kSplitRows]) {
#pragma unroll
    for (int k = 0; k < kSplitRows; ++k) {
      raw[k].zero();
      if (c0 >= a.cols || r + 8 * k >= r1) continue;
      const int64_t at = (r + 8 * k) * ld + c0;
      if (f32)
        raw[k].load(static_cast<const float*>(p) + at);
      else
        raw[k].a = *reinterpret_cast<const float4*>(static_cast<const __nv_bfloat16*>(p) + at);
    }
  };
  auto value = [&](const Raw8<float> (&raw)[kSplitRows], int f32, float (&v)[kSplitRows][8]) {
#pragma unroll
    for (int k = 0; k < kSplitRows; ++k) {
      if (f32) {
        raw[k].get(v[k]);
      } else {
        const float4 w = raw[k].a;
        widen2(__float_as_uint(w.x), v[k][0], v[k][1]);
        widen2(__float_as_uint(w.y), v[k][2], v[k][3]);
        widen2(__float_as_uint(w.z), v[k][4], v[k][5]);
        widen2(__float_as_uint(w.w), v[k][6], v[k][7]);
      }
    }
  };
  auto fetch = [&](const void* p, int f32, int64_t ld, int64_t r, float (&v)[kSplitRows][8]) {
    with_type(p, f32, [&](auto q) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(q)>>;
      const T* const last = q + (a.rows - 1) * ld + a.cols;
#pragma unroll
      for (int k = 0; k < kSplitRows; ++k)
        load8_shifted(q + (r + 8 * k) * ld + c0, q, last, c0 < a.cols && r + 8 * k < r1, v[k]);
    });
  };
  for (int64_t r = r0 + warp; r < r1; r += 8 * kSplitRows) {
    float v[kSplitRows][8], z[kSplitRows][8];
    if constexpr (VEC) {
      Raw8<float> src[kSplitRows], pre[kSplitRows];
      words(a.src, a.src_f32, a.ld_src, r, src);
      if (a.act != DSPARK_ACT_NONE) {
        words(a.pre, a.pre_f32, a.ld_pre, r, pre);
        value(pre, a.pre_f32, z);
      }
      value(src, a.src_f32, v);
    } else {
      fetch(a.src, a.src_f32, a.ld_src, r, v);
      if (a.act != DSPARK_ACT_NONE) fetch(a.pre, a.pre_f32, a.ld_pre, r, z);
    }
    if (a.act != DSPARK_ACT_NONE) {
      with_act(a.act, [&](auto act) {
#pragma unroll
        for (int k = 0; k < kSplitRows; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[k][j] *= act_slope<decltype(act)::value>(z[k][j]);
      });
    }
#pragma unroll
    for (int k = 0; k < kSplitRows; ++k) {
      if (r + 8 * k >= r1 || c0 >= a.cols) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += v[k][j];
      // (an infinity or NaN, or what rounds to an infinity, is its first part alone: not a NaN beside it)
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(v[k][j]) & 0x7FFFFFFFu);
      const bool finite = most < 0x7F7F8000u;
      for (int p = 0; p < 3 && a.part[p] != nullptr; ++p) {
        uint4 h;  // (rows are padded to vectors: what lies beyond the last column is not read)
        uint32_t* const w = reinterpret_cast<uint32_t*>(&h);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = narrow2(v[k][2 * j], v[k][2 * j + 1]);
        *reinterpret_cast<uint4*>(a.part[p] + (r + 8 * k) * a.ld_dst + c0) = h;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          widen2(w[j], lo, hi);
          v[k][2 * j] -= lo;
          v[k][2 * j + 1] -= hi;
        }
        if (!finite) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!isfinite(v[k][j])) v[k][j] = 0.f;
        }
      }
    }
  }
  if (a.sums == nullptr) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) warps[warp][8 * lane + j] = sum[j];
  __syncthreads();
  const int c = here.column * 256 + threadIdx.x;
  if (c < a.cols) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += warps[w][threadIdx.x];
    a.sums[static_cast<int64_t>(here.row) * a.cols + c] = s;
  }
}

// What a call's operands need, in one launch: x, W and dz, each by blocks of its own.  (With as many for each as
// the widest and the tallest need, most of which ended at once, 8192 x 33 x 50257 took 600 to 650 us instead of 370.)
struct SplitJobs {
  SplitArgs job[SplitBlocks::kMost];
  SplitBlocks blocks;
};
__global__ void __launch_bounds__(256, 3) linear_split_kernel(const __grid_constant__ SplitJobs jobs) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float warps[8][256];
  const SplitBlocks::Place here = jobs.blocks.place(blockIdx.x);
  const SplitArgs& a = jobs.job[here.job];
  a.vec ? split_rows<true>(a, here, warps) : split_rows<false>(a, here, warps);
}

// Column sums of the blocks' sums, in a fixed order. A column has `share` threads (1 or 8), each of every
// share-th part: one thread alone took 28 us for the 895 parts of 7164 rows of 128, eight take 7.
__global__ void __launch_bounds__(256) linear_sums_kernel(const float* part, int parts, int cols, int share, float* out) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float sums[256];
  const int width = 256 / share, c = blockIdx.x * width + threadIdx.x % width;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int p = threadIdx.x / width; p < parts; p += share) s += part[static_cast<int64_t>(p) * cols + c];
  }
  sums[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x >= width || c >= cols) return;
  for (int k = 1; k < share; ++k) s += sums[threadIdx.x + k * width];
  out[c] = s;
}

// ------------------------------------------------------------------ host side
// A bf16 matrix as TMA reads it.
struct Matrix {
  const void* p;
  int64_t rows, cols, ld;
};

bool tma_rows(const void* p, int64_t ld) { return rows_of_8(p, ld, DSPARK_BF16); }

class Workspace {
 public:
  explicit Workspace(void* base) : base_(static_cast<uint8_t*>(base)) {}
  bf16* take(int64_t rows, int64_t cols) {
    bf16* const p = reinterpret_cast<bf16*>(base_ + used_);
    used_ += up(rows * up(cols, 8) * 2, 256);
    return p;
  }
  int64_t used() const { return used_; }

 private:
  uint8_t* base_;
  int64_t used_ = 0;
};

struct Launcher {
  const LinearLaunch& c;
  cudaStream_t stream;
  cudaError_t error = cudaSuccess;

  bool first = true;

  bool ok() const { return error == cudaSuccess; }

  // The call's first kernel, or one that starts beside the end of the one before it (each waits for
  // that one's end, and so for all before).
  template <typename... Params, typename... Args>
  void launch(LaunchShape shape, void (*kernel)(Params...), const Args&... args) {
    if (!ok()) return;
    shape.dependent = !first;
    first = false;
    error = launch_kernel(shape, stream, kernel, args...);
    if (ok()) *c.launches += 1;
  }

  // Put down for the next prepare().
  void split(SplitArgs a) {
    const unsigned cols = static_cast<unsigned>((a.cols + 255) / 256);
    // about six blocks an SM; of column sums, as many as the scratch takes
    int64_t per = std::max<int64_t>(8, up((a.rows * cols + 6 * c.num_sms - 1) / (6 * c.num_sms), 8));
    if (a.sums != nullptr) per = std::max(per, (a.rows * a.cols * 4 + kStepScratchBytes / 2 - 1) / (kStepScratchBytes / 2));
    per = std::min(per, up(a.rows, 8));
    a.rows_per_block = static_cast<int>(per);
    a.vec = a.cols % 8 == 0 && rows_of_8(a.src, a.ld_src, a.src_f32 ? DSPARK_F32 : DSPARK_BF16) &&
            (a.act == DSPARK_ACT_NONE || rows_of_8(a.pre, a.ld_pre, a.pre_f32 ? DSPARK_F32 : DSPARK_BF16));
    sum_blocks = static_cast<int>((a.rows + per - 1) / per);
    jobs.job[jobs.blocks.count] = a;
    jobs.blocks.add(cols, static_cast<unsigned>(sum_blocks));
  }
  SplitJobs jobs{};
  int sum_blocks = 0;  // of the last split()

  void prepare() {
    const SplitBlocks& blocks = jobs.blocks;
    if (blocks.count > 0) launch({dim3(blocks.total()), 256}, linear_split_kernel, jobs);
  }

  // The matrix itself, or its copy with rows on 16-byte boundaries.
  Matrix rows_for_tma(const uint16_t* p, int64_t rows, int64_t cols, int64_t ld, Workspace& ws) {
    if (tma_rows(p, ld)) return {p, rows, cols, ld};
    bf16* const to = ws.take(rows, cols);
    SplitArgs a{};
    a.src = p;
    a.rows = rows;
    a.ld_src = ld;
    a.ld_dst = up(cols, 8);
    a.cols = static_cast<int>(cols);
    a.part[0] = to;
    split(a);
    return {to, rows, cols, a.ld_dst};
  }

  template <int BN, bool A_MN, bool B_MN>
  void gemm_sized(GemmArgs& g, GemmEpilogue epi, bool pair) {
    auto run = [&](auto kernel, uint32_t smem, int blocks = 1) {
      const int64_t most = c.num_sms / blocks;
      error = (*c.opt_in)(kernel, smem);
      launch({dim3(static_cast<unsigned>(std::min(g.units, most) * blocks)), kGemmThreads, smem, blocks}, kernel, g);
    };
    if constexpr (BN == 256) {
      if (pair) return run(linear_gemm_kernel<BN, A_MN, B_MN, kEpiTma, true>, GemmShape<BN, kEpiTma, true>::kSmem, 2);
    }
    if (epi == kEpiElements)
      run(linear_gemm_kernel<BN, A_MN, B_MN, kEpiElements>, GemmShape<BN, kEpiElements>::kSmem);
    else if (epi == kEpiTma)
      run(linear_gemm_kernel<BN, A_MN, B_MN, kEpiTma>, GemmShape<BN, kEpiTma>::kSmem);
    if constexpr (!A_MN && B_MN) {  // (the gradients' products have no residual)
      if (epi == kEpiResidual)
        run(linear_gemm_kernel<BN, A_MN, B_MN, kEpiResidual>, GemmShape<BN, kEpiResidual>::kSmem);
      else if (epi == kEpiElementsF32)
        run(linear_gemm_kernel<BN, A_MN, B_MN, kEpiElementsF32>, GemmShape<BN, kEpiElementsF32>::kSmem);
      else if (epi == kEpiElementsBf16)
        run(linear_gemm_kernel<BN, A_MN, B_MN, kEpiElementsBf16>, GemmShape<BN, kEpiElementsBf16>::kSmem);
    }
  }

  // A product as it will be launched.
  struct Plan {
    GemmArgs g{};
    JoinArgs j{};  // of splits
    int BN = 256;
    int64_t S = 1;
    bool pair = false;
    GemmEpilogue epi = kEpiTma;
  };

  static bool tma(const void* p, int64_t ld, int f32) {  // rows that TMA takes
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % (f32 ? 4 : 8) == 0;
  }
  // Rows that TMA stores: it writes whole 16 bytes, zeros into the last ones where a row ends within them.
  static bool tma_out(const void* p, int64_t ld, int f32, int64_t width) {
    return tma(p, ld, f32) && width % (f32 ? 4 : 8) == 0;
  }

  // out = act(A B + bias) + residual, A of parts a[0..na), B of b[0..nb); the epilogue's fields of g
  // are set. splits: this many of them, and two blocks a tile where TMA stores its outputs; 0: as pays.
  template <bool A_MN, bool B_MN>
  Plan plan(GemmArgs g, const Matrix* a, int na, const Matrix* b, int nb, int64_t I, int J, int64_t Kc,
            int64_t splits = 0) {
    Plan p;
    bool by_tma = tma_out(g.out, g.ld_out, g.out_f32, J) && (g.residual == nullptr || tma(g.residual, g.ld_res, g.res_f32)) &&
                  (g.pre == nullptr || (tma(g.pre, g.ld_pre, g.out_f32) && g.residual == nullptr));
    g.blocks_k = (Kc + 63) / 64;
    g.steps = g.blocks_k * std::max(na, nb);
    const int64_t ld_part = up(J, 4);
    // The tile and the number of splits that end soonest by this reckoning (us): a stage's four
    // products take 0.3 at least and as long as its operands need from L2 (0.52 at a width of 256, 0.36
    // where two blocks share a tile), a tile's start 0.5, the last one's outputs 3 by TMA and 10 by
    // elements at a width of 256, the join of splits its launch and its bytes at 4 TB/s.
    // The splits are chosen as if by TMA, so that equal inputs give equal bits wherever they lie.
    double best = 1e30;
    auto consider = [&](int64_t s, double outputs, bool pairs_too) {
      const int64_t per = (g.steps + s - 1) / s;
      if ((g.steps + per - 1) / per != s) return;
      const double join = s > 1 ? 3.0 + static_cast<double>(2 * s * I * ld_part * 4) / 4e6 : 0.0;
      for (int bn : {256, 128, 64}) {
        if (bn != 64 && J <= bn / 2) continue;
        const int64_t tiles = (I + 127) / 128 * ((J + bn - 1) / bn);
        const int64_t waves = (tiles * s + c.num_sms - 1) / c.num_sms;
        const double stage = std::max(0.3, 0.18 + 0.34 * bn / 256);
        const double t = static_cast<double>(waves) * (stage * static_cast<double>(per) + 0.5) + outputs * bn / 256 + join;
        if (t < best) best = t, p.BN = bn, p.S = s, p.pair = false;
      }
      if (pairs_too && I > 128 && J > 128 && g.residual == nullptr) {
        const int64_t tiles = (I + 255) / 256 * ((J + 255) / 256), pairs = c.num_sms / 2;
        const double t = static_cast<double>((tiles * s + pairs - 1) / pairs) * (0.36 * static_cast<double>(per) + 0.5) +
                         outputs + 1.0 + join;
        if (t < best) best = t, p.BN = 256, p.S = s, p.pair = true;
      }
    };
    if (splits > 0) {
      const int64_t per = (g.steps + splits - 1) / splits;
      p.S = (g.steps + per - 1) / per;
      p.pair = true;
    } else {
      for (int64_t s = 1; s <= std::min<int64_t>(g.steps, 64) && (s == 1 || s * I * ld_part * 4 <= kStepScratchBytes); ++s)
        consider(s, 3.0, true);
    }
    if (p.S == 1 && !by_tma) {
      best = 1e30;
      consider(1, 10.0, false);
    }
    g.I = I;
    g.J = J;
    g.tiles_i = p.pair ? (I + 255) / 256 : (I + 127) / 128;
    g.tiles_j = (J + p.BN - 1) / p.BN;
    g.splits = static_cast<int>(p.S);
    g.streams = 1;
    g.per_split = (g.steps + p.S - 1) / p.S;
    g.units = g.tiles_i * g.tiles_j * p.S;
    g.a_parts = na;
    g.b_parts = nb;
    bool maps = true;
    auto encode = [&](CUtensorMap* m, const Matrix& x, uint32_t height) {
      maps = maps && encode_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x.p, x.cols, x.rows, x.ld * 2, 64, height);
    };
    for (int i = 0; i < na; ++i) encode(&g.a[i], a[i], A_MN ? 64 : 128);
    for (int i = 0; i < nb; ++i) encode(&g.b[i], b[i], B_MN ? 64 : p.pair ? p.BN / 2 : p.BN);
    g.status = c.status;
    g.timeout_ns = c.timeout_ns;
    g.skip_cta = c.debug_skip_cta;
    if (p.S > 1) {  // sums of parts first, the epilogue where they are joined
      JoinArgs& j = p.j;
      j.part = c.scratch;
      j.I = I;
      j.ld_part = ld_part;
      j.stride = I * ld_part;
      j.J = J;
      j.splits = static_cast<int>(p.S);
      j.bias = g.bias;
      j.residual = g.residual;
      j.ld_res = g.ld_res;
      j.ld_out = g.ld_out;
      j.ld_pre = g.ld_pre;
      j.res_f32 = g.res_f32;
      j.out_f32 = g.out_f32;
      j.act = g.act;
      j.vec = J % 4 == 0 && tma(g.out, g.ld_out, g.out_f32) && (g.pre == nullptr || tma(g.pre, g.ld_pre, g.out_f32));
      j.out = g.out;
      j.pre = g.pre;
      g.bias = nullptr;
      g.residual = nullptr;
      g.pre = nullptr;
      g.act = DSPARK_ACT_NONE;
      g.out = c.scratch;
      g.out_f32 = 1;
      g.ld_out = ld_part;
      g.split_stride = j.stride;
      by_tma = true;
    }
    if (by_tma) {
      auto encode_out = [&](CUtensorMap* m, const void* to, int64_t ld, int f32, int64_t parts) {
        const uint64_t size = f32 ? 4 : 2;
        maps = maps && encode_3d(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, to, J, I, parts,
                                 ld * size, I * ld * size, f32 ? 32 : 64, 32, 1);
      };
      encode_out(&g.out_map, g.out, g.ld_out, g.out_f32, p.S);
      if (g.pre != nullptr) encode_out(&g.pre_map, g.pre, g.ld_pre, g.out_f32, 1);
      if (g.residual != nullptr)
        maps = maps && encode_2d(&g.res_map, g.res_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                 g.residual, J, I, g.ld_res * (g.res_f32 ? 4 : 2), g.res_f32 ? 32 : 64, 32);
    }
    if (!maps && ok()) error = cudaErrorInvalidValue;
    const bool res = g.residual != nullptr;
    p.epi = by_tma ? (res ? kEpiResidual : kEpiTma) : res ? (g.res_f32 ? kEpiElementsF32 : kEpiElementsBf16) : kEpiElements;
    p.g = g;
    return p;
  }

  template <bool A_MN, bool B_MN>
  void run(Plan p) {
    if (!ok()) return;
    if (p.BN == 256)
      gemm_sized<256, A_MN, B_MN>(p.g, p.epi, p.pair);
    else if (p.BN == 128)
      gemm_sized<128, A_MN, B_MN>(p.g, p.epi, false);
    else
      gemm_sized<64, A_MN, B_MN>(p.g, p.epi, false);
    if (p.S > 1) join(p.j);
  }

  // Both products of a gradient in one launch, where dz passes what L2 keeps between two launches
  // (64 MB of its 129, the other streams taking their share) and dz W^T is of so few tiles that splits
  // of it keep half the blocks busy. Returns whether it did. Sizes and types alone decide, so that equal
  // inputs give equal bits wherever they lie: a dW that TMA does not store gets a launch of its own
  // beside the same splits of dx.
  bool both(const GemmArgs& gx, const GemmArgs& gw, const Matrix* dz, int parts, const Matrix& W, const Matrix& x) {
    const int64_t M = x.rows, K = x.cols, N = dz[0].cols, pairs = c.num_sms / 2;
    const int64_t tiles_x = (M + 255) / 256 * ((K + 255) / 256), units_w = (K + 255) / 256 * ((N + 255) / 256);
    if (M * N * 2 * parts < (64ll << 20) || tiles_x > pairs / 2 || N % (gw.out_f32 ? 4 : 8) != 0) return false;
    const int64_t steps_x = (N + 63) / 64 * parts, steps_w = (M + 63) / 64 * parts;
    // Time until the later of the two is done: a stage of dz W^T takes 0.36 us, one of x^T dz (both of its
    // operands MN-major) 0.45.
    int64_t S = 0, best = INT64_MAX;
    for (int64_t s = 2; s * tiles_x < pairs && s <= steps_x && s * M * up(K, 4) * 4 <= kStepScratchBytes; ++s) {
      const int64_t left = pairs - s * tiles_x;
      const int64_t t = std::max(4 * ((steps_x + s - 1) / s), 5 * ((units_w + left - 1) / left * steps_w));
      if (t < best) best = t, S = s;
    }
    // Two launches, each split by itself, where more than 2 / 7 of the pairs' time would be waiting: 1024 x 23960
    // of 2048 rows with sigmoid (0.76 of it) took 1249 us in one and 638 in two, 256 x 41112 of 2048 (0.06) 95
    // and 117; they meet near 0.3.
    if (S == 0 || 5 * best * pairs > 7 * (4 * tiles_x * steps_x + 5 * units_w * steps_w)) return false;
    Plan px = plan<false, false>(gx, dz, parts, &W, 1, M, static_cast<int>(K), N, S);
    Plan pw = plan<true, true>(gw, &x, 1, dz, parts, K, static_cast<int>(N), M, 1);
    if (!pw.pair) {
      run<false, false>(px);
      run<true, true>(pw);
    }
    if (!ok() || !pw.pair) return true;
    GemmBoth both;
    both.dx = px.g;
    both.dw = pw.g;
    both.dw.streams = static_cast<int>(std::min<int64_t>(px.S, pw.g.tiles_j));
    both.dx_pairs = static_cast<int>(px.g.units);
    // dW passes through L2, which has dz to keep for its second reading (221 us for 2048 x 151936 of 256, 222
    // without, 271 in two launches)
    both.dw.out_first = 1;
    constexpr uint32_t smem = GemmShape<256, kEpiTma, true>::kSmem;
    error = (*c.opt_in)(linear_both_kernel, smem);
    launch({dim3(static_cast<unsigned>(2 * pairs)), kGemmThreads, smem, 2}, linear_both_kernel, both);
    if (px.S > 1) join(px.j);
    return true;
  }

  void join(const JoinArgs& j) {
    if (!ok()) return;
    const int64_t n = j.I * ((j.J + 3) / 4);
    const int64_t blocks = std::min<int64_t>((n + 255) / 256, 8 * c.num_sms);
    launch({dim3(static_cast<unsigned>(blocks)), 256}, linear_join_kernel, j);
  }
};

// Whether dz is the given dy itself, bf16 with rows that TMA reads.
bool dz_as_it_is(const LinearGradArgs& a) {
  return a.act == DSPARK_ACT_NONE && a.dy_dtype == DSPARK_BF16 && tma_rows(a.dy, a.ld_dy);
}
// The bf16 numbers that stand for an element of dz: itself, or three (2^-25 of it lost, less than a rounding to
// fp32).  Two lose 2^-17: far less than a bf16 output's own rounding, but of the odd gate's dx 0.20% of the elements
// then lay a step beside the nearest bf16 number, with three 0.03% (fp32 throughout: 0.02%).  The third costs a bf16
// dx its share of the time: 3885 x 256 x 12880 with sigmoid 216 -> 236 us, 2048 x 1024 x 23960 530 -> 627.
int parts_of(const LinearGradArgs& a) { return a.act == DSPARK_ACT_NONE && a.dy_dtype == DSPARK_BF16 ? 1 : 3; }

}  // namespace

int64_t linear_workspace(const LinearArgs& a) {
  Workspace w(nullptr);
  if (a.M == 0) return 0;
  if (!tma_rows(a.x, a.ld_x)) w.take(a.M, a.K);
  if (!tma_rows(a.W, a.ld_w)) w.take(a.K, a.N);
  return w.used();
}

int64_t linear_grad_workspace(const LinearGradArgs& a) {
  Workspace w(nullptr);
  if (a.M == 0) return 0;
  if (a.dW != nullptr && !tma_rows(a.x, a.ld_x)) w.take(a.M, a.K);
  if (a.dx != nullptr && !tma_rows(a.W, a.ld_w)) w.take(a.K, a.N);
  if ((a.dx != nullptr || a.dW != nullptr) && !dz_as_it_is(a)) {
    for (int p = 0; p < parts_of(a); ++p) w.take(a.M, a.N);
  }
  return w.used();
}

cudaError_t launch_linear(const LinearArgs& a, const LinearLaunch& c, void* workspace, cudaStream_t stream) {
  if (a.M == 0) return cudaSuccess;
  Launcher l{c, stream};
  Workspace ws(workspace);
  const Matrix x = l.rows_for_tma(a.x, a.M, a.K, a.ld_x, ws);
  const Matrix W = l.rows_for_tma(a.W, a.K, a.N, a.ld_w, ws);
  l.prepare();
  GemmArgs g{};
  g.bias = a.bias;
  g.residual = a.residual;
  g.ld_res = a.ld_res;
  g.res_f32 = a.res_dtype == DSPARK_F32;
  g.act = a.act;
  g.out = a.y;
  g.ld_out = a.ld_y;
  g.out_f32 = a.y_dtype == DSPARK_F32;
  g.pre = a.pre;
  g.ld_pre = a.ld_pre;
  l.run<false, true>(l.plan<false, true>(g, &x, 1, &W, 1, a.M, a.N, a.K));
  return l.error;
}

cudaError_t launch_linear_grad(const LinearGradArgs& a, const LinearLaunch& c, void* workspace, cudaStream_t stream) {
  Launcher l{c, stream};
  if (a.M == 0) {  // sums of nothing
    JoinArgs j{};
    j.J = a.N;
    j.I = a.K;
    j.out = a.dW;
    j.ld_out = a.ld_dw;
    j.out_f32 = a.dw_dtype == DSPARK_F32;
    if (a.dW != nullptr) l.join(j);
    j.I = 1;
    j.out = a.dbias;
    j.ld_out = a.N;
    j.out_f32 = 1;
    if (a.dbias != nullptr) l.join(j);
    return l.error;
  }
  Workspace ws(workspace);
  Matrix x{}, W{};
  if (a.dW != nullptr) x = l.rows_for_tma(a.x, a.M, a.K, a.ld_x, ws);
  if (a.dx != nullptr) W = l.rows_for_tma(a.W, a.K, a.N, a.ld_w, ws);
  Matrix dz[3] = {{a.dy, a.M, a.N, a.ld_dy}};
  const bool products = a.dx != nullptr || a.dW != nullptr;
  if (a.dbias != nullptr || (products && !dz_as_it_is(a))) {
    SplitArgs s{};
    s.src = a.dy;
    s.src_f32 = a.dy_dtype == DSPARK_F32;
    s.ld_src = a.ld_dy;
    s.pre = a.pre;
    s.pre_f32 = a.pre_dtype == DSPARK_F32;
    s.ld_pre = a.ld_pre;
    s.act = a.act;
    s.rows = a.M;
    s.cols = a.N;
    s.ld_dst = up(a.N, 8);
    if (products && !dz_as_it_is(a)) {
      for (int p = 0; p < parts_of(a); ++p) {
        s.part[p] = ws.take(a.M, a.N);
        dz[p] = {s.part[p], a.M, a.N, s.ld_dst};
      }
    }
    s.sums = a.dbias != nullptr ? c.scratch : nullptr;
    l.split(s);
  }
  l.prepare();
  if (a.dbias != nullptr) {
    const int share = l.sum_blocks > 16 ? 8 : 1, width = 256 / share;
    l.launch({dim3((a.N + width - 1) / width), 256}, linear_sums_kernel, c.scratch, l.sum_blocks, a.N, share, a.dbias);
  }
  GemmArgs gx{}, gw{};
  gx.out = a.dx;
  gx.ld_out = a.ld_dx;
  gx.out_f32 = a.dx_dtype == DSPARK_F32;
  gw.out = a.dW;
  gw.ld_out = a.ld_dw;
  gw.out_f32 = a.dw_dtype == DSPARK_F32;
  const int parts = parts_of(a);
  if (a.dx != nullptr && a.dW != nullptr && l.both(gx, gw, dz, parts, W, x)) return l.error;
  if (a.dx != nullptr) l.run<false, false>(l.plan<false, false>(gx, dz, parts, &W, 1, a.M, a.K, a.N));
  if (a.dW != nullptr) l.run<true, true>(l.plan<true, true>(gw, &x, 1, dz, parts, a.K, a.N, a.M));
  return l.error;
}

}  // namespace dspark
