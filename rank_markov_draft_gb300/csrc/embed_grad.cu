// embed_grad.cu -- the gradient of embedding rows by their table: per token, the sum of its rows.
//
// The rows are put in the order of their tokens (equal tokens in the order of the rows), and the
// sorted list is cut into equal pieces, so that a token of a tenth of all rows costs no more than ten
// thousand tokens of one row each; sums of tokens that lie in several pieces are joined in their order.
// No atomics decide an order: equal inputs give equal bits.  The launches:
//   sort: one cluster sorts; beside it zeros are stored to all table rows, by the other clusters of its
//     launch, or, beside a cluster of 8 or 16 (few of which find room at a time: the zeros of 156 MB then
//     took 42 us instead of 25, those of 65 MB 16 instead of 13), by a launch that overlaps it;
//   sums: a group of lanes a piece, a row a group at a time, joined within the block;
//   join: tokens that lie in several blocks.
// 131072 rows of 256 bf16 into 151936 x 256 of fp32: 28 us for the sort, under which the zeros hide, 26 for
// the sums (rows, sums, and the zeros on their way from L2 to DRAM: 5 to 6 TB/s), 4.5 for the join.

#include <algorithm>

#include "async_copy.cuh"
#include "cta_pair.cuh"
#include "dependent.h"
#include "dspark.h"
#include "sm103.cuh"
#include "step.h"
#include "typed.cuh"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ sort
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortMaxCluster = 16, kSortMaxBits = 9, kSortMaxPasses = 3;

struct SortArgs {
  const int32_t* ids;
  int64_t N;
  int V;
  int bits, passes;   // of a pass; their number
  int cluster;        // blocks that sort
  uint32_t* totals;   // [passes][cluster][bins]
  uint2* half;        // [N] after every other pass
  uint2* sorted;      // [N] token (V: padding) and row
  int* status;
  // zeros beside it
  void* grad;         // null: none
  int64_t ld_grad;    // elements
  int D, size;        // of a row, bytes of an element
};

// Rows [0, V) of the gradient set to zero by `blocks` blocks, from the last: the first rows, which
// common tokens have, are stored last and still in L2 when their sums follow.
__device__ __forceinline__ void store_zeros(const SortArgs& a, int block, int blocks) {
  uint8_t* const base = static_cast<uint8_t*>(a.grad);
  const int64_t row_bytes = static_cast<int64_t>(a.D) * a.size, ld = a.ld_grad * a.size;
  const bool packed = a.ld_grad == a.D;
  const int64_t rows = packed ? 1 : a.V, bytes = packed ? row_bytes * a.V : row_bytes;
  const int64_t stride = static_cast<int64_t>(blocks) * kSortThreads, me = static_cast<int64_t>(block) * kSortThreads + threadIdx.x;
  if ((reinterpret_cast<uintptr_t>(base) & 15) == 0 && (packed || (ld & 15) == 0)) {
    const int64_t per_row = bytes / 16;
    if (packed) {
#pragma unroll 4
      for (int64_t u = per_row - 1 - me; u >= 0; u -= stride)
        reinterpret_cast<uint4*>(base)[u] = make_uint4(0, 0, 0, 0);
    } else {
      for (int64_t u = me; u < rows * per_row; u += stride) {
        const int64_t r = u / per_row;
        reinterpret_cast<uint4*>(base + (rows - 1 - r) * ld)[u - r * per_row] = make_uint4(0, 0, 0, 0);
      }
    }
    const int tail = static_cast<int>(bytes - per_row * 16) / a.size;  // elements behind the vectors
    for (int64_t u = me; u < rows * tail; u += stride) {
      uint8_t* const p = base + (u / tail) * ld + per_row * 16 + (u % tail) * a.size;
      if (a.size == 4)
        *reinterpret_cast<uint32_t*>(p) = 0;
      else
        *reinterpret_cast<uint16_t*>(p) = 0;
    }
  } else {
    const int64_t n = bytes / a.size;
    for (int64_t u = me; u < rows * n; u += stride) {
      uint8_t* const p = base + (u / n) * ld + (u % n) * a.size;
      if (a.size == 4)
        *reinterpret_cast<uint32_t*>(p) = 0;
      else
        *reinterpret_cast<uint16_t*>(p) = 0;
    }
  }
}

// Stable counting sort by `bits` bits of the token a pass, over one cluster: each warp counts the
// digits of its stretch of the list, the counts of all blocks give each warp's first place of every
// digit, and the warps place their elements. Elements are taken 32 at a time, and each finds the lanes
// of its digit: for the low digits by an OR of their bits into a word of shared memory (4400 clocks for
// 8192 elements), for the high ones, which text has mostly alike, by a vote a bit (8700 clocks, where
// the ORs would take 9400; the match instruction took as long for either).
// Where a warp's stretch fits its registers (131072 entries in 16 blocks) the places found while
// counting are kept, and the low digits' elements are put in order within the block first, so that
// their stores go to runs of some 16 of them (4 clocks an element otherwise, a sector each).
constexpr int kSortHeld = 8;  // elements of a lane in registers

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(SortArgs a) {
  extern __shared__ uint32_t counts[];  // [warps][bins], 2 [bins], lanes or elements
  __shared__ uint32_t warp_sum[kSortWarps], warp_local[kSortWarps];
  griddep_launch_dependents();
  const int c = blockIdx.x;
  if (c >= a.cluster) {
    store_zeros(a, c - a.cluster, gridDim.x - a.cluster);
    return;
  }
  const int bins = 1 << a.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* const mine = counts + warp * bins;
  uint32_t* const base = counts + kSortWarps * bins;
  uint32_t* const local = base + bins;  // the block's elements of lower digits
  uint32_t* const lanes = local + bins + warp * bins;
  uint2* const staged = reinterpret_cast<uint2*>(local + bins);
  const int64_t stretch = (a.N + static_cast<int64_t>(a.cluster) * kSortThreads - 1) /
                          (static_cast<int64_t>(a.cluster) * kSortThreads) * 32;  // a warp's
  const int64_t lo = min(a.N, (static_cast<int64_t>(c) * kSortWarps + warp) * stretch);
  const int64_t hi = min(a.N, lo + stretch);
  const bool held = stretch <= 32 * kSortHeld;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const bool spread = pass + 1 < a.passes;
    const bool last_is_odd = (a.passes - pass) & 1;
    uint2* const dst = last_is_odd ? a.sorted : a.half;
    const uint2* const src = last_is_odd ? a.half : a.sorted;
    uint2 e[kSortHeld];
    uint32_t place[kSortHeld];  // among the warp's elements of its digit
    auto digit_of = [&](const uint2& x) { return (x.x >> shift) & (bins - 1); };
    // elements [i0, i0 + 32 kSortHeld) of the stretch (beyond it: none)
    auto fetch = [&](int64_t i0) {
#pragma unroll
      for (int j = 0; j < kSortHeld; ++j) {
        const int64_t i = i0 + 32 * j + lane;
        e[j] = make_uint2(0xFFFFFFFFu, static_cast<uint32_t>(i));
        if (i < hi) {
          if (pass > 0)
            e[j] = __ldcg(src + i);
          else
            e[j].x = static_cast<uint32_t>(a.ids[i]);
        }
      }
      if (pass > 0) return;
      bool bad = false;
#pragma unroll
      for (int j = 0; j < kSortHeld; ++j) {
        const bool in = i0 + 32 * j + lane < hi;
        const int32_t id = static_cast<int32_t>(e[j].x);
        bad |= in && id >= a.V;
        e[j].x = !in ? 0xFFFFFFFFu : static_cast<uint32_t>(id < 0 || id >= a.V ? a.V : id);
      }
      if (bad) record_error(a.status, kStatusDeviceOob);
    };
    // counts them on
    auto count = [&](int64_t i0) {
#pragma unroll
      for (int j = 0; j < kSortHeld; ++j) {
        if (i0 + 32 * j >= hi) break;
        const bool in = e[j].x != 0xFFFFFFFFu;
        const uint32_t digit = digit_of(e[j]);
        unsigned same = 0;
        if (spread) {
          if (in) atomicOr(lanes + digit, 1u << lane);
          __syncwarp();
          same = in ? lanes[digit] : 0;
        } else {
          same = __ballot_sync(0xFFFFFFFFu, in);
#pragma unroll
          for (int bit = 0; bit < kSortMaxBits; ++bit) {
            const bool one = digit & (1u << bit);
            const unsigned set = __ballot_sync(0xFFFFFFFFu, one);
            same &= one ? set : ~set;
          }
        }
        const uint32_t at = in ? mine[digit] : 0;
        place[j] = at + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (in && (same >> lane) == 1) {  // the last of them
          mine[digit] = at + __popc(same);
          if (spread) lanes[digit] = 0;
        }
        __syncwarp();
      }
    };
    auto put = [&](bool with_warp) {
#pragma unroll
      for (int j = 0; j < kSortHeld; ++j)
        if (e[j].x != 0xFFFFFFFFu) {
          const uint32_t d = digit_of(e[j]);
          dst[base[d] + place[j] + (with_warp ? mine[d] : 0)] = e[j];
        }
    };
    fetch(lo);
    for (int i = threadIdx.x; i < kSortWarps * bins / 4; i += kSortThreads) {
      reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
      if (spread) reinterpret_cast<uint4*>(staged)[i] = make_uint4(0, 0, 0, 0);  // (the words of `lanes`)
    }
    __syncthreads();
    count(lo);
    for (int64_t i0 = lo + 32 * kSortHeld; i0 < hi; i0 += 32 * kSortHeld) {
      fetch(i0);
      count(i0);
    }
    __syncthreads();
    uint32_t* const totals = a.totals + static_cast<int64_t>(pass) * a.cluster * bins;
    uint32_t here = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = counts[w * bins + threadIdx.x];
        counts[w * bins + threadIdx.x] = here;
        here += n;
      }
      totals[c * bins + threadIdx.x] = here;
    }
    cluster_sync();
    uint32_t below = 0, all = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (int k = 0; k < kSortMaxCluster; ++k) {
        const uint32_t n = k < a.cluster ? __ldcg(totals + k * bins + threadIdx.x) : 0;
        below += k < c ? n : 0;
        all += n;
      }
    }
    uint32_t incl = all, incl_here = here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, incl, o), m = __shfl_up_sync(0xFFFFFFFFu, incl_here, o);
      incl += lane >= o ? n : 0;
      incl_here += lane >= o ? m : 0;
    }
    if (lane == 31) warp_sum[warp] = incl, warp_local[warp] = incl_here;
    __syncthreads();
    uint32_t before = lane < warp ? warp_sum[lane] : 0, before_here = lane < warp ? warp_local[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
      before_here += __shfl_xor_sync(0xFFFFFFFFu, before_here, o);
    }
    if (threadIdx.x < bins) {
      base[threadIdx.x] = before + incl - all + below;
      local[threadIdx.x] = before_here + incl_here - here;
    }
    __syncthreads();
    if (held && spread) {
#pragma unroll
      for (int j = 0; j < kSortHeld; ++j)
        if (e[j].x != 0xFFFFFFFFu) {
          const uint32_t d = digit_of(e[j]);
          staged[local[d] + mine[d] + place[j]] = e[j];
        }
      __syncthreads();
      const int n = static_cast<int>(min(a.N, (c + 1) * kSortWarps * stretch) - min(a.N, c * kSortWarps * stretch));
#pragma unroll 4
      for (int i = threadIdx.x; i < n; i += kSortThreads) {
        const uint2 x = staged[i];
        const uint32_t d = digit_of(x);
        dst[base[d] + i - local[d]] = x;
      }
    } else if (held) {
      put(true);
    } else {  // `mine` goes on as a running count
      for (int64_t i0 = lo; i0 < hi; i0 += 32 * kSortHeld) {
        fetch(i0);
        count(i0);
        put(false);
      }
    }
    if (pass + 1 < a.passes) cluster_sync();
  }
}

// The zeros as a launch of their own, which ends after the sort that it overlaps.
__global__ void __launch_bounds__(kSortThreads) embed_zeros_kernel(SortArgs a) {
  griddep_launch_dependents();
  store_zeros(a, blockIdx.x, gridDim.x);
  if (blockIdx.x + 1 == gridDim.x) griddep_wait();  // (all of them would hold their SMs meanwhile)
}

// ------------------------------------------------------------------ sums
constexpr int kSumThreads = 512, kSumBlocks = 2;  // of an SM
// Rows under way a group, by asynchronous copies (VEC; 64 KB of shared memory a block): registers
// would hold as many, but the few counters a warp waits on make it wait for later loads too.
template <typename T>
constexpr int kSumAhead = sizeof(T) == 2 ? 8 : 4;
constexpr int kSumBatch = 2;  // otherwise, in registers

struct SumArgs {
  const uint2* sorted;
  const void* de;
  int64_t N, ld_de, ld_grad;
  int V, D;
  int lanes;        // of a group (8, 16 or 32): 8 columns each
  int piece;        // list entries of a group
  float scale;
  bool accumulate;
  void* grad;
  float *head, *tail;  // [slices][blocks][8 lanes]: sums of the tokens that reach in from the block
                       // before, and out to the next
};

// The eight columns of a lane: neighbours (VEC) or `lanes` apart.
template <typename T, bool VEC>
struct Columns {
  Raw8<T> raw;
  float one[VEC ? 1 : 8];
  __device__ __forceinline__ void load(const T* row, int col, int lanes, int D) {
    if constexpr (VEC) {
      raw.load(row + col);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) one[j] = col + j * lanes < D ? load1(row + col + j * lanes) : 0.f;
    }
  }
  __device__ __forceinline__ void add_to(float (&s)[8]) const {
    if constexpr (VEC) {
      float v[8];
      raw.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += v[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += one[j];
    }
  }
};

template <typename T, bool VEC>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t token, int col, const float (&s)[8]) {
  if (col >= a.D) return;
  T* const row = static_cast<T*>(a.grad) + static_cast<int64_t>(token) * a.ld_grad;
  float v[8] = {};
  if (a.accumulate) {
    Columns<T, VEC> old;
    old.load(row, col, a.lanes, a.D);
    old.add_to(v);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fmaf(a.scale, s[j], v[j]);
  if constexpr (VEC) {
    store8(row + col, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j * a.lanes < a.D) store1(row + col + j * a.lanes, v[j]);
  }
}

__device__ __forceinline__ int first_column(int slice, int lane, int lanes, bool vec) {
  return slice * lanes * 8 + (vec ? lane * 8 : lane);
}

// A piece's runs of equal tokens that begin and end in it are done where they end.  `head` is the sum
// of a run that reaches in from the piece before, `tail` of one that begins here and reaches out;
// `through` says that the head reaches out too.
template <typename Tin, typename Tout, bool VEC>
__global__ void __launch_bounds__(kSumThreads, kSumBlocks) embed_sum_kernel(SumArgs a) {
  __shared__ float heads[kSumThreads * 8], tails[kSumThreads * 8];
  __shared__ uint32_t tokens[kSumThreads];
  __shared__ uint8_t has_head[kSumThreads], has_tail[kSumThreads], through[kSumThreads];
  constexpr int kHalves = sizeof(Tin) / 2;  // 16-byte copies of a lane's columns
  __shared__ uint4 ring[VEC ? kSumAhead<Tin> * kHalves * kSumThreads : 1];
  auto slot = [&](int j, int h) { return ring + (j * kHalves + h) * kSumThreads + threadIdx.x; };
  const int group = threadIdx.x / a.lanes, lane = threadIdx.x % a.lanes, groups = kSumThreads / a.lanes;
  const int col = first_column(blockIdx.y, lane, a.lanes, VEC);
  const int64_t begin = min(a.N, (static_cast<int64_t>(blockIdx.x) * groups + group) * a.piece);
  const int64_t end = min(a.N, begin + a.piece);
  const uint32_t none = static_cast<uint32_t>(a.V);
  if (lane == 0) has_head[group] = has_tail[group] = through[group] = 0;
  griddep_wait();
  float s[8] = {};
  auto deposit = [&](float* where) {
#pragma unroll
    for (int j = 0; j < 8; ++j) where[j * kSumThreads + threadIdx.x] = s[j];
  };
  // (entries of the warp's first group, the longest: its groups go on together)
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * groups + (threadIdx.x & ~31) / a.lanes) * a.piece;
  const int64_t longest = min(static_cast<int64_t>(a.piece), a.N - first);
  if (longest > 0) {
    uint32_t token = begin < end ? a.sorted[begin].x : none;
    bool reaches_in = begin > 0 && begin < end && a.sorted[begin - 1].x == token;
    auto entry = [&](int64_t i) { return i < end ? a.sorted[i] : make_uint2(none, 0); };
    // the next row's token: what has been summed for another is done
    auto turn_to = [&](uint32_t next) {
      if (next == token) return;
      if (reaches_in) {
        deposit(heads);
        if (lane == 0) has_head[group] = 1;
      } else {
        write_row<Tout, VEC>(a, token, col, s);
      }
      reaches_in = false;
      token = next;
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] = 0.f;
    };
    if constexpr (VEC) {
      // entries arrive a window of a group's lanes at a time, an entry a lane
      constexpr int kAhead = kSumAhead<Tin>;
      uint2 now = entry(begin + lane), after = entry(begin + a.lanes + lane);
      auto fetch = [&](int j, const uint2& w, int at) {  // the row of a window's entry
        const uint32_t token_at = __shfl_sync(0xFFFFFFFFu, w.x, at, a.lanes);
        const uint32_t n = __shfl_sync(0xFFFFFFFFu, w.y, at, a.lanes);
        if (token_at != none && col < a.D) {
          const Tin* const row = static_cast<const Tin*>(a.de) + n * a.ld_de + col;
#pragma unroll
          for (int h = 0; h < kHalves; ++h) cp_async_16(slot(j, h), row + h * 4);
        }
        cp_async_commit();
      };
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(j, now, j);
      for (int64_t i = 0; i < longest; i += a.lanes) {
        for (int at = 0; at < a.lanes && i + at < longest; at += kAhead) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const uint32_t t = __shfl_sync(0xFFFFFFFFu, now.x, at + j, a.lanes);
            cp_async_wait_group<kAhead - 1>();
            if (t != none) {
              turn_to(t);
              if (col < a.D) {
                Columns<Tin, VEC> row;
                row.raw.load_halves(slot(j, 0), slot(j, kHalves - 1));
                row.add_to(s);
              }
            }
            if (at + kAhead < a.lanes)
              fetch(j, now, at + kAhead + j);
            else
              fetch(j, after, j);
          }
        }
        now = after;
        after = entry(begin + i + 2 * a.lanes + lane);
      }
    } else {
      for (int64_t i = begin; i < end; i += kSumBatch) {
        Columns<Tin, VEC> rows[kSumBatch];
        uint2 e[kSumBatch];
#pragma unroll
        for (int j = 0; j < kSumBatch; ++j) {
          e[j] = entry(i + j);
          if (e[j].x != none && col < a.D)
            rows[j].load(static_cast<const Tin*>(a.de) + e[j].y * a.ld_de, col, a.lanes, a.D);
        }
#pragma unroll
        for (int j = 0; j < kSumBatch; ++j) {
          if (e[j].x == none) continue;
          turn_to(e[j].x);
          if (col < a.D) rows[j].add_to(s);
        }
      }
    }
    if (token != none) {
      const bool reaches_out = end < a.N && a.sorted[end].x == token;
      if (reaches_in) {
        deposit(heads);
        if (lane == 0) has_head[group] = 1, through[group] = reaches_out;
      } else if (reaches_out) {
        deposit(tails);
        if (lane == 0) has_tail[group] = 1, tokens[group] = token;
      } else {
        write_row<Tout, VEC>(a, token, col, s);
      }
    }
  }
  __syncthreads();
  auto add_head = [&](int g) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += heads[j * kSumThreads + g * a.lanes + lane];
  };
  auto keep = [&](float* where) {
    float* const p = where + ((static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * a.lanes + lane) * 8;
    store8(p, s);
  };
  if (group == 0 && has_head[0]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.f;
    add_head(0);
    int g = 0;
    while (through[g] && g + 1 < groups) add_head(++g);
    keep(a.head);
  }
  if (has_tail[group]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = tails[j * kSumThreads + threadIdx.x];
    int g = group;
    bool out = true;
    while (out && g + 1 < groups) {
      add_head(++g);
      out = through[g];
    }
    if (out)
      keep(a.tail);
    else
      write_row<Tout, VEC>(a, tokens[group], col, s);
  }
}

// Runs over several blocks: a group for each block that one begins in.
template <typename Tout, bool VEC>
__global__ void __launch_bounds__(kSumThreads) embed_join_kernel(SumArgs a, int blocks) {
  griddep_wait();
  const int group = threadIdx.x / a.lanes, lane = threadIdx.x % a.lanes, groups = kSumThreads / a.lanes;
  const int64_t per_block = static_cast<int64_t>(a.piece) * groups;
  const int b = blockIdx.x * groups + group;
  if (b + 1 >= blocks) return;
  auto token_at = [&](int64_t i) { return a.sorted[i].x; };
  const int64_t begin = b * per_block, end = begin + per_block;  // (a later block is not empty)
  const uint32_t token = token_at(end - 1);
  if (token == static_cast<uint32_t>(a.V) || token_at(end) != token) return;
  if (begin > 0 && token_at(begin - 1) == token) return;  // begins in an earlier block
  float s[8];
  auto at = [&](const float* p, int block) {
    return p + ((static_cast<int64_t>(blockIdx.y) * blocks + block) * a.lanes + lane) * 8;
  };
  Raw8<float> first;
  first.load(at(a.tail, b));
  first.get(s);
  constexpr int kAhead = 8;
  bool on = true;  // the run reaches into block k
  for (int k0 = b + 1; k0 < blocks && on; k0 += kAhead) {
    Raw8<float> r[kAhead];
    bool out[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j;
      const int64_t next = (k + 1) * per_block;
      out[j] = k < blocks && next < a.N && token_at(next) == token;
      r[j].zero();
      if (k < blocks) r[j].load(at(a.head, k));  // (of a block without a head: unused)
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (on) {
        float v[8];
        r[j].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += v[i];
      }
      on = on && out[j];
    }
  }
  write_row<Tout, VEC>(a, token, first_column(blockIdx.y, lane, a.lanes, VEC), s);
}

template <typename Tin, typename Tout, bool VEC>
cudaError_t sums(const SumArgs& s, int blocks, int slices, int* launches, cudaStream_t stream) {
  cudaError_t e = launch_kernel({dim3(blocks, slices), kSumThreads}, stream, embed_sum_kernel<Tin, Tout, VEC>, s);
  if (e != cudaSuccess) return e;
  *launches += 1;
  if (blocks == 1) return e;
  const int groups = kSumThreads / s.lanes;
  e = launch_kernel({dim3((blocks + groups - 1) / groups, slices), kSumThreads}, stream,
                    embed_join_kernel<Tout, VEC>, s, blocks);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

}  // namespace

cudaError_t launch_embed_grad(const EmbedGradArgs& a, const EmbedGradLaunch& c, cudaStream_t stream) {
  if (a.N == 0 && a.accumulate) return cudaSuccess;
  // the scratch: digit counts, the list after each pass, partial sums
  uint8_t* p = c.scratch;
  SortArgs t{};
  t.totals = reinterpret_cast<uint32_t*>(p);
  p += (kSortMaxPasses * kSortMaxCluster * 4) << kSortMaxBits;
  t.half = reinterpret_cast<uint2*>(p);
  p += kEmbedGradMaxRows * 8;
  t.sorted = reinterpret_cast<uint2*>(p);
  p += kEmbedGradMaxRows * 8;
  t.ids = a.ids;
  t.N = a.N;
  t.V = a.V;
  t.status = a.status;
  int bits = 1;
  while ((a.V >> bits) != 0) ++bits;  // tokens 0 .. V
  t.passes = (bits + kSortMaxBits - 1) / kSortMaxBits;
  t.bits = std::max(5, (bits + t.passes - 1) / t.passes);
  // 2048 entries a block: below that another block costs more than its share saves
  t.cluster = 1;
  while (t.cluster < kSortMaxCluster && a.N > 2048 * static_cast<int64_t>(t.cluster)) t.cluster *= 2;
  int grid = t.cluster;
  if (!a.accumulate) {
    t.grad = a.grad;
    t.ld_grad = a.ld_grad;
    t.D = a.D;
    t.size = a.grad_dtype == DSPARK_F32 ? 4 : 2;
    if (t.cluster <= 4) grid = c.num_sms / t.cluster * t.cluster;
  }
  // counts, two words a digit, and the larger of the lanes' words and the elements in order
  auto sort_smem = [](int bits) { return ((kSortWarps + 2) << bits) * 4 + std::max((kSortWarps << bits) * 4, kSortThreads * kSortHeld * 8); };
  const int smem = sort_smem(t.bits);
  cudaError_t e = (*c.opt_in)(embed_sort_kernel, sort_smem(kSortMaxBits));
  if (e != cudaSuccess) return e;
  if (t.cluster > 8) {
    e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  e = launch_kernel({dim3(grid), kSortThreads, static_cast<size_t>(smem), t.cluster, false}, stream, embed_sort_kernel, t);
  if (e != cudaSuccess) return e;
  *c.launches += 1;
  if (!a.accumulate && t.cluster > 4) {
    // (64 KB a block: the SMs that sort leave theirs to the others)
    const int64_t chunks = static_cast<int64_t>(a.V) * a.D * t.size / 65536;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(std::max<int64_t>(chunks, 1), 8192));
    e = launch_kernel({dim3(blocks), kSortThreads}, stream, embed_zeros_kernel, t);
    if (e != cudaSuccess) return e;
    *c.launches += 1;
  }
  if (a.N == 0) return e;

  SumArgs s{};
  s.sorted = t.sorted;
  s.de = a.de;
  s.N = a.N;
  s.ld_de = a.ld_de;
  s.ld_grad = a.ld_grad;
  s.V = a.V;
  s.D = a.D;
  s.scale = a.scale;
  s.accumulate = a.accumulate;
  s.grad = a.grad;
  const bool vec = a.D % 8 == 0 && rows_of_8(a.de, a.ld_de, a.de_dtype) && rows_of_8(a.grad, a.ld_grad, a.grad_dtype);
  s.lanes = 32;
  while (vec && s.lanes > 8 && s.lanes * 4 >= a.D) s.lanes /= 2;
  const int slices = (a.D + s.lanes * 8 - 1) / (s.lanes * 8), groups = kSumThreads / s.lanes;
  // one wave of blocks over list and columns
  const int64_t most = kSumBlocks * c.num_sms * groups;
  s.piece = static_cast<int>(std::max<int64_t>(8, (a.N * slices + most - 1) / most));
  if (s.piece > s.lanes / 2) s.piece = (s.piece + s.lanes - 1) / s.lanes * s.lanes;  // whole windows
  const int blocks = static_cast<int>((a.N + static_cast<int64_t>(s.piece) * groups - 1) / (static_cast<int64_t>(s.piece) * groups));
  s.head = reinterpret_cast<float*>(p);
  s.tail = s.head + static_cast<int64_t>(blocks) * slices * s.lanes * 8;
  auto run = [&](auto in, auto out) {
    using Tin = decltype(in);
    using Tout = decltype(out);
    return vec ? sums<Tin, Tout, true>(s, blocks, slices, c.launches, stream)
               : sums<Tin, Tout, false>(s, blocks, slices, c.launches, stream);
  };
  if (a.de_dtype == DSPARK_F32)
    return a.grad_dtype == DSPARK_F32 ? run(float(), float()) : run(float(), bf16());
  return a.grad_dtype == DSPARK_F32 ? run(bf16(), float()) : run(bf16(), bf16());
}

}  // namespace dspark
