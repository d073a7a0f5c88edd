// embed.cu -- rows of an embedding table by token, scaled and converted.
//
// The Markov head reads W1[x_{k-1}] (DSpark explainer, "The Markov head"); in training the same
// rows are gathered for given predecessors. Bytes bound it: 131072 rows of 256 from fp32 to bf16 take 27 us
// (202 MB at 7.4 TB/s, common rows coming from L2), with four vectors under way a thread.

#include <algorithm>

#include "dspark.h"
#include "sm103.cuh"
#include "step.h"
#include "typed.cuh"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // units under way a thread
constexpr int kRound = kThreads * kUnroll;  // units of a block

// A unit is eight elements of a row (one, where rows do not lie on 16-byte boundaries or D is no
// multiple of eight: VEC false).  A block takes `rows` rows, or one of the `pieces` of a row of more
// than kRound units (a row's elements may number 2^31 - 1: no index goes beyond its piece).
template <typename Tin, typename Tout, bool VEC>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedArgs a, int rows, int pieces) {
  const int per_row = VEC ? a.D / 8 : a.D;
  const int64_t row0 = pieces > 1 ? blockIdx.x / pieces : static_cast<int64_t>(blockIdx.x) * rows;
  const int first = pieces > 1 ? static_cast<int>(blockIdx.x % pieces) * kRound : 0;  // unit of the row
  const int width = pieces > 1 ? min(kRound, per_row - first) : per_row;
  const int units = static_cast<int>(min(static_cast<int64_t>(rows), a.N - row0)) * width;
  int row[kUnroll], at[kUnroll], id[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const int u = threadIdx.x + j * kThreads;
    row[j] = u < units ? u / width : -1;
    at[j] = row[j] >= 0 ? (first + u - row[j] * width) * (VEC ? 8 : 1) : 0;
    id[j] = row[j] >= 0 ? __ldg(a.ids + row0 + row[j]) : -1;
    if (id[j] >= a.V) {
      record_error(a.status, kStatusDeviceOob);
      id[j] = -1;
    }
  }
  if constexpr (VEC) {
    Raw8<Tin> raw[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      raw[j].zero();
      if (id[j] >= 0) raw[j].load(static_cast<const Tin*>(a.table) + id[j] * a.ld_table + at[j]);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (row[j] < 0) continue;
      float v[8];
      raw[j].get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= a.scale;
      store8(static_cast<Tout*>(a.out) + (row0 + row[j]) * a.ld_out + at[j], v);
    }
  } else {
    float v[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      v[j] = id[j] >= 0 ? load1(static_cast<const Tin*>(a.table) + id[j] * a.ld_table + at[j])
                        : 0.f;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (row[j] >= 0)
        store1(static_cast<Tout*>(a.out) + (row0 + row[j]) * a.ld_out + at[j], v[j] * a.scale);
  }
}

template <typename Tin, typename Tout>
void embed_typed(const EmbedArgs& a, cudaStream_t stream) {
  const bool vec = a.D % 8 == 0 && rows_of_8(a.table, a.ld_table, a.table_dtype) &&
                   rows_of_8(a.out, a.ld_out, a.out_dtype);
  const int per_row = vec ? a.D / 8 : a.D;
  // one round of units a block (few rows are spread over more blocks)
  const int rows = std::max(1, kRound / per_row);
  const int pieces = static_cast<int>((static_cast<int64_t>(per_row) + kRound - 1) / kRound);
  const int64_t blocks = pieces > 1 ? a.N * pieces : (a.N + rows - 1) / rows;
  if (vec)
    embed_kernel<Tin, Tout, true><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, rows, pieces);
  else
    embed_kernel<Tin, Tout, false><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, rows, pieces);
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs& a, int* launches, cudaStream_t stream) {
  if (a.N == 0) return cudaSuccess;
  if (a.table_dtype == DSPARK_F32)
    a.out_dtype == DSPARK_F32 ? embed_typed<float, float>(a, stream)
                              : embed_typed<float, bf16>(a, stream);
  else
    a.out_dtype == DSPARK_F32 ? embed_typed<bf16, float>(a, stream)
                              : embed_typed<bf16, bf16>(a, stream);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace dspark
