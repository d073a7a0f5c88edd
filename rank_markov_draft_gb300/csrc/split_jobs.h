// split_jobs.h -- up to three matrices of different shapes worked on by one launch: each has its own blocks,
// one after another, so that none is launched for what another's shape alone would need.
#pragma once

#include <cuda_runtime.h>

namespace dspark {

struct SplitBlocks {
  static constexpr int kMost = 3;
  int count = 0;
  unsigned first[kMost + 1] = {};  // blocks before each matrix, and of all
  unsigned wide[kMost] = {};       // blocks across its columns

  // The next matrix: its blocks across the columns, and down the rows.
  void add(unsigned columns, unsigned rows) {
    wide[count] = columns;
    first[count + 1] = first[count] + columns * rows;
    ++count;
  }
  unsigned total() const { return first[count]; }

  // The matrix of a block, and its place there.
  struct Place {
    int job;
    unsigned column, row;
  };
  __host__ __device__ Place place(unsigned block) const {
    int job = 0;
    while (job + 1 < count && block >= first[job + 1]) ++job;
    const unsigned n = block - first[job];
    return {job, n % wide[job], n / wide[job]};
  }
};

}  // namespace dspark
