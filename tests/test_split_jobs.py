"""How the blocks of one launch are shared out among matrices of different shapes (csrc/split_jobs.h), on the CPU."""

import os
import subprocess

from rank_markov_draft_gb300 import build

PROGRAM = r"""
#include "split_jobs.h"
#include <cstdio>
#include <set>
#include <tuple>

using dspark::SplitBlocks;

// Every block has a place of its own, and there are as many as the matrices have.
static bool right(std::initializer_list<std::pair<unsigned, unsigned>> shapes) {
  SplitBlocks b;
  unsigned n = 0;
  for (auto [columns, rows] : shapes) b.add(columns, rows), n += columns * rows;
  if (b.total() != n || b.count != static_cast<int>(shapes.size())) return false;
  std::set<std::tuple<int, unsigned, unsigned>> places;
  for (unsigned k = 0; k < n; ++k) {
    const SplitBlocks::Place p = b.place(k);
    if (p.job < 0 || p.job >= b.count) return false;
    const auto shape = shapes.begin()[p.job];
    if (p.column >= shape.first || p.row >= shape.second) return false;
    places.insert({p.job, p.column, p.row});
  }
  return places.size() == n;
}

int main() {
  // a tall matrix of few columns beside two wide ones of few rows: 512 + 985 + 985 blocks, not 3 * 197 * 512
  bool ok = right({{1, 512}, {197, 5}, {197, 5}});
  ok = ok && right({{1, 1}}) && right({{1, 1}, {1, 1}, {1, 1}}) && right({{7, 3}, {1, 40}}) && right({{300, 1}, {2, 2}, {1, 65535}});
  std::puts(ok ? "ok" : "wrong");
  return ok ? 0 : 1;
}
"""


def test_each_matrix_has_its_own_blocks_and_no_more(tmp_path):
    src, exe = tmp_path / "jobs.cpp", tmp_path / "jobs"
    src.write_text(PROGRAM)
    toolkit = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", os.path.join(toolkit, "include"), str(src), "-o", str(exe)],
                   check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"


def test_the_linear_layers_launch_no_others():
    with open(os.path.join(build.CSRC, "linear.cu")) as f:
        source = f.read()
    assert "launch({dim3(blocks.total()), 256}, linear_split_kernel" in source
