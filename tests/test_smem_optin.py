"""The opt-in of kernels to more shared memory belongs to a kernel on one device: the launchers'
record of it (csrc/smem_optin.h), run on the CPU against a stand-in of the runtime's call."""

import os
import re
import subprocess

from rank_markov_draft_gb300 import build

PROGRAM = r"""
#include "smem_optin.h"
#include <cstdio>

static int device = 0, calls = 0;
static bool refuse = false, opted[2][2];
void first(int) {}
void second(int) {}

extern "C" cudaError_t cudaFuncSetAttribute(const void* fn, cudaFuncAttribute attr, int bytes) {
  ++calls;
  if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize || bytes != 50000) return cudaErrorInvalidValue;
  if (refuse) return cudaErrorMemoryAllocation;
  opted[device][fn == reinterpret_cast<const void*>(&first) ? 0 : 1] = true;
  return cudaSuccess;
}

int main() {
  dspark::SmemOptIn contexts[2];  // one on each device
  refuse = true;
  const bool failed = contexts[0](first, 50000) != cudaSuccess;
  refuse = false;
  bool ok = failed && contexts[0](first, 50000) == cudaSuccess && opted[0][0] && calls == 2;
  ok = ok && contexts[0](first, 50000) == cudaSuccess && calls == 2;  // once
  ok = ok && contexts[0](second, 50000) == cudaSuccess && opted[0][1] && calls == 3;
  device = 1;
  for (auto fn : {first, second}) ok = ok && contexts[1](fn, 50000) == cudaSuccess;
  ok = ok && opted[1][0] && opted[1][1] && calls == 5;
  std::puts(ok ? "ok" : "wrong");
  return ok ? 0 : 1;
}
"""


def test_each_context_opts_in_for_its_own_device_and_a_failure_is_not_kept(tmp_path):
    src, exe = tmp_path / "optin.cpp", tmp_path / "optin"
    src.write_text(PROGRAM)
    toolkit = os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc())))
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", os.path.join(toolkit, "include"), str(src), "-o", str(exe)],
                   check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"


def test_no_launcher_keeps_an_answer_of_the_runtime_for_the_process():
    for name in sorted(os.listdir(build.CSRC)):
        with open(os.path.join(build.CSRC, name)) as f:
            assert not re.search(r"static\s+(const\s+)?cudaError_t\s+\w+(\[\w*\])?\s*=", f.read()), name
