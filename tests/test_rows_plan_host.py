"""Host-side invariants of the row losses' launch plans (lik_rows_kernels.h), on
the CPU: a small C++ program includes the header and checks the LDS that the
distillation kernels are launched with and allowed.

What a kernel is allowed is one attribute for all host threads, so it must not
depend on the call: the most of any call, within a CU's LDS beside what the kernel
declares itself (at most 256 bytes)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "maxsim_scoring_02_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

PROGRAM = r"""
#include <cstdio>
#include "lik_rows_kernels.h"
using namespace lik;

int main() {
  int fails = 0;
  const int kernels[][2] = {{64, 0}, {256, 0}, {512, 0}, {1024, 0}, {1024, 9}};
  for (auto& k : kernels) {
    const int threads = k[0], held = k[1];
    const size_t most = distill_lds_most(threads, held);
    const int64_t longest = held ? kDistillLdsK : kDistillMaxK;
    size_t before = 0;
    bool reached = false;
    for (int64_t K = 0; K <= longest; ++K) {
      const size_t lds = distill_lds(K, threads, held);
      const size_t lists = threads == 64 ? 4 : 1;
      // four words an entry, the flags and a word a thread have to fit
      if (lds > most || lds < before || lds % 16 ||
          lds < (size_t)held * threads * 16 + lists * (16 * K + 4 + 4 * threads)) ++fails;
      before = lds;
      reached |= lds == most;
    }
    if (!reached || most > 160 * 1024 - 256) ++fails;
    std::printf("%d threads, %d pieces: %zu\n", threads, held, most);
  }
  // which lists go to which kernels: long ones beside rows in LDS are not held
  if (kRegisterBytes != 16 * 1024 * 16 || kHeldBytes <= kRegisterBytes) ++fails;
  std::printf("fails %d\n", fails);
  return fails != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include", "hip")),
                    reason="needs a host C++ compiler and the HIP headers")
def test_lds_of_the_distillation_kernels(tmp_path):
    src, exe = tmp_path / "lds_check.cpp", tmp_path / "lds_check"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", CSRC, "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROCM, "include"), str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "fails 0" in r.stdout, r.stdout + r.stderr
