"""The plan of the FP8 product (csrc/fp8_plan.hpp, host arithmetic) compiled with the host
compiler and swept over shapes: every launch it leads to has work."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "group_wise_bit_amd", "csrc")
CXX = shutil.which("g++") or shutil.which("c++")

SWEEP = r"""
#include <cstdio>
#include "fp8_plan.hpp"
using namespace gwb;
static int bad = 0;
static long split = 0;
static void check(int64_t M, int64_t N, int64_t K, bool exact) {
  const GemmPlan p = fp8_gemm_plan(M, N, K, exact);
  bool ok = p.splits >= 1 && p.splits <= (K + 127) / 128 && p.threads > 0 && p.wide > 0 && p.wide <= N;
  if (p.kernel != kTile256) ok = ok && p.wide == N;
  else if (p.wide < N) {
    ++split;                                             // whole tile columns stay
    ok = ok && p.wide % 256 == 0;
  }
  if (!ok && bad++ < 10)
    printf("M=%ld N=%ld K=%ld exact=%d: kernel %d splits %d wide %ld\n", (long)M, (long)N, (long)K, exact, p.kernel, p.splits, (long)p.wide);
}
int main() {
  const int64_t Ns[] = {1, 16, 127, 128, 129, 200, 255, 256, 257, 384, 512, 513, 768, 1024, 1280, 2048, 3840, 5120, 8191, 34816};
  for (int64_t N : Ns)
    for (int64_t M = 1; M < 700000; M += 1 + M / 97)
      for (bool exact : {false, true}) check(M, N, 144, exact);
  for (int64_t M = 65500; M < 140000; M += 13)          // more tile rows than compute units
    for (int64_t N : {129, 200, 256, 384, 512}) check(M, N, 144, false);
  for (int64_t N = 1; N < 40000; N += 1 + N / 97)
    for (int64_t M : {1, 17, 33, 65, 129, 300, 1000, 2048, 4096, 65537})
      for (int64_t K : {16, 5120, 17408}) check(M, N, K, false);
  if (!split) { puts("no shape splits its columns"); return 1; }
  return bad != 0;
}
"""


@pytest.mark.skipif(CXX is None, reason="no host C++ compiler")
def test_every_launch_has_work(tmp_path):
    src, exe = tmp_path / "sweep.cpp", tmp_path / "sweep"
    src.write_text(SWEEP)
    subprocess.run([CXX, "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
