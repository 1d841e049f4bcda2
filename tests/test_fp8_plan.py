"""The plan of the FP8 product (csrc/fp8_plan.hpp, host arithmetic) compiled with the host
compiler and swept over shapes: every launch it leads to has work."""
import os
import re
import shutil
import subprocess

import pytest

import _fp8_shapes

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


PRINT = r"""
#include <cstdio>
#include <cstdlib>
#include "fp8_plan.hpp"
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    const gwb::GemmPlan p = gwb::fp8_gemm_plan(atol(argv[i]), atol(argv[i + 1]), atol(argv[i + 2]), false);
    printf("%d %d %d\n", p.kernel, p.splits > 1, p.wide < atol(argv[i + 1]));
  }
}
"""


@pytest.mark.skipif(CXX is None, reason="no host C++ compiler")
def test_the_shapes_of_the_gpu_tests_reach_every_kernel(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PRINT)
    subprocess.run([CXX, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    text = open(os.path.join(CSRC, "fp8_plan.hpp")).read()
    names = re.search(r"enum \{([^}]*)\}", text).group(1).replace("\n", " ").replace(" ", "").split(",")
    for table in (_fp8_shapes.SHAPES, _fp8_shapes.LONG):
        args = [str(v) for shape in table.values() for v in shape]
        out = subprocess.run([str(exe), *args], capture_output=True, text=True, check=True).stdout.split("\n")
        got = []
        for line in out[:-1]:
            kernel, split, tail = map(int, line.split())
            got.append(names[kernel] + (" split" if split else "") + (" tail" if tail else ""))
        assert got == list(table)
    assert {n.split()[0] for n in _fp8_shapes.SHAPES} == set(names)
    assert {n.split()[0] for n in _fp8_shapes.LONG} == {n for n in names if n.startswith("kTile")}
    assert all((k + 127) // 128 > 64 for _, _, k in _fp8_shapes.LONG.values())
