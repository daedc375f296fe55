"""The shapes of serve_paths.py take the ways that they are named for, by the
library's own planner (CPU only)."""
import os
import shutil
import subprocess
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import serve_paths as paths  # noqa: E402

from software_pipelined_tiled_pipeline_amd import build  # noqa: E402

PROGRAM = r"""
#include "serve.hpp"
#include <cstdio>
using namespace pgemm;
int main() {
  char op;
  long long a, b, c, d, e;
  while (scanf(" %c %lld %lld %lld %lld %lld", &op, &a, &b, &c, &d, &e) == 6) {
    if (op == 'i') {  // M, N, K, gated
      const I8Plan p = plan_i8(a, b, c, d != 0, true);
      printf("%d %d %lld %lld\n", p.few, p.tiles.large, (long long)p.tiles.cut_m, (long long)p.tiles.cut_n);
    } else {  // M, D, F, E, top_k
      const MoeCut h = moe_cut(a, d, b, c, e, false), s = moe_cut(a, d, b, c, e, true);
      printf("%d %d %d %d\n", h.blocks, h.waves, s.blocks, s.waves);
    }
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("no compiler or HIP headers")
    d = tmp_path_factory.mktemp("paths")
    (d / "paths.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", build.CSRC, "-I",
                    os.path.join(build.ROOT, "include"), str(d / "paths.cpp"), "-o", str(d / "paths")], check=True)

    def run(*case):
        out = subprocess.run([str(d / "paths")], input=" ".join(map(str, case)), capture_output=True, text=True, check=True)
        return tuple(int(n) for n in out.stdout.split())
    return run


@pytest.mark.parametrize("M,N,K,gated,what", paths.I8_CUTS)
def test_cuts_of_8_bit_products(plan, M, N, K, gated, what):
    few, large, rows, columns = plan("i", M, N, K, int(gated), 0)
    assert not few and large
    assert (0 < rows < M and not columns) if what == "rows" else (0 < columns < N and not rows)


@pytest.mark.parametrize("M,N,gated", paths.I8_LONGEST)
def test_longest_sums_of_few_tokens(plan, M, N, gated):
    assert plan("i", M, N, paths.LONGEST, int(gated), 0)[0]


@pytest.mark.parametrize("shape,hidden,second", paths.MOE)
def test_cuts_of_a_mixture(plan, shape, hidden, second):
    assert plan("m", *shape) == hidden + second


def test_every_cut_of_a_mixture_is_run():
    every = {(1, 8), (1, 4), (2, 8), (2, 4), (4, 4)}
    assert {h for _, h, _ in paths.MOE} == every == {s for _, _, s in paths.MOE}
