"""The fused operators' largest launches, from their host planner and entry
points on the CPU: a dispatch has fewer than 2^32 work-items, and rows past a
matrix's last ones stay below 2^31."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from software_pipelined_tiled_pipeline_amd import build, pgemm

OK, SHAPE = 0, 2
A = 4096  # a pointer that is aligned and never read
LIMIT = 1 << 32

# work-items of every launch that a plan makes, as the launch templates make them
PROGRAM = r"""
#include "fused.hpp"
#include <cstdio>
using namespace pgemm;
static void tiles(const char *what, int64_t M, int64_t N, bool dual, const Tiling &t) {
  if (M == 0 || N == 0) return;
  auto grid = [&](int64_t m, int64_t n, bool large) {
    const int64_t w = large ? 256 : 128;
    printf("%s %lld\n", what, (long long)(per(m, w) * per(n, dual ? w / 2 : w) * t.split * (large ? 256 : 512)));
  };
  if (!t.large) return grid(M, N, false);
  const int64_t m = t.cut_m && t.cut_m < M ? t.cut_m : M, n = t.cut_n && t.cut_n < N ? t.cut_n : N;
  grid(m, n, true);
  if (m < M || n < N) grid(m < M ? M - m : M, n < N ? N - n : N, false);
}
int main() {
  char op;
  long long M, N, K;
  while (scanf(" %c %lld %lld %lld", &op, &M, &N, &K) == 4) {
    if (op == 'g') {
      for (int bwd = 0; bwd < 2; ++bwd) {
        const GatedPlan p = plan_gated(M, N, K, bwd, false);
        if (!p.skinny) tiles("projections", M, N, true, p.forward);
        if (bwd) tiles("dx", M, K, false, p.dx), tiles("dw", 2 * N, K, false, p.dw);
      }
    } else {
      const XentPlan f = plan_xent(M, N, K, false), b = plan_xent(M, N, K, true);
      tiles("logits", M, N, false, f.logits);
      printf("join %lld\n", (long long)(join_groups(M) * 1024));
      tiles("dz", M, b.piece, false, b.logits);
      tiles("dw", b.piece, K, false, b.dw);
      tiles("dx", M, K, false, b.dx);
    }
    puts("end");
  }
}
"""


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("no compiler or HIP headers")
    d = tmp_path_factory.mktemp("plans")
    (d / "plans.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", build.CSRC, "-I",
                    os.path.join(build.ROOT, "include"), str(d / "plans.cpp"), "-o", str(d / "plans")], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(d / "plans")], input=text, capture_output=True, text=True, check=True).stdout
        found = [[]]
        for line in out.splitlines():
            if line == "end":
                found.append([])
            else:
                name, n = line.split()
                found[-1].append((name, int(n)))
        return found[:-1]
    return run


def accepted(L, op, M, N, K):
    n = ctypes.c_int64()
    return L.pgemm_fused_workspace({"g": 2, "x": 4}[op], M, N, K, ctypes.byref(n)) == OK


def test_every_launch_of_an_accepted_call_fits(launches):
    L = pgemm.lib()
    rng = random.Random(1)

    def size(top):
        return min(top, max(1, int(2 ** rng.uniform(0, top.bit_length())) + rng.randrange(-3, 4)))
    cases = [("x", 1 << 26, 256, 8), ("x", 1360628991, 257, 8), ("x", (1 << 31) - 256, 1, 1), ("x", 1, (1 << 31) - 256, 1),
             ("g", (1 << 31) - 256, 1, 1), ("g", 1 << 30, 128, 8), ("g", 1360628991, 129, 8), ("g", 1, 1 << 21, 1 << 22)]
    cases += [("x", size((1 << 31) - 256), size((1 << 31) - 256), size(1 << 22)) for _ in range(6000)]
    cases += [("g", size((1 << 31) - 256), size(1 << 21), size(1 << 22)) for _ in range(6000)]
    # about the largest that are taken: M by N in few and in many columns
    cases += [("x", (1 << 31) - 256 - rng.randrange(1 << rng.randrange(31)), rng.randrange(1, 2000), rng.randrange(1, 70))
              for _ in range(6000)]
    cases = [c for c in cases if accepted(L, *c)]
    assert len(cases) > 5000
    for case, found in zip(cases, launches(cases)):
        assert found
        for name, n in found:
            assert 0 < n < LIMIT, (case, name, n)


def test_rows_past_the_last_tile_stay_below_2_31():
    L = pgemm.lib()
    for op in "gx":
        assert accepted(L, op, (1 << 31) - 256, 1, 1)
        for M in ((1 << 31) - 255, (1 << 31) - 1):
            assert not accepted(L, op, M, 1, 1)
    assert accepted(L, "x", 1, (1 << 31) - 256, 1) and not accepted(L, "x", 1, (1 << 31) - 255, 1)
    for fmt in ("f16", "bf16"):
        for M, V in (((1 << 31) - 255, 1), (1, (1 << 31) - 255)):
            assert getattr(L, f"pgemm_{fmt}_xent")(A, A, A, A, A, M, V, 1, -100, None) == SHAPE
            assert getattr(L, f"pgemm_{fmt}_xent_bwd")(A, 1, A, A, A, A, A, A, M, V, 1, -100, None) == SHAPE
        assert getattr(L, f"pgemm_{fmt}_gated")(A, A, A, None, (1 << 31) - 255, 1, 1, 0, None) == SHAPE
        assert getattr(L, f"pgemm_{fmt}_gated_bwd")(A, A, A, None, A, A, (1 << 31) - 255, 1, 1, 0, None) == SHAPE
