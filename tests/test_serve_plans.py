"""The serving operators' largest launches and workspaces, from their host planner
and entry points on the CPU: a dispatch has fewer than 2^32 work-items, its other
dimensions fewer than 2^16 workgroups, and workspaces hold what the plans place in them."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from software_pipelined_tiled_pipeline_amd import build, pgemm

OK = 0
LIMIT = 1 << 32

# every launch as the launch templates make it, and every piece of a workspace
PROGRAM = r"""
#include "serve.hpp"
#include <cstdio>
using namespace pgemm;
static void grid(const char *what, int64_t x, int64_t y = 1, int64_t z = 1) {
  printf("%s %lld %lld %lld\n", what, (long long)x, (long long)y, (long long)z);
}
static void tiles(int64_t M, int64_t N, bool dual, const Tiling &t) {
  auto some = [&](int64_t m, int64_t n, bool large) {
    const int64_t w = large ? 256 : 128;
    grid("tiles", per(m, w) * per(n, dual ? w / 2 : w) * t.split * (large ? 256 : 512));
  };
  if (!t.large) return some(M, N, false);
  const int64_t m = t.cut_m && t.cut_m < M ? t.cut_m : M, n = t.cut_n && t.cut_n < N ? t.cut_n : N;
  some(m, n, true);
  if (m < M || n < N) some(m < M ? M - m : M, n < N ? N - n : N, false);
}
static void piece(int64_t at, int64_t bytes) { printf("piece %lld %lld 1\n", (long long)at, (long long)bytes); }
int main() {
  char op;
  long long a, b, c, d, e;
  while (scanf(" %c %lld %lld %lld %lld %lld", &op, &a, &b, &c, &d, &e) == 6) {
    if (op == 'i') {  // M, N, K, gated, quantized
      const I8Plan p = plan_i8(a, b, c, d != 0, e != 0);
      if (p.few) {
        const int64_t cols = per(b, d ? 16 : 32), mt = a <= 16 ? 16 : a <= 32 ? 32 : 64;
        grid("few", cols * (cols * per(a, mt) <= 512 ? 512 : 256), per(a, mt));
      } else {
        tiles(a, b, d != 0, p.tiles);
      }
      if (!e && !p.own) piece(p.q, a * up_to(c, 16)), piece(p.s, a * 4);
      if (!p.few && p.tiles.split > 1) piece(p.part, p.tiles.split * a * up_to(b, 4) * 4);
      printf("bytes %lld 1 1\n", (long long)p.bytes);
    } else {  // M, E, D, F, top_k
      const MoePlan p = plan_moe(a, b, c, d, e);
      const int64_t chunks = per(a, kMoeChunkTokens);
      grid("logits", b * 256, a <= 4 ? a : per(a, 4));
      grid("choice", a * 1024);
      if (d) grid("hidden", per(d, 16) * 512, p.slots, chunks);
      if (c) grid("second", per(c, 32) * 512, p.slots, chunks);
      piece(p.logits, a * b * 8), piece(p.experts, a * e * 4), piece(p.weights, a * e * 4);
      piece(p.h, a * e * d * 4), piece(p.tops, a * e * 4);
      if (e > 1) piece(p.products, a * e * c * 4);
      printf("bytes %lld 1 1\n", (long long)p.bytes);
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
                name, *n = line.split()
                found[-1].append((name, *map(int, n)))
        return found[:-1]
    return run


def workspace(L, op, *sizes):
    """Bytes that the library asks for, None if it takes no such call."""
    n = ctypes.c_int64()
    return n.value if {"i": L.pgemm_i8_workspace, "m": L.pgemm_moe_workspace}[op](*sizes, ctypes.byref(n)) == OK else None


def sizes(rng, top):
    return min(top, max(1, int(2 ** rng.uniform(0, top.bit_length())) + rng.randrange(-3, 4)))


def test_every_launch_and_workspace_fits(launches):
    L, rng = pgemm.lib(), random.Random(1)
    big = (1 << 31) - 256
    cases = [("i", M, N, K, g, q) for M, N, K in ((big, 1, 1), (1, big // 2, 16), (1, 1 << 27, (1 << 17) - 16), (256, 1 << 26, 64),
                                                  (4, 1 << 26, 8192), (257, 1 << 23, 131056)) for g in (0, 1) for q in (0, 1)]
    cases += [("m", M, E, D, F, k) for M in (1, 64, 65, 32767) for E, k in ((1, 1), (16, 16), (1024, 1), (1024, 32))
              for D, F in ((0, 0), (1 << 22, 1), (1, 1 << 17), (1 << 22, 1 << 17))]
    for _ in range(6000):
        cases.append(("i", sizes(rng, big), sizes(rng, big), rng.randrange(0, (1 << 17) - 15), rng.randrange(2), rng.randrange(2)))
        cases.append(("i", sizes(rng, 512), sizes(rng, big), sizes(rng, (1 << 17) - 16), rng.randrange(2), rng.randrange(2)))
        E = sizes(rng, 1024)
        cases.append(("m", sizes(rng, 32767), E, sizes(rng, 1 << 22), sizes(rng, 1 << 17), rng.randrange(1, min(E, 32) + 1)))
    wanted = [workspace(L, *c) for c in cases]
    cases, wanted = zip(*[(c, w) for c, w in zip(cases, wanted) if w is not None])
    assert sum(c[0] == "i" for c in cases) > 5000 and sum(c[0] == "m" for c in cases) > 5000
    for case, want, found in zip(cases, wanted, launches(cases)):
        assert found.pop()[:2] == ("bytes", want)
        end = 0
        for name, x, y, z in sorted(found, key=lambda f: f[1] if f[0] == "piece" else -1):
            if name == "piece":
                assert x >= end and x % 16 == 0, (case, found)
                end = x + y
            else:
                assert 0 < x < LIMIT and 0 < y < 1 << 16 and 0 < z < 1 << 16, (case, name, x, y, z)
        assert end <= want, (case, end, want)


def test_reach_of_offsets_in_a_launch():
    """Sixteen weight rows, and a chunk's tokens and hidden values, stay below 2^31 bytes: the reach of their offsets."""
    widest, hidden, chunk, top_k, values = (1 << 17) - 16, 1 << 17, 64, 32, 1 << 22
    L = pgemm.lib()
    assert workspace(L, "i", 1, 1, widest, 0, 0) is not None and workspace(L, "i", 1, 1, widest + 1, 0, 0) is None
    assert workspace(L, "m", 64, 32, values, hidden, top_k) is not None
    assert workspace(L, "m", 64, 64, 8, 8, top_k + 1) is None
    assert workspace(L, "m", 64, 32, values + 1, 8, 2) is None and workspace(L, "m", 64, 32, 8, hidden + 1, 2) is None
    assert 16 * (widest + 16) < 1 << 31 and 16 * values * 2 < 1 << 31
    assert chunk * values * 2 < 1 << 31 and chunk * top_k * hidden * 4 < 1 << 31
    # the longest sums of 8-bit products stay in int32
    assert widest * 128 * 128 < 1 << 31 <= (widest + 16) * 128 * 128
