"""Every way through the 8-bit products and the mixture of experts on the GPU
(shapes of serve_paths.py), against 64-bit references."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import serve_paths as paths  # noqa: E402
import serve_reference as ref  # noqa: E402
from test_gpu_fused import TYPES, call, check, pg  # noqa: E402,F401
from test_gpu_fused_edges import check_range  # noqa: E402
from test_gpu_moe_values import layer  # noqa: E402
from test_gpu_serve import equal, i8_case, moe_case  # noqa: E402

pytestmark = pytest.mark.gpu
FMT = ["f16", "bf16"]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K,gated,what", paths.I8_CUTS)
def test_i8_cuts(pg, fmt, M, N, K, gated, what):
    x, w, ws = i8_case(M + N + K, fmt, M, N, K, gated)
    q, xs = ref.quant(x)
    act = "gelu" if gated else None
    want = ref.i8(q, xs, w, ws, TYPES[fmt], act)
    if gated:
        y = call(pg, fmt, "i8_gated", q, w, ws, xs=xs, act=act)
    else:
        y = call(pg, fmt, "i8", q, w, ws, xs=xs)
    check(what, y, want)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,gated", paths.I8_LONGEST)
def test_i8_largest_sums_of_few_tokens(pg, fmt, M, N, gated):
    # -128 times -128 over the longest K: 2^31 - 2^18; scales whose product the type holds, though neither order of
    # multiplication keeps all partial products in fp32
    K, rows = paths.LONGEST, 2 * N if gated else N
    q = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    q[1, ::2] = 127
    w = torch.full((rows, K), -128, dtype=torch.int8, device="cuda")
    w[1::4] = 127
    xs = torch.full((M,), 2.0 ** -40, device="cuda")
    xs[0], xs[1], xs[2] = 2.0 ** 100, 2.0 ** -126, 2.0 ** -149
    ws = torch.tensor([2.0 ** 9, 2.0 ** -130, 2.0 ** 95, 2.0 ** 118], device="cuda").repeat(rows // 4)
    some = torch.unique(torch.cat([torch.arange(min(N, 40)), torch.arange(max(N - 40, 0), N)])).cuda()
    if gated:
        ws[N:] = 2.0 ** -20
        both = torch.cat([some, some + N])
        want = ref.i8(q, xs, w[both], ws[both], TYPES[fmt], "silu")
        y = call(pg, fmt, "i8_gated", q, w, ws, xs=xs)
    else:
        want = ref.i8(q, xs, w[some], ws[some], TYPES[fmt])
        y = call(pg, fmt, "i8", q, w, ws, xs=xs)
    check_range("y", y[:, some], *want)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("shape,hidden,second", paths.MOE)
def test_moe_cuts(pg, fmt, shape, hidden, second):
    M, D, F, E, k = shape
    ops = moe_case(5 * M + D, fmt, M, D, F, E)
    y, experts, _ = call(pg, fmt, "moe", *ops, k, act="gelu", routing=True)
    want, bounded = layer(*ops, k, "gelu", True)
    equal("experts", experts, want)
    check(f"{hidden} {second}", y, bounded)
