"""The mixture of experts against its definition, rounded once: hidden values
go into the second products as two numbers of 16 bits, so that what a result is
off by is fp32 sums and half a step of its own type."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import serve_reference as ref  # noqa: E402
from fused_reference import SLOPE, STEPS, U32, activation, half_step, product, tiny  # noqa: E402
from test_gpu_fused import TYPES, call, check, pg, randn  # noqa: E402,F401
from test_gpu_serve import equal, moe_case  # noqa: E402

pytestmark = pytest.mark.gpu
FMT = ["f16", "bf16"]


def layer(x, router, w, down, k, act, normalize):
    """(experts, (y, bound)) in 64 bits."""
    dtype = x.dtype
    (M, D), (E, _, F) = x.shape, down.shape
    experts, (p, ep) = ref.route(x, router, k, normalize)
    y, e, size = (torch.zeros((M, D), dtype=torch.float64, device=x.device) for _ in range(3))
    for j in range(E):
        row, place = torch.nonzero(experts == j, as_tuple=True)
        if len(row) == 0:
            continue
        g, eg = product(x[row], w[j, :F])
        u, eu = product(x[row], w[j, F:])
        a, _ = activation(act, g)
        ea = SLOPE * eg + STEPS * U32 * (a.abs() + g.abs() * 0.5 + U32)
        h, eh = a * u, ea * u.abs() + a.abs() * eu + ea * eu
        # a number and its rest, each off by half a step of what it is: half_step(t)^2; and the spacing of the subnormals, in
        # f16 after a power of two that takes a row's largest to 2^14 or more
        eh = eh + half_step(dtype) ** 2 * (h.abs() + eh)
        eh = eh + (2.0 ** -25 * 2.0 ** -14 * h.abs().amax(1, keepdim=True) if dtype == torch.float16 else tiny(dtype))
        d = down[j].double()
        v = h @ d.t()
        # sums of the numbers, and of the rests, which are half_step(t) as large
        ev = eh @ d.abs().t() + (1 + half_step(dtype)) * (F + 8) * U32 * ((h.abs() + eh) @ d.abs().t())
        pj, epj = p[row, place][:, None], ep[row, place][:, None]
        y[row] += pj * v
        e[row] += pj * ev + epj * (v.abs() + ev)
        size[row] += pj * (v.abs() + ev)
    e = e + (k + 25) * U32 * size  # the weight, an expert's runs on several waves, both parts, and the choices' sum
    return experts, (y, e + half_step(dtype) * (y.abs() + e) + tiny(dtype))


# M, D, F, E, k: each count of token blocks on eight waves and on four, a whole pass of tokens and one more, widths below
# eight, odd widths, a last chunk of one token
SHAPES = [(1, 16, 5, 1, 1), (1, 256, 200, 8, 2), (3, 70, 33, 5, 2), (8, 96, 64, 2, 1), (9, 96, 64, 1, 1), (17, 130, 257, 1, 1),
          (33, 64, 40, 1, 1), (65, 72, 96, 2, 2), (30, 128, 96, 12, 4), (64, 200, 6, 8, 2), (37, 2050, 301, 60, 4),
          (64, 2100, 1050, 8, 2), (64, 2100, 1050, 16, 2), (64, 1000, 700, 2, 1)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("act,normalize", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("M,D,F,E,k", SHAPES)
def test_rounded_once(pg, fmt, act, normalize, M, D, F, E, k):
    ops = moe_case(7 * M + D + F + E, fmt, M, D, F, E)
    y, experts, _ = call(pg, fmt, "moe", *ops, k, act=act, normalize=normalize, routing=True)
    want, bounded = layer(*ops, k, act, normalize)
    equal("experts", experts, want)
    check("y", y, bounded)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,F", [(1, 64), (9, 5), (20, 333)])
def test_infinite_weights_of_second_products(pg, fmt, M, F):
    # an infinity times a hidden value is an infinity of its sign, and not that of a rest with the other one
    D, E = 24, 2
    x, router, w, down = moe_case(61, fmt, M, D, F, E)
    down[:, 3, F // 2], down[:, 7, F // 2] = math.inf, -math.inf
    y, experts, _ = call(pg, fmt, "moe", x, router, w, down, 1, routing=True)
    for m in range(M):
        wide = w[experts[m, 0]].double()
        g, u = wide[F // 2] @ x[m].double(), wide[F + F // 2] @ x[m].double()
        sign = torch.sign(g * u)
        assert y[m, 3] == sign * math.inf and y[m, 7] == -sign * math.inf
    others = [c for c in range(D) if c not in (3, 7)]
    assert torch.isfinite(y[:, others]).all()


@pytest.mark.parametrize("M", [1, 20])
def test_infinite_hidden_values(pg, M):
    # a gate past fp32: infinite hidden values have no rest
    D, F, E = 24, 40, 3
    x, router, w, down = moe_case(62, "bf16", M, D, F, E)
    x[:, 0] = 3e38
    router[:, 0] = 0
    w[:, :, 0] = 0
    w[:, 5, 0] = 2.0
    y, experts, _ = pg.pgemm_bf16_moe(x, router, w, down, 1, routing=True)
    for m in range(M):
        e = experts[m, 0]
        up = w[e, F + 5].double() @ x[m].double()
        want = torch.sign(up * down[e, :, 5].double()) * math.inf
        assert torch.equal(y[m].double(), want)
