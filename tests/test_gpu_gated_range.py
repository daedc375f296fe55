"""The range of the gated block's f16 gradients: the derivative by the
projections, which is rounded to 16 bits inside the call, keeps its bits where
dh is small and does not overflow where dx or dW do not."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fused_reference as ref  # noqa: E402
from test_gpu_fused import TYPES, call, check, pg, randn  # noqa: E402,F401
from test_gpu_fused_edges import check_range  # noqa: E402

pytestmark = pytest.mark.gpu


def norm(t):
    """What stands for the largest norm of a row: the sums of squares of 4096 values at a time, as they lie, and of as many as a row may touch (of the last, values may count twice)."""
    flat = torch.nn.functional.pad(t.double().flatten() ** 2, (0, -t.numel() % 4096))
    return (2 * (-(-(t.shape[1] - 1) // 4096) + 1) * flat.view(-1, 4096).sum(1).max()).sqrt()


def gradients(x, w, act, dh):
    """Gradients whose derivative by the projections is rounded relative to
    itself alone, but for what is 2^39 below the largest that dh and the norms
    of x's and W's rows allow (half a step of a subnormal, with that largest one
    taken to at least 2^14)."""
    F = w.shape[0] // 2
    g, eg = ref.product(x, w[:F])
    u, eu = ref.product(x, w[F:])
    a, s = ref.activation(act, g)
    ea = ref.SLOPE * eg + ref.STEPS * ref.U32 * (a.abs() + g.abs() * 0.5 + ref.U32)
    d = dh.double()
    es = ref.BEND * eg + ref.STEPS * ref.U32 * (s.abs() + 1)
    dg, du = d * u * s, d * a
    eg2 = d.abs() * (eu * s.abs() + u.abs() * es + eu * es + 4 * ref.U32 * (u * s).abs())
    eu2 = d.abs() * ea
    dy, edy = torch.cat([dg, du], 1), torch.cat([eg2, eu2], 1)
    lowest = d.abs().max() * norm(x) * norm(w) * 2.0 ** -39
    edy = edy + ref.half_step(x.dtype) * (dy.abs() + edy) + lowest
    return {"dx": ref._times(dy, edy, w.double().t(), x.dtype),
            "dw": ref._times(dy.t().contiguous(), edy.t().contiguous(), x.double().t(), x.dtype)}


# one token and hidden value, so that a gradient shows what its derivative lost;
# odd sizes; K in pieces; large tiles and their rest in small ones
SIZES = [(1, 1, 40), (1, 3, 8), (3, 1, 1), (130, 70, 64), (129, 65, 1001), (600, 100, 1024), (40, 3000, 104), (2100, 1500, 130)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("size", [1e-7, 1e-5, 1e-3, 1.0])
@pytest.mark.parametrize("wide", [64.0, 1 / 64])  # x's entries; W's are the inverse, over the root of D
@pytest.mark.parametrize("M,F,D", SIZES)
def test_small_derivatives_keep_their_bits(pg, act, size, wide, M, F, D):
    gen = torch.Generator().manual_seed(M + F + D)
    x = randn(gen, M, D, scale=wide).half().cuda()
    w = randn(gen, 2 * F, D, scale=D ** -0.5 / wide).half().cuda()
    dh = randn(gen, M, F, scale=size).half().cuda()
    want = gradients(x, w, act, dh)
    _, saved = pg.pgemm_f16_gated(x, w, act=act, save=True)
    for keep in (saved, None):
        dx, dw = pg.pgemm_f16_gated_bwd(dh, x, w, saved=keep, act=act)
        check("dx", dx, want["dx"])
        check("dw", dw, want["dw"])


@pytest.mark.parametrize("wide", [2000.0, 0.01])
@pytest.mark.parametrize("M", [1, 150])
def test_derivatives_past_the_type(pg, wide, M):
    # dh u is some 1e5: past f16's end, where dx (wide 2000) or dW (0.01) is not
    D, F = 64, 1
    gen = torch.Generator().manual_seed(5)
    x = (torch.rand((M, D), generator=gen) + 0.5).mul_(wide).half().cuda()
    w = ((torch.rand((2 * F, D), generator=gen) + 0.5) * (200.0 / wide)).half().cuda()
    sign = torch.where(torch.arange(M) % 2 == 0, 1.0, -1.0)[:, None].expand(M, F)
    dh = (sign * 8).half().cuda()
    want = gradients(x, w, "silu", dh)
    assert ((dh.double() * (x.double() @ w[F:].double().t())).abs() > 70000).all()
    finite = "dx" if wide > 1 else "dw"
    assert (want[finite][0].abs() < 60000).all()
    _, saved = pg.pgemm_f16_gated(x, w, save=True)
    for keep in (saved, None):
        got = dict(zip(("dx", "dw"), pg.pgemm_f16_gated_bwd(dh, x, w, saved=keep)))
        for name in got:
            check_range(name, got[name], *want[name])


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_what_is_not_finite_leaves_the_rest(pg, fmt):
    # an infinity or NaN in one token's dh or x: the other tokens' dx as without it
    gen = torch.Generator().manual_seed(6)
    M, F, D = 140, 40, 72
    x = randn(gen, M, D).to(TYPES[fmt]).cuda()
    w = randn(gen, 2 * F, D, scale=D ** -0.5).to(x.dtype).cuda()
    dh = randn(gen, M, F, scale=1e-5).to(x.dtype).cuda()
    want = ref.gated(x, w, "silu", dh)["dx"] if fmt == "bf16" else gradients(x, w, "silu", dh)["dx"]
    rest = torch.arange(M, device="cuda") != 7
    for poison in (math.inf, -math.inf, math.nan):
        for where in ("dh", "x"):
            px, pd = x.clone(), dh.clone()
            (px if where == "x" else pd)[7, 3] = poison
            _, saved = call(pg, fmt, "gated", px, w, save=True)
            for keep in (saved, None):
                dx, _ = call(pg, fmt, "gated_bwd", pd, px, w, saved=keep)
                check("dx", dx[rest], (want[0][rest], want[1][rest]))
                assert not dx[7].isfinite().any()
    # nothing but zeros
    dx, dw = call(pg, fmt, "gated_bwd", torch.zeros_like(dh), x, w)
    assert not dx.any() and not dw.any()


def test_range_in_a_graph(pg):
    # the factor is found anew by every replay
    gen = torch.Generator().manual_seed(7)
    M, F, D = 300, 90, 104
    x = randn(gen, M, D).half().cuda()
    w = randn(gen, 2 * F, D, scale=D ** -0.5).half().cuda()
    dh = randn(gen, M, F).half().cuda()

    def step():
        _, saved = pg.pgemm_f16_gated(x, w, save=True)
        return [*pg.pgemm_f16_gated_bwd(dh, x, w, saved=saved), *pg.pgemm_f16_gated_bwd(dh, x, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for size in (1e-6, 1.0, 1e-3, 30.0):
        dh.copy_(randn(gen, M, F, scale=size).half())
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        check("dx", out[0], gradients(x, w, "silu", dh)["dx"])
    pg.release_workspace(side)
