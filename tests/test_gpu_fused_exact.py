"""The gated block and the cross entropy on operands whose results are exact:
whatever a tile, a piece of K or a remainder adds or leaves out shows, where a
bound of fp32's rounding over thousands of products would hide it.

Gated block: gates of 34 to 46, where the activation is the identity and its
slope 1 to fp32's last bit, up projections of at most 6 and dh of -1, 0 or 1, so
that the derivative by the projections is of small integers.  Cross entropy:
tokens that are a multiple of a code of +-1, with the codes of the vocabulary's
rows some distance apart, so that each softmax, rounded to 16 bits, is 1 at one
row and 0 at the others."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_fused import TYPES, call, pg  # noqa: E402,F401

FMT = ["f16", "bf16"]
# What tokens are times their code, and how far below a row's largest logit the
# others then have to lie to round to 0: 2^-39 in f16, where a derivative is
# multiplied by 2^14, and bf16's smallest, 2^-133.  The largest logit, some
# 1.5e3 and 6e3, is known to 2^-24 of itself twice over, which leaves 1 within
# half a step of it (2^-12 and 2^-9).
TIMES, GAP = {"f16": 4, "bf16": 16}, {"f16": 28, "bf16": 96}


def gated_case(seed, fmt, M, F, D):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randint(-1, 2, (M, D), generator=gen).float()
    x[:, 0] = 1
    w = torch.zeros(2 * F, D)
    at = torch.randint(1, D, (2 * F, 6), generator=gen)  # a place may come twice: the last value stays
    w.scatter_(1, at, torch.randint(-1, 2, (2 * F, 6), generator=gen).float())
    w[:F, 0] = 40
    dh = torch.randint(-1, 2, (M, F), generator=gen).float()
    assert max(F * (40 * 6 + 46), M * 46) < 1 << 24  # every partial sum is exact
    return tuple(t.to(TYPES[fmt]) for t in (x, w, dh))


def gated_exact(x, w, dh):
    F = w.shape[0] // 2
    x64, w64, d = x.double(), w.double(), dh.double()
    g, u = x64 @ w64[:F].t(), x64 @ w64[F:].t()
    assert g.min() >= 34 and g.max() <= 46 and u.abs().max() <= 6
    dy = torch.cat([d * u, d * g], 1)
    return [t.float().to(x.dtype) for t in (g * u, dy @ w64, dy.t().contiguous() @ x64)]


# sizes about the tiles' edges, large tiles with their rest by rows and by
# columns, small ones alone on a CU and two to one, and pieces of K for each product
GATED = [(1, 1, 8), (65, 33, 70), (257, 127, 1001), (300, 1500, 72), (40, 6000, 104), (129, 5000, 260), (600, 100, 1024),
         (2100, 3000, 130), (3200, 40, 4100), (130, 1600, 4104), (4095, 2731, 1001), (4352, 2200, 520), (5000, 1024, 264)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,F,D", GATED)
def test_gated_exact(pg, fmt, act, M, F, D):
    x, w, dh = (t.cuda() for t in gated_case(M + F + D, fmt, M, F, D))
    h, dx, dw = gated_exact(x, w, dh)
    assert torch.equal(call(pg, fmt, "gated", x, w, act=act), h)
    got, saved = call(pg, fmt, "gated", x, w, act=act, save=True)
    assert torch.equal(got, h)
    for keep in (saved, None):
        a, b = call(pg, fmt, "gated_bwd", dh, x, w, saved=keep, act=act)
        assert torch.equal(a, dx)
        assert torch.equal(b, dw)


def xent_case(seed, fmt, M, V, D):
    gen = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 2, (V, D), generator=gen).float() * 2 - 1
    top = torch.randint(0, V, (M,), generator=gen)
    target = (top + torch.randint(1, V, (M,), generator=gen)) % V  # another one
    target[torch.rand(M, generator=gen) < 0.1] = -100
    assert M * TIMES[fmt] < 1 << 24 and D * TIMES[fmt] < 6000
    return (codes[top] * TIMES[fmt]).to(TYPES[fmt]), codes.to(TYPES[fmt]), target, top


def xent_exact(x, w, target, top):
    """loss, lse, dx and dw for dloss of 1."""
    V = w.shape[0]
    own = (x.float() * w[top].float()).sum(1)
    counts = target != -100
    t = torch.where(counts, target, top)
    loss = own - (x.float() * w[t].float()).sum(1)
    x64, c = x.double(), counts.double()[:, None]
    dw = torch.zeros(V, x.shape[1], dtype=torch.float64, device=x.device)
    dw.index_add_(0, top, x64 * c)
    dw.index_add_(0, t, -x64 * c)
    dx = (w[top].double() - w[t].double()) * c
    return loss, own, dx.float().to(x.dtype), dw.float().to(x.dtype)


def distance(x, w, top):
    """How far below the largest logit of its row any other is."""
    least = float("inf")
    for i in range(0, x.shape[0], 512):
        z = x[i:i + 512].float() @ w.float().t()
        own = z.gather(1, top[i:i + 512, None])
        z.scatter_(1, top[i:i + 512, None], float("-inf"))
        least = min(least, float((own - z.max(1).values[:, None]).min()))
    return least


# (4100, 66000, 80) and (2100, 130001, 96): the derivative by the logits takes pieces
XENT = [(1, 7, 64), (65, 1000, 72), (130, 257, 136), (200, 3001, 129), (75, 13120, 352), (700, 20000, 80), (2049, 6200, 130),
        (1021, 50021, 100), (4100, 66000, 80), (2100, 130001, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,V,D", XENT)
def test_xent_exact(pg, fmt, M, V, D):
    x, w, target, top = (t.cuda() for t in xent_case(M + V + D, fmt, M, V, D))
    assert distance(x, w, top) >= GAP[fmt]
    loss, lse, dx, dw = xent_exact(x, w, target, top)
    got = call(pg, fmt, "xent", x, w, target)
    # the largest logit's exponential and the sum of it and 0's logarithm: 2^-24 of the logit each, and the result's rounding
    off = 3 * 2.0 ** -24 * lse.max()
    assert (got[0] - loss).abs().max() <= off and (got[1] - lse).abs().max() <= off
    for dloss in (torch.ones((), device="cuda"), torch.ones(M, device="cuda")):
        a, b = call(pg, fmt, "xent_bwd", dloss, x, w, target, got[1])
        assert torch.equal(a, dx)
        assert torch.equal(b, dw)


@pytest.mark.parametrize("fmt", FMT)
def test_the_comparison_finds_planted_faults(fmt):
    # a K tile of 64 that a product left out
    x, w, dh = gated_case(3, fmt, 300, 1500, 72)
    h, dx, dw = gated_exact(x, w, dh)
    less = dh.clone()
    less[:, 640:704] = 0  # of dx's, which runs over the hidden columns
    assert (gated_exact(x, w, less)[1] != dx).float().mean() > 0.5
    less = dh.clone()
    less[64:128] = 0  # of dW's, over the tokens
    assert (gated_exact(x, w, less)[2] != dw).float().mean() > 0.5
    x, w, target, top = xent_case(4, fmt, 300, 1000, 80)
    assert distance(x, w, top) >= GAP[fmt]
    loss, lse, dx, dw = xent_exact(x, w, target, top)
    less = target.clone()
    less[64:128] = -100
    assert (xent_exact(x, w, less, top)[3] != dw).any(1).sum() > 80
