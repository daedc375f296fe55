"""The serving operators on the GPU against 64-bit references
(tests/serve_reference.py): whole numbers equal, others element by element
within derived bounds."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import serve_reference as ref  # noqa: E402
from test_gpu_fused import TYPES, call, check, pg, randn  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def equal(what, got, want):
    assert got.dtype == want.dtype and got.shape == want.shape, what
    bad = got != want.to(got.device)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {[int(i) for i in bad.nonzero()[0]]}"


# one row and more than a grid has, a value, rows of every alignment, each of the kernels' lengths and past them
QUANT = [(1, 1), (1, 4096), (3, 7), (5, 16), (2, 1000), (33, 1025), (4, 4097), (2, 8200), (1, 20001), (70000, 24)]


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", QUANT)
def test_quant(pg, fmt, M, K):
    gen = torch.Generator().manual_seed(M + K)
    x = (randn(gen, M, K) * torch.exp(randn(gen, K))).to(TYPES[fmt]).cuda()
    q, scale = call(pg, fmt, "quant_i8", x)
    want, ws = ref.quant(x)
    assert torch.equal(scale, ws)
    equal("q", q, want)


def i8_case(seed, fmt, M, N, K, gated):
    gen = torch.Generator().manual_seed(seed)
    rows = 2 * N if gated else N
    x = randn(gen, M, K).to(TYPES[fmt]).cuda()
    w = torch.randint(-128, 128, (rows, ref.width(K)), generator=gen).to(torch.int8)
    w[:, K:] = 0
    ws = (torch.rand(rows, generator=gen) + 0.5) * (K ** -0.5 / 74)
    return x, w.cuda(), ws.cuda()


# few tokens: as many as make their own integers and more, each count of token blocks, odd rows; blocks of 256 bytes of K
# with and without a rest; many tokens: small and large tiles, pieces of K
I8 = [(1, 1, 1), (1, 33, 16), (2, 17, 100), (4, 300, 257), (4, 64, 8192), (3, 40, 8208), (5, 100, 1000), (16, 48, 512),
      (17, 130, 700), (32, 64, 4096), (33, 65, 31), (64, 200, 1300), (1, 20000, 64), (65, 33, 40), (128, 128, 1024),
      (200, 260, 2049), (130, 100, 16384), (700, 2100, 130), (2100, 3000, 264)]


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", I8)
def test_i8(pg, fmt, M, N, K):
    x, w, ws = i8_case(M + N + K, fmt, M, N, K, False)
    q, xs = ref.quant(x)
    want = ref.i8(q, xs, w, ws, TYPES[fmt])
    given = call(pg, fmt, "i8", q, w, ws, xs=xs)
    check("integers", given, want)
    assert torch.equal(call(pg, fmt, "i8", x, w, ws), given)  # the same integers


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,F,K", I8)
def test_i8_gated(pg, fmt, act, M, F, K):
    x, w, ws = i8_case(M * F + K, fmt, M, F, K, True)
    q, xs = ref.quant(x)
    want = ref.i8(q, xs, w, ws, TYPES[fmt], act)
    given = call(pg, fmt, "i8_gated", q, w, ws, xs=xs, act=act)
    check("integers", given, want)
    assert torch.equal(call(pg, fmt, "i8_gated", x, w, ws, act=act), given)


# M, D, F, E, k: one token and one expert, widths below eight, rows of odd widths; fewer choices than experts and more;
# each count of token blocks, more than one for an expert; two chunks of tokens, the last one short
MOE = [(1, 1, 1, 1, 1), (1, 8, 8, 4, 2), (2, 5, 3, 3, 3), (3, 70, 33, 5, 2), (1, 1024, 512, 8, 2), (7, 130, 257, 60, 4),
       (16, 256, 128, 100, 8), (37, 205, 101, 6, 2), (64, 64, 40, 3, 1), (64, 128, 96, 2, 2), (65, 96, 72, 16, 4),
       (130, 40, 24, 4, 1), (66, 64, 32, 200, 1), (20, 33, 20, 1024, 32), (5, 2050, 1001, 3, 1)]


def moe_case(seed, fmt, M, D, F, E, spread=1.5):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[fmt]
    return (randn(gen, M, D).to(t).cuda(), randn(gen, E, D, scale=spread * D ** -0.5).to(t).cuda(),
            randn(gen, E, 2 * F, D, scale=D ** -0.5).to(t).cuda(), randn(gen, E, D, F, scale=2 * F ** -0.5).to(t).cuda())


def check_moe(got, want):
    equal("experts", got[1], want[1])
    check("weights", got[2], want[2])
    check("y", got[0], want[0])


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("act,normalize", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("M,D,F,E,k", MOE)
def test_moe(pg, fmt, act, normalize, M, D, F, E, k):
    ops = moe_case(M + D + F + E, fmt, M, D, F, E)
    got = call(pg, fmt, "moe", *ops, k, act=act, normalize=normalize, routing=True)
    check_moe(got, ref.moe(*ops, k, act, normalize))
    assert torch.equal(call(pg, fmt, "moe", *ops, k, act=act, normalize=normalize), got[0])


def settings(gen, M):
    off = torch.rand(4, M, generator=gen) < 0.3
    t = (torch.rand(M, generator=gen) * 1.5 + 0.1).masked_fill_(torch.rand(M, generator=gen) < 0.1, 0.0)
    k = torch.randint(1, 60, (M,), generator=gen, dtype=torch.int32).masked_fill_(off[1], 0)
    p = (torch.rand(M, generator=gen) * 0.9 + 0.1).masked_fill_(off[2], 1.0)
    q = (torch.rand(M, generator=gen) * 0.2).masked_fill_(off[3], 0.0)
    return t, k, p, q


def on_gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("M,V", [(1, 1), (5, 2), (64, 7), (40, 1000), (20, 8193), (9, 50021), (3, 200000)])
@pytest.mark.parametrize("scale", [0.02, 2.5, 40.0])
def test_sample(pg, fmt, M, V, scale):
    gen = torch.Generator().manual_seed(M + V)
    z = randn(gen, M, V, scale=scale).to(TYPES[fmt])
    u = torch.rand(M, generator=gen)
    for some in ((None,) * 4, settings(gen, M)):
        got = call(pg, fmt, "sample", z.cuda(), u.cuda(), *on_gpu(*some))
        equal("token", got.cpu(), ref.sample(z, u, *some))
