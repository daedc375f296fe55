"""The fused operators on the GPU against 64-bit references, element by
element within derived bounds (tests/fused_reference.py)."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fused_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from software_pipelined_tiled_pipeline_amd import pgemm
    pgemm.lib()
    return pgemm


def call(pg, fmt, name, *args, **more):
    return getattr(pg, f"pgemm_{fmt}_{name}")(*args, **more)


def randn(gen, *shape, scale=1.0):
    return torch.randn(shape, generator=gen, dtype=torch.float32).mul_(scale)


def check(what, got, want):
    value, bound = want
    got = got.double()
    assert got.shape == value.shape, what
    off = (got - value).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} elements outside the bound, worst "
                           f"{float((off / bound.clamp(min=1e-300))[bad].max()):.3g} times it, first at "
                           f"{[int(i) for i in bad.nonzero()[0]]}")


def block(seed, fmt, M, F, D):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[fmt]
    return (randn(gen, M, D).to(t).cuda(), randn(gen, 2 * F, D, scale=max(D, 1) ** -0.5).to(t).cuda(),
            randn(gen, M, F, scale=0.1).to(t).cuda())


# one row, tile edges on either side, odd widths and hidden sizes, one K tile
# and several, large tiles for each of the products
GATED = [(1, 1, 1), (1, 8, 8), (3, 5, 7), (64, 64, 64), (65, 33, 70), (128, 64, 128), (129, 65, 136), (300, 260, 200),
         (257, 127, 1001), (512, 1000, 192), (1000, 771, 129), (2100, 3000, 130), (3200, 40, 4100), (130, 1600, 4104)]


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,F,D", GATED)
def test_gated(pg, fmt, act, M, F, D):
    x, w, dh = block(M + F + D, fmt, M, F, D)
    want = ref.gated(x, w, act, dh)
    check("h", call(pg, fmt, "gated", x, w, act=act), want["h"])
    h, saved = call(pg, fmt, "gated", x, w, act=act, save=True)
    check("h (saved)", h, want["h"])
    for keep in (saved, None):
        dx, dw = call(pg, fmt, "gated_bwd", dh, x, w, saved=keep, act=act)
        check("dx", dx, want["dx"])
        check("dw", dw, want["dw"])


# (4100, 66000, 40): the derivative by the logits takes two pieces
XENT = [(1, 1, 1), (1, 7, 5), (3, 128, 64), (65, 1000, 72), (130, 257, 136), (200, 3001, 129), (700, 20000, 64),
        (2049, 6200, 130), (4100, 66000, 40)]


def head(seed, fmt, M, V, D):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[fmt]
    x, w = randn(gen, M, D).to(t).cuda(), randn(gen, V, D, scale=2 * D ** -0.5).to(t).cuda()
    target = torch.randint(0, V, (M,), generator=gen)
    target[torch.rand(M, generator=gen) < 0.2] = -100
    return x, w, target.cuda(), (torch.rand(M, generator=gen) + 0.1).cuda()


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("M,V,D", XENT)
def test_xent(pg, fmt, M, V, D):
    x, w, target, dloss = head(M + V + D, fmt, M, V, D)
    want = ref.xent(x, w, target, dloss=dloss)
    loss, lse = call(pg, fmt, "xent", x, w, target)
    check("lse", lse, want["lse"])
    check("loss", loss, want["loss"])
    dx, dw = call(pg, fmt, "xent_bwd", dloss, x, w, target, lse)
    check("dx", dx, want["dx"])
    check("dw", dw, want["dw"])


# one token and as many as a launch takes at once and more, tails of a block of
# 128 and of 32 along K, groups finer and coarser than a block, no whole group
Q4 = [(1, 16, 128, 128), (1, 33, 64, 32), (2, 17, 1, 32), (16, 100, 1000, 64), (17, 300, 500, 96), (33, 64, 257, 160),
      (64, 130, 4096, 128), (70, 50, 1024, 256), (5, 4100, 640, 32), (13, 48, 2500, 4096)]


def q4_case(seed, fmt, M, N, K, group, zeros):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[fmt]
    groups = -(-K // group)
    x = randn(gen, M, K).to(t).cuda()
    values = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8).cuda()
    scale = (randn(gen, N, groups).abs() * 0.05 + 0.01).to(t).cuda()
    zero = torch.randint(0, 16, (N, groups), generator=gen, dtype=torch.uint8).cuda() if zeros else None
    return x, values, scale, zero


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", Q4)
def test_q4(pg, fmt, zeros, M, N, K, group):
    x, values, scale, zero = q4_case(M + N + K, fmt, M, N, K, group, zeros)
    y = call(pg, fmt, "q4", x, pg.pack_q4(values), scale, zero, group=group)
    check("y", y, ref.q4(x, values, scale, zero, group))


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("act,zeros", [("silu", True), ("gelu", False)])
@pytest.mark.parametrize("M,F,K,group", Q4)
def test_q4_gated(pg, fmt, act, zeros, M, F, K, group):
    x, values, scale, zero = q4_case(M * F + K, fmt, M, 2 * F, K, group, zeros)
    y = call(pg, fmt, "q4_gated", x, pg.pack_q4(values), scale, zero, group=group, act=act)
    check("h", y, ref.q4(x, values, scale, zero, group, act=act))
