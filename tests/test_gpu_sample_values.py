"""Sampling from rows with more logits of one value than 16 bits count, where
the value is an infinity: its count's neighbour is a NaN's; and at a border that
the last bits of the shares' sums decide."""
import math
import os
import sys
from decimal import Decimal, localcontext

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import serve_reference as ref  # noqa: E402
from test_gpu_fused import TYPES, pg, randn  # noqa: E402,F401
from test_gpu_serve import equal  # noqa: E402
from test_gpu_serve_edges import sampled  # noqa: E402

pytestmark = pytest.mark.gpu
FMT = ["f16", "bf16"]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("V", [65535, 65536, 70000, 131072, 200001])
def test_infinite_logits(pg, fmt, V):
    # alone, they share the probability evenly; beside finite ones they have all of it
    gen = torch.Generator().manual_seed(V)
    M = 6
    u = torch.rand(M, generator=gen)
    z = torch.full((M, V), math.inf)
    assert sampled(pg, fmt, z, u).tolist() == [int(x) for x in (u.double() * V).floor()]
    k = torch.full((M,), 3, dtype=torch.int32)
    assert sampled(pg, fmt, z, u, top_k=k).tolist() == [int(x) for x in (u.double() * 3).floor()]
    z = torch.cat([z, randn(gen, M, 999, scale=2.0)], 1)[:, torch.randperm(V + 999, generator=gen)].contiguous()
    for kw in ({}, dict(temperature=torch.full((M,), math.inf)), dict(top_p=torch.full((M,), 0.3)), dict(top_k=k), dict(min_p=torch.full((M,), 0.5))):
        equal(str(list(kw)), sampled(pg, fmt, z, u, **kw), ref.sample(z.to(TYPES[fmt]), u, **kw))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("where", [0, 40000, 139999])
@pytest.mark.parametrize("value", [math.inf, 3.0, -math.inf])
def test_nan_among_many_equal_logits(pg, fmt, where, value):
    # the row has no token, whatever its counts did; nor does one of nothing but NaN
    z = torch.full((3, 140000), value)
    z[0, where] = math.nan
    z[1, where] = -math.nan
    z[2] = math.nan
    assert sampled(pg, fmt, z, torch.full((3,), 0.4)).tolist() == [-1, -1, -1]


@pytest.mark.parametrize("fmt,first,temperature", [("bf16", 1 + 127 / 128, "0x1.828e4cp-1"), ("f16", 1 + 127 / 1024, "0x1.828e4cp-4")])
def test_a_border_between_two_values(pg, fmt, first, temperature):
    # 15014 logits of the largest value, and 55877 of 1, the last of the 64 values that are summed as powers of one
    # exponential: half of all shares is more than the first ones have, by 2^-43.6 of it.  The 63rd power of an exponential
    # that is off by 2^-52, and 64 roundings of 2^-53, are 2^-45.4
    a, b, T = 15014, 55877, float.fromhex(temperature)
    with localcontext() as c:
        c.prec = 50
        over = Decimal(b) * ((Decimal(1) - Decimal(first)) / Decimal(T)).exp() / a - 1
        assert Decimal(2) ** Decimal("-43.7") < over < Decimal(2) ** Decimal("-43.6")
    z = torch.cat([torch.full((a,), first), torch.full((b,), 1.0)]).repeat(2, 1)
    z[1] = z[1].flip(0)
    got = sampled(pg, fmt, z, torch.tensor([0.5, 0.5]), temperature=torch.tensor([T, T]))
    assert got.tolist() == [a, 0]
