"""4-bit products whose fp32 sums are exact in any order: every weight, scale and
zero point shows, however long the row is.

x is -1, 0 or 1 and scales are 1, 2 or 4, so that all partial sums are integers
below 2^24 (at most K (16 + 15) 4 on the way, which bounds K at 2^17); the result
then is the exact value rounded once."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fused_reference as ref  # noqa: E402
from test_gpu_fused import TYPES, call, pg  # noqa: E402,F401

# one stretch of scales and several, in every arrangement of waves; groups that
# do not divide a block of 128 or a stretch; rows that end inside a group
SIZES = [(M, N, K, group) for M, N in ((1, 40), (3, 40), (4, 8200), (5, 70), (16, 70), (33, 50)) for K, group in
         ((40000, 32), (33000, 96), (20000, 64), (8200, 32))] + [
    (24, 16420, 4500, 32), (48, 16400, 4500, 64), (64, 16500, 4500, 32), (2, 33, 70000, 128), (33, 40, 40000, 16384)]


def exact_case(seed, fmt, M, N, K, group):
    gen = torch.Generator().manual_seed(seed)
    groups = -(-K // group)
    x = torch.randint(-1, 2, (M, K), generator=gen).to(TYPES[fmt])
    values = torch.randint(0, 16, (N, K), generator=gen, dtype=torch.uint8)
    scale = (2.0 ** torch.randint(0, 3, (N, groups), generator=gen)).to(TYPES[fmt])
    zero = torch.randint(0, 16, (N, groups), generator=gen, dtype=torch.uint8)
    assert K * 31 * 4 < 1 << 24
    return x, values, scale, zero


def rounded(x, values, scale, zero, group):
    y = x.double() @ ref.weights(values, scale, zero, group).t()
    return y.float().to(x.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,group", SIZES)
def test_exact_sums(pg, fmt, M, N, K, group):
    x, values, scale, zero = (t.cuda() for t in exact_case(M + N + K, fmt, M, N, K, group))
    packed = pg.pack_q4(values)
    for z in (zero, None):
        got = call(pg, fmt, "q4", x, packed, scale, z, group=group)
        assert torch.equal(got, rounded(x, values, scale, z, group))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("K,group", [(40000, 32), (20000, 96), (4500, 64), (2500, 4096)])
def test_one_weight_at_a_time(pg, fmt, K, group):
    # a token for each of the places where something begins or ends
    edges = sorted({k + d for k in (0, group, 128, 32 * 128, 64 * 128, 16 * 128, 2 * 64 * 128, K - 32, K) for d in (-1, 0)
                    if 0 <= k + d < K})
    _, values, scale, zero = exact_case(K, fmt, 1, 70, K, group)
    x = torch.zeros(len(edges), K, dtype=TYPES[fmt])
    x[torch.arange(len(edges)), edges] = 1
    want = ref.weights(values, scale, zero, group)[:, edges].t().to(x.dtype)
    packed = pg.pack_q4(values).cuda()
    for rows in (slice(0, 1), slice(0, 4), slice(0, None)):
        got = call(pg, fmt, "q4", x[rows].cuda(), packed, scale.cuda(), zero.cuda(), group=group)
        assert torch.equal(got.cpu(), want[rows])


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_the_comparison_finds_planted_faults(fmt):
    M, N, K, group = 3, 40, 40000, 32
    x, values, scale, zero = exact_case(1, fmt, M, N, K, group)
    want = rounded(x, values, scale, zero, group)

    def seen(*planted):
        return float((rounded(*planted, group) != want).float().mean())
    at = 64 * 128 // group  # the first group of a second stretch of scales
    dropped = x.clone()
    dropped[:, at * group:(at + 1) * group] = 0
    assert seen(dropped, values, scale, zero) > 0.5
    tail = x.clone()
    tail[:, -8:] = 0
    assert seen(tail, values, scale, zero) > 0.2
    for change in (0.5, 2.0):
        other = scale.clone()
        other[:, at] *= change
        assert seen(x, values, other, zero) > 0.3
    shifted = scale.clone()
    shifted[:, 1:] = scale[:, :-1]
    assert seen(x, values, shifted, zero) > 0.9
    moved = zero.clone()
    moved[:, at] ^= 1
    assert seen(x, values, scale, moved) > 0.1
