"""4-bit products of values that fp32 sums do not forgive: infinities, and
values whose sums leave fp32 where the result does not."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fused_reference as ref  # noqa: E402
from test_gpu_fused import call, check, pg, q4_case  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# tokens and rows of every arrangement of waves, short rows, ends of groups and blocks
SIZES = [(1, 70, 1024, 128), (3, 50, 5, 32), (4, 70, 1000, 32), (13, 130, 260, 64), (33, 48, 2500, 96), (24, 16420, 200, 32),
         (48, 16400, 300, 64), (64, 16500, 130, 128)]


def definition(x, values, scale, zero, group):
    """The definition in 64 bits where x is not finite: group by group, an infinity times a weight of zero being NaN."""
    K = x.shape[1]
    y = torch.zeros(x.shape[0], values.shape[0], dtype=torch.float64, device=x.device)
    for g in range(scale.shape[1]):
        at = slice(g * group, min(K, (g + 1) * group))
        z = 8.0 if zero is None else zero[:, g:g + 1].double()
        w = values[:, at].double() - z
        y += (x[:, None, at].double() * w[None]).sum(2) * scale[:, g].double()
    return y


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", SIZES)
def test_infinite_activations(pg, fmt, zeros, M, N, K, group):
    x, values, scale, zero = q4_case(M + N + K, fmt, M, N, K, group, zeros)
    scale[::3] *= -1
    packed = pg.pack_q4(values)
    clean = ref.q4(x, values, scale, zero, group)
    for places in ([0], [K - 1], [K // 2], [0, K - 1]):
        y, row = x.clone(), M // 2
        for i, k in enumerate(places):
            y[row, k] = math.inf if i == 0 else -math.inf
        got = call(pg, fmt, "q4", y, packed, scale, zero, group=group)
        rest = torch.arange(M, device="cuda") != row
        check("y", got[rest], (clean[0][rest], clean[1][rest]))
        want = definition(y[row:row + 1], values, scale, zero, group)[0]
        assert not want.isfinite().any() and (N < 48 or want.isinf().any())
        assert torch.equal(got[row].isnan(), want.isnan())
        inf = want.isinf()
        assert torch.equal(got[row][inf].double(), want[inf])


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("M,F,K,group", SIZES[:6])
def test_infinite_activations_of_the_gated_block(pg, fmt, M, F, K, group):
    x, values, scale, zero = q4_case(M + F + K, fmt, M, 2 * F, K, group, True)
    packed = pg.pack_q4(values)
    row = M // 2
    x[row, K - 1] = math.inf
    got = call(pg, fmt, "q4_gated", x, packed, scale, zero, group=group, act="gelu")[row]
    y = definition(x[row:row + 1], values, scale, zero, group)[0]
    g, u = y[:F], y[F:]
    want = torch.where(g > 0, g, torch.full_like(g, math.nan)) * u  # gelu of minus infinity: 0 times infinity
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[want.isinf()].double(), want[want.isinf()])


@pytest.mark.parametrize("M,N,K,group", SIZES)
def test_sums_that_leave_fp32_early(pg, M, N, K, group):
    # 2e37 times 16 + 15 is past fp32's end, 2e37 times a weight less its zero point is not
    x, values, scale, zero = q4_case(M + N + K, "bf16", M, N, K, group, True)
    x = torch.zeros_like(x)
    row = M // 2
    x[row, K - 1] = 2e37
    got = pg.pgemm_bf16_q4(x, pg.pack_q4(values), scale, zero, group=group)
    want = definition(x, values, scale, zero, group)
    check("y", got, (want, (ref.half_step(x.dtype) + 4 * ref.U32) * want.abs()))
