"""The loss's gradients where some rows' dloss is not finite."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fused_reference as ref  # noqa: E402
from test_gpu_fused import call, check, head, pg  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1e-6, 1.0, 300.0])
@pytest.mark.parametrize("poison", [math.inf, -math.inf, math.nan])
def test_a_row_that_is_not_finite_leaves_the_rest(pg, fmt, size, poison):
    M, V, D = 140, 700, 72
    x, w, target, dloss = head(50, fmt, M, V, D)
    target[7] = 3
    dloss = dloss * size
    one = dloss.clone()
    one[7] = 0
    want = ref.xent(x, w, target, dloss=one)["dx"]
    one[7] = poison
    _, lse = call(pg, fmt, "xent", x, w, target)
    dx, dw = call(pg, fmt, "xent_bwd", one, x, w, target, lse)
    rest = torch.arange(M, device="cuda") != 7
    check("dx", dx[rest], (want[0][rest], want[1][rest]))
    assert not dx[7].isfinite().any() and not dw.isfinite().any()
    # in a row that does not count it is nothing at all
    target[7] = -100
    one[7] = 0
    want = ref.xent(x, w, target, dloss=one)
    one[7] = poison
    dx, dw = call(pg, fmt, "xent_bwd", one, x, w, target, lse)
    check("dx", dx, want["dx"])
    check("dw", dw, want["dw"])


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_no_gradient_where_dloss_is_zero(pg, fmt):
    # whatever the row's target is; its loss says that it is none of the vocabulary's
    M, V, D = 130, 500, 64
    x, w, target, dloss = head(52, fmt, M, V, D)
    dloss[17], dloss[18] = 0.0, -0.0
    want = None
    for wrong in (3, -1, V, 1 << 40):
        target[17:19] = wrong
        loss, lse = call(pg, fmt, "xent", x, w, target)
        assert loss[17:19].isnan().all() == (wrong != 3) and loss.isnan().sum() == (0 if wrong == 3 else 2)
        got = call(pg, fmt, "xent_bwd", dloss, x, w, target, lse)
        assert not got[0][17:19].any()
        want = want or got
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_rows_than_one_join_of_a_dispatch(pg):
    # 2^26 rows and a few: some of them in every turn of the statistics' join
    M, V, D = (1 << 26) + 5, 10, 8
    gen = torch.Generator(device="cuda").manual_seed(51)
    x = torch.randn(M, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(V, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    target = torch.randint(0, V, (M,), generator=gen, device="cuda")
    rows = torch.cat([torch.arange(20), (1 << 24) + torch.arange(-20, 20), torch.randint(0, M, (2000,)),
                      (1 << 26) + torch.arange(-20, 5)]).cuda()
    one = torch.ones((), device="cuda")
    want = ref.xent(x[rows], w, target[rows], dloss=one)
    loss, lse = pg.pgemm_bf16_xent(x, w, target)
    check("lse", lse[rows], want["lse"])
    check("loss", loss[rows], want["loss"])
    dx, dw = pg.pgemm_bf16_xent_bwd(one, x, w, target, lse)
    check("dx", dx[rows], want["dx"])
    assert dw.isfinite().all()
    del x, target, loss, lse, dx
    pg.release_workspace()
    torch.cuda.empty_cache()
