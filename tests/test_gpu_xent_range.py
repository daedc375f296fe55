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
