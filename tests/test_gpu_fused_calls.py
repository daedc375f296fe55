"""How the fused operators' Python calls take their arguments, the same on the
short way and beside it."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_fused import block, call, pg  # noqa: E402,F401

pytestmark = pytest.mark.gpu


class Undecided:
    def __bool__(self):
        raise ArithmeticError("neither")


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("M", [2, 70])
def test_save_is_taken_for_its_truth(pg, fmt, M):
    import numpy
    x, w, _ = block(60, fmt, M, 40, 72)
    h, saved = call(pg, fmt, "gated", x, w, save=True)
    for own in (None, torch.empty_like(h)):  # with an output of one's own a call leaves the short way
        for yes in (True, 1, "yes", [0], numpy.bool_(True), torch.ones(1)):
            got = call(pg, fmt, "gated", x, w, out=own, save=yes)
            assert isinstance(got, tuple) and torch.equal(got[0], h) and got[1].shape == saved.shape
        for no in (False, 0, "", [], None, numpy.bool_(False), torch.zeros(1)):
            got = call(pg, fmt, "gated", x, w, out=own, save=no)
            assert isinstance(got, torch.Tensor) and got.shape == h.shape
        with pytest.raises(ArithmeticError):
            call(pg, fmt, "gated", x, w, out=own, save=Undecided())
