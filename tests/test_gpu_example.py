"""The example that trains on the fused operators and serves with 4-bit weights."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_gated_lm_learns_and_serves():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_lm
    losses, right = gated_lm.main(["--vocab", "1000", "--width", "128", "--hidden", "256", "--tokens", "1024",
                                   "--steps", "150"])
    assert all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(1000)) < 2.0  # nothing learnt yet
    assert losses[-1] < 0.5 and right > 0.9
