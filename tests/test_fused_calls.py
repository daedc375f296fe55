"""Integers that the fused operators' binding takes, without a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
from software_pipelined_tiled_pipeline_amd import fused, pgemm  # noqa: E402


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("name", ["q4", "q4_gated"])
@pytest.mark.parametrize("group", [0, -32, 48, 1 << 31, (1 << 64) + 32, -(1 << 64) + 32])
def test_group(fmt, name, group):
    # 2^64 + 32 would reach the library as 32, and have it read scales that one group a row does not have
    assert ctypes.c_int64((1 << 64) + 32).value == 32
    x, q, s = torch.zeros(2, 64), torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="group"):
        getattr(pgemm, f"pgemm_{fmt}_{name}")(x, q, s, group=group)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("index", [1 << 63, (1 << 64) + 5, -(1 << 63) - 1])
def test_ignore_index(fmt, index):
    x, w, t, f = torch.zeros(2, 8), torch.zeros(4, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    with pytest.raises(ValueError, match="ignore_index"):
        getattr(pgemm, f"pgemm_{fmt}_xent")(x, w, t, ignore_index=index)
    with pytest.raises(ValueError, match="ignore_index"):
        getattr(pgemm, f"pgemm_{fmt}_xent_bwd")(f, x, w, t, f, ignore_index=index)


def test_ignore_index_of_64_bits():
    for index in (-100, (1 << 63) - 1, -(1 << 63)):
        assert fused._ignored(index) == index
