"""The sampling's settings and random numbers are tensors: other values are
refused by name, before anything else is looked at (CPU only)."""
import pytest

torch = pytest.importorskip("torch")
from software_pipelined_tiled_pipeline_amd import pgemm  # noqa: E402


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("key,value", [("temperature", 0.7), ("temperature", 0), ("top_k", 50), ("top_p", 0.9), ("min_p", False),
                                       ("min_p", [0.1, 0.2]), ("u", 0.5), ("u", None)])
def test_plain_values_are_refused_by_name(fmt, key, value):
    z = torch.zeros(2, 16, dtype=torch.float16 if fmt == "f16" else torch.bfloat16)
    call = dict(u=torch.zeros(2))
    call[key] = value
    with pytest.raises(ValueError, match=f"{key} must be a tensor"):
        getattr(pgemm, f"pgemm_{fmt}_sample")(z, **call)
