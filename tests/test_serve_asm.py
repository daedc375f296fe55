"""Hazards in the serving operators' kernels that the compiler does not check
for (CPU only: hipcc cross-compiles); see test_fused_asm.py.  Their tiled 8-bit
products are the fused kernels with another MFMA, written as inline assembly."""
import os
import re
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import mfma_hazards  # noqa: E402
from test_fused_asm import kernels, lds_load_faults  # noqa: E402
from test_mfma_hazards import device_asm, hipcc_available  # noqa: E402

from software_pipelined_tiled_pipeline_amd import build  # noqa: E402

UNITS = [u for u in build.UNITS if u.startswith(("serve_i8", "serve_moe"))]
TILED = [u for u in UNITS if u.startswith("serve_i8")]


@pytest.fixture(scope="module")
def unit_asm():
    if not hipcc_available():
        pytest.skip("hipcc not available")
    with tempfile.TemporaryDirectory() as tmp:
        def one(u):
            return u, device_asm(os.path.join(build.CSRC, u), os.path.join(tmp, u + ".s"))
        with ThreadPoolExecutor(len(UNITS)) as pool:
            return dict(pool.map(one, UNITS))


@pytest.mark.parametrize("unit", UNITS)
def test_operands_of_mfmas(unit_asm, unit):
    hazards, mfmas = mfma_hazards.check_asm(unit_asm[unit])
    assert mfmas > 200
    hazards = [h for h in hazards if h.kind in ("VALU_TO_MFMA", "LOAD_TO_MFMA")]
    assert not hazards, "\n".join(f"{h.kind} line {h.line}: {h.text} ({h.detail})" for h in hazards[:20])


@pytest.mark.parametrize("unit", TILED)
def test_tiled_products(unit_asm, unit):
    hazards, _ = mfma_hazards.check_asm(unit_asm[unit])
    hazards = [h for h in hazards if "fused_kernel" in h.function]
    assert not hazards, "\n".join(f"{h.kind} line {h.line}: {h.text} ({h.detail})" for h in hazards[:20])
    seen = 0
    for name, body in kernels(unit_asm[unit]):
        faults, loads = lds_load_faults(body)
        assert not faults and loads >= 8, name + "\n" + "\n".join(faults[:10])
        assert "v_mfma_i32_16x16x64_i8" in body and "v_mfma_f32" not in body, name
        for block in re.split(r"\n(?=\.LBB)", body):
            # a spilled accumulator would be read without an MFMA's wait states
            if block.count("v_mfma") >= 8:
                assert "scratch_" not in block, name
        seen += 1
    assert seen == 9  # plain, gated and in pieces: large tiles, small ones with two and four slots
