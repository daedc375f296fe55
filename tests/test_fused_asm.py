"""Hazards in the fused kernels that the compiler does not check for (CPU
only: hipcc cross-compiles).

The tiled kernels write their MFMAs, and those with transposing reads their
direct-to-LDS loads too, as inline assembly: wait states around the MFMAs, the
LDS address in M0 and scalar registers that a vector instruction wrote are
theirs to mind.  These tests read the assembly that the library's own flags
give for every unit of fused kernels.
"""
import os
import re
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import mfma_hazards  # noqa: E402
from test_mfma_hazards import device_asm, hipcc_available  # noqa: E402

from software_pipelined_tiled_pipeline_amd import build  # noqa: E402

UNITS = [u for u in build.UNITS if u.startswith(("fused_gated", "fused_xent"))]
ALL = UNITS + [u for u in build.UNITS if u.startswith("fused_q4")]
SGPR_WAIT = 5  # wait states from a vector instruction's scalar result to a load that reads it


@pytest.fixture(scope="module")
def unit_asm():
    if not hipcc_available():
        pytest.skip("hipcc not available")
    with tempfile.TemporaryDirectory() as tmp:
        def one(u):
            return u, device_asm(os.path.join(build.CSRC, u), os.path.join(tmp, u + ".s"))
        with ThreadPoolExecutor(len(ALL)) as pool:
            return dict(pool.map(one, ALL))


@pytest.mark.parametrize("unit", ALL)
def test_operands_of_mfmas(unit_asm, unit):
    # the products with few rows leave their MFMAs to the compiler, which does
    # not know what an inline-assembly instruction before one writes
    hazards, mfmas = mfma_hazards.check_asm(unit_asm[unit])
    assert mfmas > 500
    hazards = [h for h in hazards if h.kind in ("VALU_TO_MFMA", "LOAD_TO_MFMA")]
    assert not hazards, "\n".join(f"{h.kind} line {h.line}: {h.text} ({h.detail})" for h in hazards[:20])


@pytest.mark.parametrize("unit", UNITS)
def test_no_mfma_hazards(unit_asm, unit):
    hazards, mfmas = mfma_hazards.check_asm(unit_asm[unit])
    assert mfmas > 500
    hazards = [h for h in hazards if "fused_kernel" in h.function]  # the others' MFMAs are the compiler's
    assert not hazards, "\n".join(f"{h.kind} line {h.line}: {h.text} ({h.detail})" for h in hazards[:20])


def kernels(asm):
    for m in re.finditer(r"^(_ZN5pgemm\S*fused_kernel\S*):.*?\n(.*?)s_endpgm", asm, re.S | re.M):
        yield m.group(1), m.group(2)


def scalars(text):
    """Scalar registers that an operand string names."""
    found = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        found.update(range(int(a), int(b) + 1))
    found.update(int(n) for n in re.findall(r"\bs(\d+)\b", text))
    return found


def lds_load_faults(body):
    """Loads into LDS whose M0 was not set for them, or that read a scalar too
    soon after a vector instruction wrote it."""
    faults, base, since, since_vector, loads = [], None, {}, 0, 0
    for line in body.splitlines():
        line = line.split(";")[0].strip()
        if not line or line.startswith(".") and not line.endswith(":"):
            continue
        if line.endswith(":") or line.startswith(("s_branch", "s_cbranch")):
            base = None  # M0 is set again in every block
            if line.endswith(":"):
                continue
        op = line.split()[0]
        states = int(line.split()[1]) + 1 if op == "s_nop" else 1
        for r in list(since):
            since[r] += states
        if re.search(r"\bm0\b", line) and op.startswith(("s_", "v_")) and re.match(r"\S+\s+m0\b", line):
            base = line
        if op.startswith("buffer_load") and line.endswith(" lds"):
            loads += 1
            if base is None:
                faults.append("M0 not set in this block: " + line)
            soon = [r for r in scalars(line) if since.get(r, SGPR_WAIT + 1) <= SGPR_WAIT]
            if soon:
                faults.append(f"s{soon} written by a vector instruction just before: {line}")
        if op.startswith("v_") and not op.startswith("v_mfma"):
            for r in scalars(line.split(",")[0]):
                since[r] = 0
        elif op.startswith("s_") and len(line.split()) > 1:
            for r in scalars(line.split(",")[0]):
                since.pop(r, None)
    return faults, loads


@pytest.mark.parametrize("unit", UNITS)
def test_loads_into_lds(unit_asm, unit):
    seen = 0
    for name, body in kernels(unit_asm[unit]):
        faults, loads = lds_load_faults(body)
        assert not faults, name + "\n" + "\n".join(faults[:10])
        assert loads >= 8, name
        seen += 1
    assert seen >= 8


@pytest.mark.parametrize("unit", UNITS)
def test_no_spills_among_mfmas(unit_asm, unit):
    # a spilled accumulator would be read without an MFMA's wait states, and
    # the memory it goes to counts among the loads that the kernel waits for
    for name, body in kernels(unit_asm[unit]):
        for block in re.split(r"\n(?=\.LBB)", body):
            if block.count("v_mfma") >= 8:
                assert "scratch_" not in block, name


Q4 = re.compile(r"^(_ZN5pgemm9q4_kernelI\S*?Lb[01]ELi(\d+)ELi\d+ELi(\d+)ELi(\d+)ELi\d+ELi\d+E\S*):.*?\n(.*?)s_endpgm", re.S | re.M)


@pytest.mark.parametrize("unit", [u for u in ALL if u.startswith("fused_q4")])
def test_loads_that_waits_count(unit_asm, unit):
    # A block's weights (two loads into LDS) are waited for by the number of
    # loads after them: each pair has its tokens' loads before it, none of
    # which the compiler may leave out where it sees no use of their values.
    kernels = 0
    for m in Q4.finditer(unit_asm[unit]):
        name, per_block = m.group(1), -(-int(m.group(3)) // int(m.group(4)))
        kinds = "".join("w" if " lds" in line else "x" for line in m.group(5).splitlines()
                        if re.match(r"\s+(global_load_dwordx4|buffer_load_dwordx4\s.*\blds)\b", line))
        assert kinds.count("w") >= 4, name
        assert kinds == ("x" * per_block + "ww") * (kinds.count("w") // 2), f"{name}: {kinds}"
        kernels += 1
    assert kernels >= 60


def test_the_check_finds_planted_faults():
    good = "\ts_mov_b32 m0, s3\n\ts_nop 0\n\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds\n"
    assert lds_load_faults(good) == ([], 1)
    assert lds_load_faults(good + ".LBB0_1:\n\tbuffer_load_dwordx4 v1, s[4:7], 0 offen offset:1024 lds\n")[0]
    assert lds_load_faults("\tv_readfirstlane_b32 s5, v0\n" + good)[0]
    assert not lds_load_faults("\tv_readfirstlane_b32 s5, v0\n\ts_nop 4\n" + good)[0]
