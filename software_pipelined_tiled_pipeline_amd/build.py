"""Builds libpgemm.so (HIP, gfx950 only) in-tree with hipcc.

The library is twelve translation units: the C ABI of the products (argument
checks, planning, the int32 kernel), four units of NT kernel instances (f16
and bf16, each with the direct-to-LDS and the register-staged loader), the C
ABI of the fused operators, and their instances by operator and type.  They
are compiled in parallel and linked into one shared library.

Beside it, _binding.so: the fused operators' short way through Python, host C++
against torch's headers.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
UNITS = ["pgemm_api.hip", "inst_f16_direct.hip", "inst_f16_staged.hip", "inst_bf16_direct.hip",
         "inst_bf16_staged.hip", "fused_api.hip", "fused_gated_f16.hip", "fused_gated_bf16.hip", "fused_xent_f16.hip",
         "fused_xent_bf16.hip", "fused_q4_f16.hip", "fused_q4_bf16.hip"]
LIB = os.path.join(HERE, "libpgemm.so")
BINDING = os.path.join(HERE, "_binding.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # packed fp32 instructions are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]
_NOISE = "packed-fp32-ops"


def hipcc() -> str:
    return os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def _run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    msgs = [l for l in (res.stdout + res.stderr).splitlines() if _NOISE not in l and l.strip()]
    if res.returncode != 0:
        raise RuntimeError("hipcc failed: " + " ".join(cmd) + "\n" + "\n".join(msgs))
    return msgs


def build_binding(out: str = BINDING) -> str:
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-attributes",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include"),
           "-I", sysconfig.get_paths()["include"]]
    for path in cpp_extension.include_paths():
        cmd += ["-isystem", path]
    cmd += [os.path.join(CSRC, "binding.cpp"), "-o", out + ".tmp"]
    for path in cpp_extension.library_paths():
        cmd += ["-L", path]
    _run(cmd + ["-ltorch_python", "-ltorch_cpu", "-lc10"])
    os.replace(out + ".tmp", out)
    return out


def build(verbose: bool = False, lib: str = LIB, extra_flags=(), jobs: int = 0) -> str:
    """Compiles every unit (in parallel) and links libpgemm.so."""
    jobs = jobs or min(len(UNITS), os.cpu_count() or 1)
    with tempfile.TemporaryDirectory(prefix="pgemm_build_") as tmp:
        objs = [os.path.join(tmp, u.replace(".hip", ".o")) for u in UNITS]

        def compile_one(i):
            return _run([hipcc(), *HIPCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, UNITS[i]), "-o", objs[i]])

        with ThreadPoolExecutor(jobs) as pool:
            binding = pool.submit(build_binding) if lib == LIB else None
            msgs = [m for ms in pool.map(compile_one, range(len(UNITS))) for m in ms]
            if binding:
                binding.result()
        out = lib + ".tmp"
        msgs += _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", out])
        if verbose and msgs:
            print("\n".join(msgs), file=sys.stderr)
        os.replace(out, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
