"""Python binding of the serving operators (argument marshalling only).

Reached through :mod:`pgemm`, next to the fused operators, whose manner they
share (tensors on the current GPU, a ``stream`` of the caller's, workspaces that
are torch tensors registered on the call's stream, no autograd graph):
``pgemm_{f16,bf16}_quant_i8``, ``_i8`` and ``_i8_gated``, ``_moe``, ``_sample``.
"""
from __future__ import annotations

import ctypes
import functools

from . import fused
from .fused import _act, _first, _on, _out, _place, _recording, _rows, _run, _want

SETTINGS = {"temperature": 1, "top_k": 2, "top_p": 4, "min_p": 8}
MAX_TOP_K = 32
SERVE_SYMBOLS = tuple(f"pgemm_{t}_{op}" for t in ("f16", "bf16") for op in ("quant_i8", "i8", "i8_gated", "moe", "sample"))


def declare(L) -> None:
    """Argument types of the serving entry points of the loaded library."""
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    args = {
        "quant_i8": [P, P, P, I64, I64, P],
        "i8": [P, P, P, P, P, I64, I64, I64, P],
        "i8_gated": [P, P, P, P, P, I64, I64, I64, I, P],
        "moe": [P, P, P, P, P, P, P, I64, I64, I64, I64, I64, I, I, P],
        "sample": [P, P, P, P, P, P, I, P, I64, I64, P],
    }
    for name in SERVE_SYMBOLS:
        f = getattr(L, name)
        f.argtypes = args[name.split("_", 2)[2]]
        f.restype = I
    L.pgemm_i8_workspace.argtypes = [I64, I64, I64, I, I, ctypes.POINTER(I64)]
    L.pgemm_i8_workspace.restype = I
    L.pgemm_moe_workspace.argtypes = [I64, I64, I64, I64, I64, ctypes.POINTER(I64)]
    L.pgemm_moe_workspace.restype = I


def _bytes_of(name, *sizes):
    fused._load()
    pgemm, n = fused.pgemm, ctypes.c_int64()
    pgemm._check(getattr(pgemm.lib(), name)(*sizes, ctypes.byref(n)), name)
    return n.value


@functools.lru_cache(maxsize=1024)
def i8_workspace_bytes(M: int, N: int, K: int, gated: bool, quantized: bool) -> int:
    """Bytes of workspace of an 8-bit product."""
    return _bytes_of("pgemm_i8_workspace", M, N, K, int(gated), int(quantized))


@functools.lru_cache(maxsize=1024)
def moe_workspace_bytes(M: int, E: int, D: int, F: int, top_k: int) -> int:
    """Bytes of workspace of a mixture-of-experts layer."""
    return _bytes_of("pgemm_moe_workspace", M, E, D, F, top_k)


def _address(name):
    return fused._addresses.get(name) or fused._address(name)


def _three(name, t, dtype, shape, dev):
    """Checks a tensor with a size of None where any will do; its shape."""
    if (t.dtype is not dtype or t.get_device() != dev or t.dim() != len(shape) or not t.is_contiguous()
            or any(w is not None and n != w for n, w in zip(t.shape, shape))):
        fused._refuse(name, t, dtype, shape)
    return t.shape


def _make(fmt, dtype_name):
    def name(op):
        return f"pgemm_{fmt}_{op}"

    code_of = {"f16": 0, "bf16": 1}[fmt]
    QUANT, I8, I8_GATED, MOE, SAMPLE = map(name, ("quant_i8", "i8", "i8_gated", "moe", "sample"))

    def quant_i8(x, q=None, scale=None, stream=None):
        if stream is not None:
            return _on(stream, quant_i8, x, q, scale)
        address = _address(QUANT)
        if q is None and scale is None:
            dev, handle = _place()
            both = fused._binding.quant_i8(address, dev, handle, code_of, x)
            if both is not None:
                return both
        torch = fused.torch
        M, K, dev = _first("x", x, getattr(torch, dtype_name))
        q = _out("q", q, torch.int8, (M, -(-K // 16) * 16), dev, x)
        scale = _out("scale", scale, torch.float32, (M,), dev, x)
        _run(QUANT, dev, (x.data_ptr(), q.data_ptr(), scale.data_ptr(), M, K), 0)
        return q, scale

    quant_i8.__doc__ = (f"(q[M,B] int8, scale[M] fp32) of {dtype_name} rows x [M,K]: x = scale q to half a step, scale the row's "
                        f"largest magnitude / 127, B = K rounded up to 16, padded with zeros (library call {QUANT}).")

    def operands(x, w, scale, xs, gated):
        torch = fused.torch
        dtype = getattr(torch, dtype_name)
        M, K, dev = _first("x", x, dtype if xs is None else torch.int8)
        if xs is not None:
            if K % 16:
                raise ValueError("x of 8-bit integers must have rows of a multiple of 16, as quant_i8 gives them")
            _want("xs", xs, torch.float32, (M,), dev)
        rows = _rows("w", w, torch.int8, -(-K // 16) * 16, dev)
        _want("scale", scale, torch.float32, (rows,), dev)
        if gated and rows % 2:
            raise ValueError("w must have 2 F rows, the gate rows and then the up rows")
        return M, rows // 2 if gated else rows, K, dev, dtype

    def i8(x, w, scale, xs=None, out=None, stream=None):
        if stream is not None:
            return _on(stream, i8, x, w, scale, xs, out)
        address = _address(I8)
        if out is None:
            dev, handle = _place()
            if not _recording(dev):
                y = fused._binding.i8(address, dev, handle, code_of, x, w, scale, xs)
                if y is not None:
                    return y
        M, N, K, dev, dtype = operands(x, w, scale, xs, False)
        if out is None:
            out = x.new_empty((M, N), dtype=dtype)
        else:
            _want("out", out, dtype, (M, N), dev)
        _run(I8, dev, (x.data_ptr(), 0 if xs is None else xs.data_ptr() or 16, w.data_ptr(), scale.data_ptr(), out.data_ptr(), M, N,
                       K), i8_workspace_bytes(M, N, K, False, xs is not None))
        return out

    i8.__doc__ = (f"{dtype_name} out[M,N] = x w^T for 8-bit weights w [N,B] with a scale for each row, as quant_i8 gives them, and "
                  f"tokens x: {dtype_name} [M,K], made integers on the way, or int8 [M,B] with their scales xs (library call {I8}).")

    def i8_gated(x, w, scale, xs=None, act="silu", out=None, stream=None):
        if stream is not None:
            return _on(stream, i8_gated, x, w, scale, xs, act, out)
        address = _address(I8_GATED)
        code = _act(act)
        if out is None:
            dev, handle = _place()
            if not _recording(dev):
                h = fused._binding.i8_gated(address, dev, handle, code_of, x, w, scale, xs, code)
                if h is not None:
                    return h
        M, F, K, dev, dtype = operands(x, w, scale, xs, True)
        if out is None:
            out = x.new_empty((M, F), dtype=dtype)
        else:
            _want("out", out, dtype, (M, F), dev)
        _run(I8_GATED, dev, (x.data_ptr(), 0 if xs is None else xs.data_ptr() or 16, w.data_ptr(), scale.data_ptr(), out.data_ptr(),
                             M, F, K, code), i8_workspace_bytes(M, F, K, True, xs is not None))
        return out

    i8_gated.__doc__ = (f"{dtype_name} h[M,F] = act(x Wg^T) * (x Wu^T) for 8-bit weights of 2F rows, the gate rows and then the up "
                        f"rows, and tokens as {I8} takes them (library call {I8_GATED}).")

    def moe(x, router, w, down, top_k, act="silu", normalize=True, routing=False, out=None, stream=None):
        if stream is not None:
            return _on(stream, moe, x, router, w, down, top_k, act, normalize, routing, out)
        address = _address(MOE)
        code, top_k = _act(act), int(top_k)
        if not 1 <= top_k <= MAX_TOP_K:
            raise ValueError(f"top_k must be 1 to {MAX_TOP_K}, not {top_k}")
        if out is None:
            dev, handle = _place()
            if not _recording(dev):
                y = fused._binding.moe(address, dev, handle, code_of, x, router, w, down, top_k, normalize, code, routing)
                if y is not None:
                    return y
        torch = fused.torch
        dtype = getattr(torch, dtype_name)
        M, D, dev = _first("x", x, dtype)
        E = _rows("router", router, dtype, D, dev)
        _, rows, _ = _three("w", w, dtype, (E, None, D), dev)
        if rows % 2:
            raise ValueError("w must have 2 F rows for each expert, the gate rows and then the up rows")
        if top_k > E:
            raise ValueError(f"top_k must be at most the number of experts, {E}, not {top_k}")
        F = rows // 2
        _three("down", down, dtype, (E, D, F), dev)
        out = _out("out", out, dtype, (M, D), dev, x)
        experts = weights = None
        if routing:
            experts = x.new_empty((M, top_k), dtype=torch.int32)
            weights = x.new_empty((M, top_k), dtype=torch.float32)
        _run(MOE, dev, (x.data_ptr(), router.data_ptr(), w.data_ptr(), down.data_ptr(), out.data_ptr(),
                        experts.data_ptr() if routing else 0, weights.data_ptr() if routing else 0, M, E, D, F, top_k,
                        1 if normalize else 0, code), moe_workspace_bytes(M, E, D, F, top_k))
        return (out, experts, weights) if routing else out

    moe.__doc__ = (f"{dtype_name} y[M,D]: a mixture-of-experts layer for few tokens x [M,D], router [E,D], w [E,2F,D] (gate rows, "
                   "then up rows) and down [E,D,F]; weights are the softmax over the chosen top_k experts' logits "
                   f"(normalize=True) or over all.  With routing=True also the experts [M,top_k] and weights (library call {MOE}).")

    def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, token=None, stream=None):
        if stream is not None:
            return _on(stream, sample, logits, u, temperature, top_k, top_p, min_p, token)
        address = _address(SAMPLE)
        if token is None:
            dev, handle = _place()
            t = fused._binding.sample(address, dev, handle, code_of, logits, u, temperature, top_k, top_p, min_p)
            if t is not None:
                return t
        torch = fused.torch
        for key, t in (("u", u), *zip(SETTINGS, (temperature, top_k, top_p, min_p))):
            if not isinstance(t, torch.Tensor) and (t is not None or key == "u"):
                raise ValueError(f"{key} must be a tensor on the logits' device, not {t!r}")
        M, V, dev = _first("logits", logits, getattr(torch, dtype_name))
        _want("u", u, torch.float32, (M,), dev)
        shared, pointers = 0, []
        for (key, bit), t in zip(SETTINGS.items(), (temperature, top_k, top_p, min_p)):
            if t is None:
                pointers.append(0)
                continue
            dtype = torch.int32 if key == "top_k" else torch.float32
            _want(key, t, dtype, (M,) if t.dim() else (), dev)
            shared |= 0 if t.dim() else bit
            pointers.append(t.data_ptr())
        token = _out("token", token, torch.int64, (M,), dev, logits)
        _run(SAMPLE, dev, (logits.data_ptr(), u.data_ptr(), *pointers, shared, token.data_ptr(), M, V), 0)
        return token

    sample.__doc__ = (f"int64 token[M] from {dtype_name} logits [M,V] and random numbers u, fp32 [M] in [0,1).  temperature, top_p and "
                      "min_p (fp32) and top_k (int32) are tensors of a value for each row, or of one for all, or None; -1 for "
                      f"a row with nothing to take (library call {SAMPLE}).")

    made = {}
    for fn in (quant_i8, i8, i8_gated, moe, sample):
        full = name(fn.__name__)
        fn.__name__ = fn.__qualname__ = full
        made[full] = fn
    return made


FUNCTIONS = {**_make("f16", "float16"), **_make("bf16", "bfloat16")}
