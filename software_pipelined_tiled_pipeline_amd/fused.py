"""Python binding of the fused operators (argument marshalling only).

The functions are reached through :mod:`pgemm`, next to the products:
``pgemm_{f16,bf16}_gated`` and ``_gated_bwd``, ``_xent`` and ``_xent_bwd``,
``_q4`` and ``_q4_gated``.  Tensors live on the current GPU; what a call needs
as workspace is a torch tensor on the call's stream, registered there and kept
for later calls.  All arithmetic runs in the library's kernels.
"""
from __future__ import annotations

import ctypes

ACTS = {"silu": 0, "gelu": 1}
FUSED_OPS = {"gated": 0, "gated_save": 1, "gated_bwd": 2, "xent": 3, "xent_bwd": 4}
FUSED_SYMBOLS = tuple(f"pgemm_{t}_{op}" for t in ("f16", "bf16")
                      for op in ("gated", "gated_bwd", "xent", "xent_bwd", "q4", "q4_gated"))


def declare(L) -> None:
    """Argument types of the fused entry points of the loaded library."""
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    args = {
        "gated": [P, P, P, P, I64, I64, I64, I, P],
        "gated_bwd": [P, P, P, P, P, P, I64, I64, I64, I, P],
        "xent": [P, P, P, P, P, I64, I64, I64, I64, P],
        "xent_bwd": [P, I, P, P, P, P, P, P, I64, I64, I64, I64, P],
        "q4": [P, P, P, P, P, I64, I64, I64, I64, P],
        "q4_gated": [P, P, P, P, P, I64, I64, I64, I64, I, P],
    }
    for name in FUSED_SYMBOLS:
        f = getattr(L, name)
        f.argtypes = args[name.split("_", 2)[2]]
        f.restype = I
    L.pgemm_fused_workspace.argtypes = [I, I64, I64, I64, ctypes.POINTER(I64)]
    L.pgemm_fused_workspace.restype = I


def workspace_bytes(op: str, M: int, N: int, K: int) -> int:
    """Bytes of workspace of a call: (M, N, K) is (M, F, D) or (M, V, D)."""
    from . import pgemm
    n = ctypes.c_int64()
    pgemm._check(pgemm.lib().pgemm_fused_workspace(FUSED_OPS[op], M, N, K, ctypes.byref(n)), "pgemm_fused_workspace")
    return n.value


def _here():
    import torch
    if not torch.cuda.is_available():
        raise ValueError("pgemm needs a GPU")
    return torch.device("cuda", torch.cuda.current_device())


def _tensor(name, t, dtype, shape, here):
    """Checks one operand; a size of None in `shape` takes any size."""
    if t.dtype != dtype or not t.is_cuda or t.device != here:
        raise ValueError(f"{name} must be a {dtype} tensor on the current device {here}, not {t.dtype} on {t.device}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        want = "[" + ", ".join("any" if w is None else str(w) for w in shape) + "]"
        raise ValueError(f"{name} must have shape {want}, not {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _out(name, t, dtype, shape, here):
    import torch
    return torch.empty(shape, dtype=dtype, device=here) if t is None else _tensor(name, t, dtype, shape, here)


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, not {act!r}")
    return ACTS[act]


def _ptr(t):
    return None if t is None else (t.data_ptr() or None)


def _run(name, op, sizes, args, stream):
    from . import pgemm
    if op is not None:
        need = workspace_bytes(op, *sizes)
        if need:
            pgemm.ensure_workspace(need, stream)
    pgemm._check(getattr(pgemm.lib(), name)(*args, pgemm._stream(stream)), name)


def _saved_shape(M, F):
    return (M, -(-F // 4), 8)


def _make(fmt, dtype_name):
    def dtype():
        import torch
        return getattr(torch, dtype_name)

    def block(x, w, here):
        _tensor("x", x, dtype(), (None, None), here)
        M, D = x.shape
        _tensor("w", w, dtype(), (None, D), here)
        if w.shape[0] % 2:
            raise ValueError("w must have 2 F rows, the gate rows and then the up rows")
        return M, w.shape[0] // 2, D

    def gated(x, w, act="silu", out=None, save=False, stream=None):
        import torch
        here = _here()
        M, F, D = block(x, w, here)
        code = _act(act)
        h = _out("out", out, dtype(), (M, F), here)
        saved = torch.empty(_saved_shape(M, F), dtype=torch.float32, device=here) if save else None
        _run(f"pgemm_{fmt}_gated", "gated_save" if save else "gated", (M, F, D),
             (_ptr(x), _ptr(w), _ptr(h), _ptr(saved), M, F, D, code), stream)
        return (h, saved) if save else h

    gated.__doc__ = (f"{dtype_name} h[M,F] = act(x Wg^T) * (x Wu^T) for x [M,D] and w [2F,D], the gate rows and then the up "
                     f"rows (library call pgemm_{fmt}_gated); act is 'silu' or 'gelu' (tanh form).  With save=True also "
                     "returns the fp32 projections for the backward call, 8 bytes per value of h.")

    def gated_bwd(dh, x, w, saved=None, act="silu", dx=None, dw=None, stream=None):
        import torch
        here = _here()
        M, F, D = block(x, w, here)
        code = _act(act)
        _tensor("dh", dh, dtype(), (M, F), here)
        if saved is not None:
            _tensor("saved", saved, torch.float32, _saved_shape(M, F), here)
        dx = _out("dx", dx, dtype(), (M, D), here)
        dw = _out("dw", dw, dtype(), (2 * F, D), here)
        _run(f"pgemm_{fmt}_gated_bwd", "gated_bwd", (M, F, D),
             (_ptr(dh), _ptr(x), _ptr(w), _ptr(saved), _ptr(dx), _ptr(dw), M, F, D, code), stream)
        return dx, dw

    gated_bwd.__doc__ = (f"(dx[M,D], dw[2F,D]) of pgemm_{fmt}_gated for dh [M,F].  saved: what the forward call kept "
                         "(faster: two products fewer); None computes the projections again.")

    def xent(x, w, target, ignore_index=-100, loss=None, lse=None, stream=None):
        import torch
        here = _here()
        _tensor("x", x, dtype(), (None, None), here)
        M, D = x.shape
        _tensor("w", w, dtype(), (None, D), here)
        V = w.shape[0]
        _tensor("target", target, torch.int64, (M,), here)
        loss = _out("loss", loss, torch.float32, (M,), here)
        lse = _out("lse", lse, torch.float32, (M,), here)
        _run(f"pgemm_{fmt}_xent", "xent", (M, V, D),
             (_ptr(x), _ptr(w), _ptr(target), _ptr(loss), _ptr(lse), M, V, D, int(ignore_index)), stream)
        return loss, lse

    xent.__doc__ = (f"(loss[M], lse[M]) in fp32: softmax cross entropy of the logits x w^T for {dtype_name} x [M,D] and w "
                    f"[V,D], without storing them (library call pgemm_{fmt}_xent).  Rows whose target is ignore_index have "
                    "loss 0; any other target outside the vocabulary makes its loss NaN.")

    def xent_bwd(dloss, x, w, target, lse, ignore_index=-100, dx=None, dw=None, stream=None):
        import torch
        here = _here()
        _tensor("x", x, dtype(), (None, None), here)
        M, D = x.shape
        _tensor("w", w, dtype(), (None, D), here)
        V = w.shape[0]
        _tensor("target", target, torch.int64, (M,), here)
        _tensor("lse", lse, torch.float32, (M,), here)
        if dloss.dtype != torch.float32 or not dloss.is_cuda or dloss.device != here:
            raise ValueError(f"dloss must be a torch.float32 tensor on the current device {here}")
        if dloss.dim() == 0:
            step = 0
        elif tuple(dloss.shape) == (M,) and (M <= 1 or dloss.stride(0) in (0, 1)):
            step = 0 if M > 1 and dloss.stride(0) == 0 else 1
        else:
            raise ValueError("dloss must be a scalar, or have shape [M] and be contiguous or expanded from a scalar")
        dx = _out("dx", dx, dtype(), (M, D), here)
        dw = _out("dw", dw, dtype(), (V, D), here)
        _run(f"pgemm_{fmt}_xent_bwd", "xent_bwd", (M, V, D),
             (_ptr(dloss), step, _ptr(x), _ptr(w), _ptr(target), _ptr(lse), _ptr(dx), _ptr(dw), M, V, D,
              int(ignore_index)), stream)
        return dx, dw

    xent_bwd.__doc__ = (f"(dx[M,D], dw[V,D]) of pgemm_{fmt}_xent for dloss, fp32 [M] or a scalar that all rows share, and "
                        "the forward call's lse.")

    def q4_operands(x, q, scale, zero, group, here):
        import torch
        _tensor("x", x, dtype(), (None, None), here)
        M, K = x.shape
        if group <= 0 or group % 32:
            raise ValueError("group must be a positive multiple of 32")
        _tensor("q", q, torch.uint8, (None, -(-K // 32) * 16), here)
        rows, groups = q.shape[0], -(-K // group)
        _tensor("scale", scale, dtype(), (rows, groups), here)
        if zero is not None:
            _tensor("zero", zero, torch.uint8, (rows, groups), here)
        return M, rows, K

    def q4(x, q, scale, zero=None, group=128, out=None, stream=None):
        here = _here()
        M, N, K = q4_operands(x, q, scale, zero, group, here)
        out = _out("out", out, dtype(), (M, N), here)
        _run(f"pgemm_{fmt}_q4", None, None,
             (_ptr(x), _ptr(q), _ptr(scale), _ptr(zero), _ptr(out), M, N, K, int(group)), stream)
        return out

    q4.__doc__ = (f"{dtype_name} out[M,N] = x[M,K] w^T for few rows and 4-bit weights w[n,k] = scale[n,k/group] (q[n,k] - "
                  "zero[n,k/group]); q as pack_q4 gives it, zero None means 8 "
                  f"(library call pgemm_{fmt}_q4).")

    def q4_gated(x, q, scale, zero=None, group=128, act="silu", out=None, stream=None):
        here = _here()
        M, rows, K = q4_operands(x, q, scale, zero, group, here)
        code = _act(act)
        if rows % 2:
            raise ValueError("q must have 2 F rows, the gate rows and then the up rows")
        F = rows // 2
        out = _out("out", out, dtype(), (M, F), here)
        _run(f"pgemm_{fmt}_q4_gated", None, None,
             (_ptr(x), _ptr(q), _ptr(scale), _ptr(zero), _ptr(out), M, F, K, int(group), code), stream)
        return out

    q4_gated.__doc__ = (f"{dtype_name} h[M,F] = act(x Wg^T) * (x Wu^T) for few rows and 4-bit weights of 2F rows, the gate rows "
                        f"and then the up rows (library call pgemm_{fmt}_q4_gated).")

    made = {}
    for fn in (gated, gated_bwd, xent, xent_bwd, q4, q4_gated):
        name = f"pgemm_{fmt}_{fn.__name__}"
        fn.__name__ = fn.__qualname__ = name
        made[name] = fn
    return made


FUNCTIONS = {**_make("f16", "float16"), **_make("bf16", "bfloat16")}


def pack_q4(values):
    """The packed rows [N, 16 ceil(K/32)] of 4-bit weights given as a uint8 tensor [N, K] of values 0..15, on any device."""
    import torch
    if values.dtype != torch.uint8 or values.dim() != 2:
        raise ValueError("values must be a 2-D uint8 tensor of weights 0..15")
    if values.numel() and int(values.max()) > 15:
        raise ValueError("a 4-bit weight is 0..15")
    N, K = values.shape
    wide = torch.zeros((N, -(-K // 32) * 32), dtype=torch.uint8, device=values.device)
    wide[:, :K] = values
    return (wide[:, 0::2] | (wide[:, 1::2] << 4)).contiguous()
