"""Python binding of the fused operators (argument marshalling only).

The functions are reached through :mod:`pgemm`, next to the products:
``pgemm_{f16,bf16}_gated`` and ``_gated_bwd``, ``_xent`` and ``_xent_bwd``,
``_q4`` and ``_q4_gated``.  Tensors live on the current GPU; every function also
takes a ``stream`` to run on.  What a call needs as workspace is a torch tensor
on the call's stream, registered there and kept for later calls.  All arithmetic runs in the library's kernels.

Like the products, the functions are not part of torch's autograd: what they
return carries no graph, also where an operand requires gradients.  Each forward
call has its backward call, and examples/gated_lm.py joins them in
torch.autograd.Function.  With a `stream` of its own, a call's operands have to be
ready on that stream and to live until it has read them.
"""
from __future__ import annotations

import ctypes
import functools
import os

_BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")
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


@functools.lru_cache(maxsize=1024)
def workspace_bytes(op: str, M: int, N: int, K: int) -> int:
    """Bytes of workspace of a call: (M, N, K) is (M, F, D) or (M, V, D)."""
    _load()
    n = ctypes.c_int64()
    pgemm._check(pgemm.lib().pgemm_fused_workspace(FUSED_OPS[op], M, N, K, ctypes.byref(n)), "pgemm_fused_workspace")
    return n.value


# torch, the products' binding and the compiled short way, found by the first
# call: the package loads without torch, and the binding imports this module
torch = pgemm = _binding = None


def _load():
    global torch, pgemm, _binding
    if pgemm is None:
        import torch
        from . import pgemm
        if not os.path.exists(_BINDING_PATH):
            raise RuntimeError(f"{_BINDING_PATH} is missing: build it with __graft_entry__.build()")
        from . import _binding


def _refuse(name, t, dtype, shape):
    """Says what is wrong with one operand; a size of None in `shape` takes any size."""
    if not torch.cuda.is_available():
        raise ValueError("pgemm needs a GPU")
    here = torch.device("cuda", torch.cuda.current_device())
    if t.dtype != dtype or not t.is_cuda or t.device != here:
        raise ValueError(f"{name} must be a {dtype} tensor on the current device {here}, not {t.dtype} on {t.device}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        want = "[" + ", ".join("any" if w is None else str(w) for w in shape) + "]"
        raise ValueError(f"{name} must have shape {want}, not {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _first(name, t, dtype):
    """Checks a call's first matrix; (rows, columns, current device)."""
    dev = t.get_device()
    if dev < 0 or t.dim() != 2 or t.dtype is not dtype or dev != torch._C._cuda_getDevice() or not t.is_contiguous():
        _refuse(name, t, dtype, (None, None))
    rows, cols = t.shape
    return rows, cols, dev


def _want(name, t, dtype, shape, dev):
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _refuse(name, t, dtype, shape)


def _rows(name, t, dtype, cols, dev):
    """Checks a matrix of any number of rows; that number."""
    if t.dim() != 2 or t.shape[1] != cols or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(name, t, dtype, (None, cols))
    return t.shape[0]


def _out(name, t, dtype, shape, dev, like):
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _want(name, t, dtype, shape, dev)
    return t


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, not {act!r}")
    return ACTS[act]


def _ignored(ignore_index):
    """ignore_index as the library's 64 bits: ctypes would cut a longer one off without a word."""
    i = int(ignore_index)
    if not -(1 << 63) <= i < 1 << 63:
        raise ValueError(f"ignore_index must fit 64 bits, not {ignore_index!r}")
    return i


# A call first takes the short way: _binding checks its tensors, allocates the
# outputs and calls the library (8.3 us -> 5.4 for a product of one token).  It
# returns None for anything that is not plainly right, and where the stream's
# workspace is missing or too small; then the checks here say why, or register
# one.  Calls with outputs of their own, or that need a workspace while a graph
# is recorded, do not take it.

_entries = {}    # library functions by name
_addresses = {}  # and their addresses


def _entry(name):
    f = _entries[name] = getattr(pgemm.lib(), name)
    return f


def _address(name):
    if pgemm is None:
        _load()
    if name not in _entries:
        _entry(name)
    a = _addresses[name] = ctypes.cast(_entries[name], ctypes.c_void_p).value
    return a


def _place():
    """The current device and stream; a device of -1, which no tensor is on, in a process that has used none."""
    if not torch.cuda.is_initialized():
        return -1, 0
    dev = torch._C._cuda_getDevice()
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _recording(dev):
    return dev >= 0 and torch._C._cuda_isCurrentStreamCapturing()


def _failed(name, status):
    raise pgemm.PgemmError(status, name)


def _run(name, dev, args, need):
    """Calls the library on the current stream, with a workspace of `need` bytes."""
    f = _entries[name]
    handle = torch._C._cuda_getCurrentRawStream(dev)
    if need:
        if torch.cuda.is_current_stream_capturing():
            # A graph replays with this buffer for as long as it lives, so it is
            # the graph's own, from its memory pool, and not the stream's, which
            # a later call may replace.
            own = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev))
            pgemm._register(handle, own)
            try:
                status = f(*args, handle)
            finally:
                pgemm._register(handle, pgemm._workspaces.get((dev, handle)))
            if status != 0:
                _failed(name, status)
            return
        ws = pgemm._workspaces.get((dev, handle))
        if ws is None or ws.numel() < need:
            pgemm.ensure_workspace(need)
    status = f(*args, handle)
    if status != 0:
        _failed(name, status)


def _on(stream, fn, *args):
    """The call on another stream: its outputs and kernels then belong to that one instead of the current one."""
    if pgemm is None:
        _load()
    with torch.cuda.stream(stream):
        return fn(*args)


def _saved_shape(M, F):
    return (M, -(-F // 4), 8)


def _make(fmt, dtype_name):
    def name(op):
        return f"pgemm_{fmt}_{op}"

    code_of = {"f16": 0, "bf16": 1}[fmt]
    GATED, GATED_BWD, XENT, XENT_BWD, Q4, Q4_GATED = map(
        name, ("gated", "gated_bwd", "xent", "xent_bwd", "q4", "q4_gated"))

    def block(x, w, dtype):
        M, D, dev = _first("x", x, dtype)
        rows = _rows("w", w, dtype, D, dev)
        if rows % 2:
            raise ValueError("w must have 2 F rows, the gate rows and then the up rows")
        return M, rows // 2, D, dev

    def gated(x, w, act="silu", out=None, save=False, stream=None):
        if stream is not None:
            return _on(stream, gated, x, w, act, out, save)
        address = _addresses.get(GATED) or _address(GATED)
        code = _act(act)
        if out is None:
            dev, handle = _place()
            if not _recording(dev):
                h = _binding.gated(address, dev, handle, code_of, x, w, code, save)
                if h is not None:
                    return h
        dtype = getattr(torch, dtype_name)
        M, F, D, dev = block(x, w, dtype)
        h = _out("out", out, dtype, (M, F), dev, x)
        saved = x.new_empty(_saved_shape(M, F), dtype=torch.float32) if save else None
        _run(GATED, dev, (x.data_ptr(), w.data_ptr(), h.data_ptr(), 0 if saved is None else saved.data_ptr(), M, F, D,
                          code), workspace_bytes("gated_save" if save else "gated", M, F, D))
        return (h, saved) if save else h

    gated.__doc__ = (f"{dtype_name} h[M,F] = act(x Wg^T) * (x Wu^T) for x [M,D] and w [2F,D], the gate rows and then the up "
                     f"rows (library call {GATED}); act is 'silu' or 'gelu' (tanh form).  With save=True also "
                     "returns the fp32 projections for the backward call, 8 bytes per value of h.")

    def gated_bwd(dh, x, w, saved=None, act="silu", dx=None, dw=None, stream=None):
        if stream is not None:
            return _on(stream, gated_bwd, dh, x, w, saved, act, dx, dw)
        address = _addresses.get(GATED_BWD) or _address(GATED_BWD)
        code = _act(act)
        if dx is None and dw is None:
            dev, handle = _place()
            if not _recording(dev):
                both = _binding.gated_bwd(address, dev, handle, code_of, dh, x, w, saved, code)
                if both is not None:
                    return both
        dtype = getattr(torch, dtype_name)
        M, F, D, dev = block(x, w, dtype)
        _want("dh", dh, dtype, (M, F), dev)
        if saved is not None:
            _want("saved", saved, torch.float32, _saved_shape(M, F), dev)
        dx = _out("dx", dx, dtype, (M, D), dev, x)
        dw = _out("dw", dw, dtype, (2 * F, D), dev, x)
        _run(GATED_BWD, dev, (dh.data_ptr(), x.data_ptr(), w.data_ptr(), 0 if saved is None else saved.data_ptr(),
                              dx.data_ptr(), dw.data_ptr(), M, F, D, code), workspace_bytes("gated_bwd", M, F, D))
        return dx, dw

    gated_bwd.__doc__ = (f"(dx[M,D], dw[2F,D]) of {GATED} for dh [M,F].  saved: what the forward call kept "
                         "(faster: two products fewer); None computes the projections again.")

    def head(x, w, target, dtype):
        M, D, dev = _first("x", x, dtype)
        V = _rows("w", w, dtype, D, dev)
        _want("target", target, torch.int64, (M,), dev)
        return M, V, D, dev

    def xent(x, w, target, ignore_index=-100, loss=None, lse=None, stream=None):
        if stream is not None:
            return _on(stream, xent, x, w, target, ignore_index, loss, lse)
        address = _addresses.get(XENT) or _address(XENT)
        if loss is None and lse is None:
            dev, handle = _place()
            if not _recording(dev):
                both = _binding.xent(address, dev, handle, code_of, x, w, target, ignore_index)
                if both is not None:
                    return both
        ignore = _ignored(ignore_index)
        M, V, D, dev = head(x, w, target, getattr(torch, dtype_name))
        loss = _out("loss", loss, torch.float32, (M,), dev, x)
        lse = _out("lse", lse, torch.float32, (M,), dev, x)
        _run(XENT, dev, (x.data_ptr(), w.data_ptr(), target.data_ptr(), loss.data_ptr(), lse.data_ptr(), M, V, D,
                         ignore), workspace_bytes("xent", M, V, D))
        return loss, lse

    xent.__doc__ = (f"(loss[M], lse[M]) in fp32: softmax cross entropy of the logits x w^T for {dtype_name} x [M,D] and w "
                    f"[V,D], without storing them (library call {XENT}).  Rows whose target is ignore_index have "
                    "loss 0; any other target outside the vocabulary makes its loss NaN.")

    def xent_bwd(dloss, x, w, target, lse, ignore_index=-100, dx=None, dw=None, stream=None):
        if stream is not None:
            return _on(stream, xent_bwd, dloss, x, w, target, lse, ignore_index, dx, dw)
        address = _addresses.get(XENT_BWD) or _address(XENT_BWD)
        if dx is None and dw is None:
            dev, handle = _place()
            if not _recording(dev):
                both = _binding.xent_bwd(address, dev, handle, code_of, dloss, x, w, target, lse, ignore_index)
                if both is not None:
                    return both
        dtype, ignore = getattr(torch, dtype_name), _ignored(ignore_index)
        M, V, D, dev = head(x, w, target, dtype)
        _want("lse", lse, torch.float32, (M,), dev)
        if dloss.dtype != torch.float32 or dloss.get_device() != dev:
            raise ValueError(f"dloss must be a torch.float32 tensor on the current device cuda:{dev}")
        if dloss.dim() == 0:
            step = 0
        elif dloss.shape == (M,) and (M <= 1 or dloss.stride(0) in (0, 1)):
            step = 0 if M > 1 and dloss.stride(0) == 0 else 1
        else:
            raise ValueError("dloss must be a scalar, or have shape [M] and be contiguous or expanded from a scalar")
        dx = _out("dx", dx, dtype, (M, D), dev, x)
        dw = _out("dw", dw, dtype, (V, D), dev, x)
        _run(XENT_BWD, dev, (dloss.data_ptr(), step, x.data_ptr(), w.data_ptr(), target.data_ptr(), lse.data_ptr(),
                             dx.data_ptr(), dw.data_ptr(), M, V, D, ignore),
             workspace_bytes("xent_bwd", M, V, D))
        return dx, dw

    xent_bwd.__doc__ = (f"(dx[M,D], dw[V,D]) of {XENT} for dloss, fp32 [M] or a scalar that all rows share, and "
                        "the forward call's lse.")

    def q4_operands(x, q, scale, zero, group, dtype):
        if group <= 0 or group % 32 or group >= 1 << 31:
            raise ValueError("group must be a positive multiple of 32 below 2^31")
        M, K, dev = _first("x", x, dtype)
        rows, groups = _rows("q", q, torch.uint8, -(-K // 32) * 16, dev), -(-K // group)
        _want("scale", scale, dtype, (rows, groups), dev)
        if zero is not None:
            _want("zero", zero, torch.uint8, (rows, groups), dev)
        return M, rows, K, dev

    def q4(x, q, scale, zero=None, group=128, out=None, stream=None):
        if stream is not None:
            return _on(stream, q4, x, q, scale, zero, group, out)
        address = _addresses.get(Q4) or _address(Q4)
        if out is None:
            dev, handle = _place()
            y = _binding.q4(address, dev, handle, code_of, x, q, scale, zero, group)
            if y is not None:
                return y
        dtype = getattr(torch, dtype_name)
        M, N, K, dev = q4_operands(x, q, scale, zero, group, dtype)
        out = _out("out", out, dtype, (M, N), dev, x)
        _run(Q4, dev, (x.data_ptr(), q.data_ptr(), scale.data_ptr(), 0 if zero is None else zero.data_ptr(),
                       out.data_ptr(), M, N, K, int(group)), 0)
        return out

    q4.__doc__ = (f"{dtype_name} out[M,N] = x[M,K] w^T for few rows and 4-bit weights w[n,k] = scale[n,k/group] (q[n,k] - "
                  "zero[n,k/group]); q as pack_q4 gives it, zero None means 8 "
                  f"(library call {Q4}).")

    def q4_gated(x, q, scale, zero=None, group=128, act="silu", out=None, stream=None):
        if stream is not None:
            return _on(stream, q4_gated, x, q, scale, zero, group, act, out)
        address = _addresses.get(Q4_GATED) or _address(Q4_GATED)
        code = _act(act)
        if out is None:
            dev, handle = _place()
            h = _binding.q4_gated(address, dev, handle, code_of, x, q, scale, zero, group, code)
            if h is not None:
                return h
        dtype = getattr(torch, dtype_name)
        M, rows, K, dev = q4_operands(x, q, scale, zero, group, dtype)
        if rows % 2:
            raise ValueError("q must have 2 F rows, the gate rows and then the up rows")
        F = rows // 2
        out = _out("out", out, dtype, (M, F), dev, x)
        _run(Q4_GATED, dev, (x.data_ptr(), q.data_ptr(), scale.data_ptr(), 0 if zero is None else zero.data_ptr(),
                             out.data_ptr(), M, F, K, int(group), code), 0)
        return out

    q4_gated.__doc__ = (f"{dtype_name} h[M,F] = act(x Wg^T) * (x Wu^T) for few rows and 4-bit weights of 2F rows, the gate rows "
                        f"and then the up rows (library call {Q4_GATED}).")

    made = {}
    for fn in (gated, gated_bwd, xent, xent_bwd, q4, q4_gated):
        full = name(fn.__name__)
        fn.__name__ = fn.__qualname__ = full
        made[full] = fn
    return made


FUNCTIONS = {**_make("f16", "float16"), **_make("bf16", "bfloat16")}


def pack_q4(values):
    """The packed rows [N, 16 ceil(K/32)] of 4-bit weights given as a uint8 tensor [N, K] of values 0..15, on any device."""
    _load()
    if values.dtype != torch.uint8 or values.dim() != 2:
        raise ValueError("values must be a 2-D uint8 tensor of weights 0..15")
    if values.numel() and int(values.max()) > 15:
        raise ValueError("a 4-bit weight is 0..15")
    N, K = values.shape
    wide = torch.zeros((N, -(-K // 32) * 32), dtype=torch.uint8, device=values.device)
    wide[:, :K] = values
    return (wide[:, 0::2] | (wide[:, 1::2] << 4)).contiguous()
