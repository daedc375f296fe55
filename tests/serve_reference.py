"""The serving operators in 64 bits, with bounds on how far a result may be off
(test infrastructure).

As in fused_reference: each function takes the operands as the kernels get
them and returns (value, bound) per output; whole numbers come without a bound,
they have to be equal.  The bounds count half a step of the result's type,
fp32 accumulation, the roundings of values that are multiplied on in 16 bits,
and a few fp32 steps for the functions.
"""
import math

import torch

from fused_reference import SLOPE, STEPS, U32, activation, half_step, product, tiny

NORMAL = 2.0 ** -126  # the smallest normal number of fp32


def width(K):
    return -(-K // 16) * 16


def quant(x):
    """(q, scale): integers of the exact quotient, halves to the even one."""
    M, K = x.shape
    top = x.double().abs().amax(1) if K else torch.zeros(M, dtype=torch.float64, device=x.device)
    # 127 divides no 11-bit number, and a quotient by it repeats every 7 bits: rounding it in two steps is rounding it in one
    scale = (top / 127).clamp(min=NORMAL).float()
    bad = ~torch.isfinite(top)
    scale[bad] = math.nan
    q = torch.zeros((M, width(K)), dtype=torch.int8, device=x.device)
    v = torch.round(x.double() / scale.double()[:, None])
    v[bad] = 0
    q[:, :K] = v.to(torch.int8)
    return q, scale


def i8(q, xs, w, ws, dtype, act=None):
    s = xs.double()[:, None] * ws.double()
    y = q.double() @ w.double().t() * s  # |sums| < 2^31: exact
    e = 4 * U32 * y.abs() + 2.0 ** -149  # to fp32, and two factors
    if act is not None:
        F = y.shape[1] // 2
        g, u, eg, eu = y[:, :F], y[:, F:], e[:, :F], e[:, F:]
        a, _ = activation(act, g)
        ea = SLOPE * eg + STEPS * U32 * (a.abs() + g.abs() * 0.5 + U32)
        y, e = a * u, ea * u.abs() + a.abs() * eu + ea * eu
    return y, e + half_step(dtype) * (y.abs() + e) + tiny(dtype)


def route(x, router, k, normalize):
    """(experts, (weights, bound)): the largest logits first, the lowest index of equal ones."""
    l = x.double() @ router.double().t()
    by, at = torch.sort(l, dim=1, descending=True, stable=True)
    e = torch.exp(by - by[:, :1])
    p = e[:, :k] / (e[:, :k] if normalize else e).sum(1, keepdim=True)
    return at[:, :k].int(), (p, U32 * p + 2.0 ** -149)


def moe(x, router, w, down, k, act, normalize):
    """(y with its bound, experts, weights with theirs)."""
    dtype = x.dtype
    (M, D), (E, _, F) = x.shape, down.shape
    experts, (p, ep) = route(x, router, k, normalize)
    y = torch.zeros((M, D), dtype=torch.float64, device=x.device)
    e = torch.zeros_like(y)
    size = torch.zeros_like(y)  # of the terms of the last sum
    for j in range(E):
        row, place = torch.nonzero(experts == j, as_tuple=True)
        if len(row) == 0:
            continue
        g, eg = product(x[row], w[j, :F])
        u, eu = product(x[row], w[j, F:])
        a, _ = activation(act, g)
        ea = SLOPE * eg + STEPS * U32 * (a.abs() + g.abs() * 0.5 + U32)
        h, eh = a * u, ea * u.abs() + a.abs() * eu + ea * eu
        eh = eh + half_step(dtype) * (h.abs() + eh)
        if dtype == torch.float16:  # after a power of two that takes a row's largest to 2^14 or more
            eh = eh + 2.0 ** -25 * 2.0 ** -14 * h.abs().amax(1, keepdim=True)
        else:
            eh = eh + tiny(dtype)
        d = down[j].double()
        v = h @ d.t()
        ev = eh @ d.abs().t() + (F + 8) * U32 * ((h.abs() + eh) @ d.abs().t())
        pj, epj = p[row, place][:, None], ep[row, place][:, None]
        y[row] += pj * v
        e[row] += pj * ev + epj * (v.abs() + ev)
        size[row] += pj * (v.abs() + ev)
    e = e + (k + 24) * U32 * size  # the weight, an expert's runs on several waves, and their sum
    return (y, e + half_step(dtype) * (y.abs() + e) + tiny(dtype)), experts, (p, ep)


def sample(z, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """The tokens, row by row in Python numbers."""
    M, V = z.shape
    out = []

    def value(t, m, default):
        return default if t is None else float(t.reshape(-1)[m if t.dim() else 0])
    for m in range(M):
        row = z[m].double().cpu()
        t, k = value(temperature, m, 1.0), value(top_k, m, 0)
        p, q, r = value(top_p, m, 1.0), value(min_p, m, 0.0), float(u[m])
        if torch.isnan(row).any() or not (row > -math.inf).any() or not t >= 0 or p != p or q != q or r != r:
            out.append(-1)
            continue
        by, at = torch.sort(row, descending=True, stable=True)
        by, at = by[by > -math.inf], at[by > -math.inf]
        if t == 0:
            out.append(int(at[0]))
            continue
        d = torch.where(by == by[0], torch.zeros_like(by), (by - by[0]) / t)
        e = torch.exp(torch.nan_to_num(d, nan=-math.inf))
        n = len(by) if k <= 0 else min(len(by), int(k))
        run = e.cumsum(0)
        kept = n
        if p < 1:
            kept = min(kept, int((run[:n] < p * run[n - 1]).sum()) + 1)
        if q > 0:
            kept = min(kept, int((e >= q).sum()))
        kept = max(kept, 1)
        i = int((run[:kept] <= r * run[kept - 1]).sum())
        out.append(int(at[min(i, kept - 1)]))
    return torch.tensor(out, dtype=torch.int64)
