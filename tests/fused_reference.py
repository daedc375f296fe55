"""The fused operators in 64 bits, with bounds on how far a result may be off
(test infrastructure).

Each function takes the operands as the kernels get them and returns, per
output, (value, bound): the bound counts, element by element, half a step of
the result's type, fp32 accumulation ((n + 8) 2^-24 times the sum of the
products' magnitudes for n products in any order), the roundings of values
that are multiplied on in 16 bits (half a step each) and a few fp32 steps for
the functions.
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the subnormals."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def product(a, b):
    """a b^T in 64 bits, and fp32's accumulation bound."""
    a, b = a.double(), b.double()
    return a @ b.t(), (a.shape[1] + 8) * U32 * (a.abs() @ b.abs().t())


def activation(act, g):
    """Value, slope and a bound of the second derivative's size."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    c = math.sqrt(2 / math.pi)
    y = c * (g + 0.044715 * g ** 3)
    t = torch.tanh(y)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


# largest |a'| and |a''| of either activation; fp32 steps that computing a or
# a' costs: the exponential's argument y (|y| steps, damped by s(1-s)), the
# exponential, reciprocal and products
SLOPE, BEND, STEPS = 1.13, 1.2, 16.0


def gated(x, w, act, dh=None):
    dtype = x.dtype
    F = w.shape[0] // 2
    g, eg = product(x, w[:F])
    u, eu = product(x, w[F:])
    a, s = activation(act, g)
    ea = SLOPE * eg + STEPS * U32 * (a.abs() + g.abs() * 0.5 + U32)
    h = a * u
    eh = ea * u.abs() + a.abs() * eu + ea * eu
    out = {"h": (h, eh + half_step(dtype) * (h.abs() + eh) + tiny(dtype))}
    if dh is not None:
        d = dh.double()
        es = BEND * eg + STEPS * U32 * (s.abs() + 1)
        dg, du = d * u * s, d * a
        eg2 = d.abs() * (eu * s.abs() + u.abs() * es + eu * es + 4 * U32 * (u * s).abs())
        eu2 = d.abs() * ea
        dy, edy = torch.cat([dg, du], 1), torch.cat([eg2, eu2], 1)
        edy = edy + half_step(dtype) * (dy.abs() + edy) + tiny(dtype)
        out["dx"] = _times(dy, edy, w.double().t(), dtype)
        out["dw"] = _times(dy.t().contiguous(), edy.t().contiguous(), x.double().t(), dtype)
    return out


def _times(a, ea, b, dtype, extra=0.0):
    """a b^T for a that is known to ea, rounded to dtype."""
    b = b.contiguous()
    v = a @ b.t()
    e = ea @ b.abs().t() + (a.shape[1] + 8) * U32 * ((a.abs() + ea) @ b.abs().t()) + extra
    return v, e + half_step(dtype) * (v.abs() + e) + tiny(dtype)


def xent(x, w, target, ignore=-100, dloss=None):
    dtype = x.dtype
    V = w.shape[0]
    z, ez = product(x, w)
    lse = torch.logsumexp(z, 1)
    top = z.max(1).values
    p = torch.exp(z - lse[:, None])
    steps = (p * (2 * (z - top[:, None]).abs() + 8)).sum(1) + 256  # exponentials; sums within and between tiles
    elog = ez.max(1).values + U32 * (steps + 4 * lse.abs() + 4 * top.abs())
    counts = target != ignore
    at = torch.where(counts, target, torch.zeros_like(target))[:, None]
    loss = torch.where(counts, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    eloss = torch.where(counts, elog + ez.gather(1, at)[:, 0] + 2 * U32 * loss.abs(), torch.zeros_like(lse))
    out = {"lse": (lse, elog), "loss": (loss, eloss)}
    if dloss is not None:
        s = torch.where(counts, dloss.double().expand(target.shape), torch.zeros_like(lse))[:, None]
        hot = torch.zeros_like(z).scatter_(1, at, counts.double()[:, None])
        dz = s * (p - hot)
        ep = p * (ez + elog[:, None] + U32 * (2 * (z - lse[:, None]).abs() + 8))
        edz = s.abs() * (ep + U32 * (p + hot))
        edz = edz + half_step(dtype) * (dz.abs() + edz)
        if dtype == torch.float16:  # scaled so that the largest |dloss| is at least 2^14
            edz = edz + 2.0 ** -25 * s.abs().max() * 2.0 ** -14 * counts[:, None]
        out["dx"] = _times(dz, edz, w.double().t(), dtype)
        out["dw"] = _times(dz.t().contiguous(), edz.t().contiguous(), x.double().t(), dtype)
    return out


def weights(values, scale, zero, group):
    K = values.shape[1]
    at = torch.arange(K, device=values.device) // group
    z = 8.0 if zero is None else zero.double()[:, at]
    return (values.double() - z) * scale.double()[:, at]


def q4(x, values, scale, zero, group, act=None):
    dtype = x.dtype
    xd, K = x.double(), x.shape[1]
    y = xd @ weights(values, scale, zero, group).t()
    at = torch.arange(K, device=x.device) // group
    # a group's sums of x (16 + q) and x (16 + zero), each at most 31 sum |x|
    size = 2 * 31 * (xd.abs() @ scale.double()[:, at].abs().t())
    e = (min(group, K) + scale.shape[1] + 16) * U32 * size
    if act is not None:
        F = y.shape[1] // 2
        g, u, eg, eu = y[:, :F], y[:, F:], e[:, :F], e[:, F:]
        a, _ = activation(act, g)
        ea = SLOPE * eg + STEPS * U32 * (a.abs() + g.abs() * 0.5 + U32)
        y, e = a * u, ea * u.abs() + a.abs() * eu + ea * eu
    return y, e + half_step(dtype) * (y.abs() + e) + tiny(dtype)
