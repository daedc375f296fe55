"""Cases that measure the fused operators around a model's feed-forward block and its loss.

Three operators, each with the weights' layout of the matrix products here
(rows are output features, the contraction runs along a row):

* gated: h = act(x Wg^T) * (x Wu^T), both projections' weights in one tensor
  (the F gate rows, then the F up rows), and its gradients;
* xent: per-row softmax cross entropy of the logits x W^T, which are never
  kept, and its gradients;
* q4: products with 4-bit weights that share a scale (and a zero point) per
  group of a row, plain or as the gated block.

``run`` computes them in elementary torch operations in 32 bits, rounded
once at the end, or, where ``own`` is true, through the library.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100


def listed():
    return [
        # a training step of a block on a full batch of tokens: bound by the matrix units
        {"name": "gated_train_large", "op": "gated_train", "type": "bf16", "act": "silu", "M": 8192, "D": 4096, "F": 12288},
        # a training step with no size that suits a tile or an alignment
        {"name": "gated_train_ragged", "op": "gated_train", "type": "f16", "act": "gelu", "M": 4095, "D": 1001, "F": 2731},
        # a prompt's block when serving
        {"name": "gated_prompt", "op": "gated", "type": "bf16", "act": "silu", "M": 2048, "D": 4096, "F": 8192},
        # the block for one new token: bound by the weights' bytes
        {"name": "gated_token", "op": "gated", "type": "bf16", "act": "silu", "M": 1, "D": 4096, "F": 12288},
        # a training step's loss and gradients over a large vocabulary
        {"name": "xent_train_large", "op": "xent_train", "type": "bf16", "M": 8192, "D": 4096, "V": 65536},
        # the same with odd sizes in the narrower type
        {"name": "xent_train_ragged", "op": "xent_train", "type": "f16", "M": 1021, "D": 1000, "V": 50021},
        # scoring text: the loss alone
        {"name": "xent_score", "op": "xent", "type": "bf16", "M": 2048, "D": 2048, "V": 131072},
        # the smallest call: one token through a narrow projection, where latency counts
        {"name": "q4_token_small", "op": "q4", "type": "bf16", "M": 1, "K": 1024, "N": 1024, "group": 128, "zero": False},
        # one token through a wide projection
        {"name": "q4_token", "op": "q4", "type": "bf16", "M": 1, "K": 8192, "N": 8192, "group": 128, "zero": True},
        # several sequences' tokens at once, with odd sizes
        {"name": "q4_batch_ragged", "op": "q4", "type": "f16", "M": 13, "K": 4090, "N": 11001, "group": 64, "zero": True},
        # one token through the whole gated block
        {"name": "q4_gated_token", "op": "q4_gated", "type": "f16", "act": "silu", "M": 1, "K": 4096, "N": 12288, "group": 64, "zero": False},
        # a batch of tokens through it, with the finest groups
        {"name": "q4_gated_batch", "op": "q4_gated", "type": "bf16", "act": "gelu", "M": 48, "K": 4096, "N": 12288, "group": 32, "zero": True},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range; one in three is left odd or ragged."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 256 and rng.random() < 0.67:
        n = max(256, n // 64 * 64)
    return n


def draw(rng):
    op = rng.choice(["gated_train", "gated", "xent_train", "xent", "q4", "q4_gated"])
    case = {"op": op, "type": rng.choice(["f16", "bf16"])}
    if op.startswith("gated") or op == "q4_gated":
        case["act"] = rng.choice(["silu", "gelu"])
    if op == "gated_train":
        case.update(M=_size(rng, 128, 8192), D=_size(rng, 256, 4096), F=_size(rng, 256, 12288))
    elif op == "gated":
        case.update(M=_size(rng, 1, 4096), D=_size(rng, 256, 4096), F=_size(rng, 256, 12288))
    elif op.startswith("xent"):
        case.update(M=_size(rng, 64, 4096), D=_size(rng, 256, 4096), V=_size(rng, 4000, 131072))
    else:
        case.update(M=_size(rng, 1, 64), K=_size(rng, 256, 8192), N=_size(rng, 256, 12288), group=rng.choice([32, 64, 128]),
                    zero=rng.random() < 0.5)
    return case


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["type"]]
    op, M = case["op"], case["M"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale)

    state = {"op": op, "type": case["type"], "act": case.get("act")}
    if op in ("gated", "gated_train"):
        D, F = case["D"], case["F"]
        # normalised activations, weights that keep their variance
        state["x"] = normal(M, D).to(dtype)
        state["w"] = normal(2 * F, D, scale=D ** -0.5).to(dtype)
        if op == "gated_train":
            state["dh"] = normal(M, F, scale=0.02).to(dtype)
    elif op in ("xent", "xent_train"):
        D, V = case["D"], case["V"]
        w = normal(V, D, scale=2.0 * D ** -0.5)
        target = torch.randint(0, V, (M,), generator=gen, device=dev)
        # a model that has learnt something: activations lean towards their target's row, by different amounts
        lean = torch.rand((M, 1), generator=gen, device=dev) * 3.0
        state["x"] = (normal(M, D) + lean * w[target] * 0.5).to(dtype)
        state["w"] = w.to(dtype)
        # padding and prompts do not count
        state["target"] = torch.where(torch.rand(M, generator=gen, device=dev) < 0.06, torch.full_like(target, IGNORE), target)
        if op == "xent_train":
            # the mean over the counted tokens, with the loss scaled up as training in the narrower type needs
            count = (state["target"] != IGNORE).sum().clamp(min=1)
            state["dloss"] = (torch.ones(M, device=dev) * 1024.0 / count).float()
    else:
        K, N, group = case["K"], case["N"], case["group"]
        rows = 2 * N if op == "q4_gated" else N
        groups = -(-K // group)
        state["x"] = normal(M, K).to(dtype)
        width = -(-K // 32) * 16  # bytes of a row: two weights a byte, rows padded to 16 bytes
        state["q"] = torch.randint(0, 256, (rows, width), generator=gen, device=dev, dtype=torch.uint8)
        spread = 0.7 + 0.6 * torch.rand((rows, groups), generator=gen, device=dev)
        state["scale"] = (spread * (K ** -0.5) / 4.6).to(dtype)
        state["zero"] = torch.randint(5, 11, (rows, groups), generator=gen, device=dev, dtype=torch.uint8) if case["zero"] else None
        state["group"] = group
    return state


def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    t = torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t)


def _act_slope(name, g):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_gated(state):
    x, w = state["x"].float(), state["w"].float()
    F = w.shape[0] // 2
    g, u = x @ w[:F].t(), x @ w[F:].t()
    h = (_act(state["act"], g) * u).to(state["x"].dtype)
    if "dh" not in state:
        return {"h": h}
    dh = state["dh"].float()
    du = dh * _act(state["act"], g)
    dg = dh * u * _act_slope(state["act"], g)
    dx = dg @ w[:F] + du @ w[F:]
    dw = torch.cat([dg.t() @ x, du.t() @ x])
    return {"h": h, "dx": dx.to(h.dtype), "dw": dw.to(h.dtype)}


def _plain_xent(state):
    x, w, target = state["x"].float(), state["w"].float(), state["target"]
    z = x @ w.t()
    top = z.max(dim=1).values
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(dim=1))
    counts = target != IGNORE
    at = torch.where(counts, target, torch.zeros_like(target))
    loss = torch.where(counts, lse - z.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    if "dloss" not in state:
        return {"loss": loss, "lse": lse}
    s = torch.where(counts, state["dloss"], torch.zeros_like(lse))
    dz = torch.exp(z - lse[:, None])
    dz.scatter_add_(1, at[:, None], torch.full_like(lse, -1.0)[:, None])
    dz *= s[:, None]
    return {"loss": loss, "lse": lse, "dx": (dz @ w).to(state["x"].dtype), "dw": (dz.t() @ x).to(state["x"].dtype)}


def _plain_weights(state):
    """The 4-bit weights' values [rows, K] in 32 bits."""
    q, K, group = state["q"], state["x"].shape[1], state["group"]
    v = torch.stack([q & 15, q >> 4], dim=2).reshape(q.shape[0], -1)[:, :K].float()
    at = torch.arange(K, device=q.device) // group
    zero = 8.0 if state["zero"] is None else state["zero"].float()[:, at]
    return (v - zero) * state["scale"].float()[:, at]


def _plain_q4(state):
    y = state["x"].float() @ _plain_weights(state).t()
    if state["op"] == "q4_gated":
        F = y.shape[1] // 2
        y = _act(state["act"], y[:, :F]) * y[:, F:]
    return {"y": y.to(state["x"].dtype)}


def _own(state):
    from software_pipelined_tiled_pipeline_amd import pgemm

    op, fmt = state["op"], state["type"]

    def call(name, *args, **more):
        return getattr(pgemm, f"pgemm_{fmt}_{name}")(*args, **more)

    if op == "gated":
        return {"h": call("gated", state["x"], state["w"], act=state["act"])}
    if op == "gated_train":
        h, saved = call("gated", state["x"], state["w"], act=state["act"], save=True)
        dx, dw = call("gated_bwd", state["dh"], state["x"], state["w"], saved=saved, act=state["act"])
        return {"h": h, "dx": dx, "dw": dw}
    if op in ("xent", "xent_train"):
        loss, lse = call("xent", state["x"], state["w"], state["target"], ignore_index=IGNORE)
        if op == "xent":
            return {"loss": loss, "lse": lse}
        dx, dw = call("xent_bwd", state["dloss"], state["x"], state["w"], state["target"], lse, ignore_index=IGNORE)
        return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
    if op == "q4":
        return {"y": call("q4", state["x"], state["q"], state["scale"], state["zero"], group=state["group"])}
    return {"y": call("q4_gated", state["x"], state["q"], state["scale"], state["zero"], group=state["group"], act=state["act"])}


def run(state):
    if own:
        return _own(state)
    if state["op"].startswith("gated"):
        return _plain_gated(state)
    if state["op"].startswith("xent"):
        return _plain_xent(state)
    return _plain_q4(state)


def work(case):
    """Inputs read once, outputs written once, and the products that the definition has."""
    op, M = case["op"], case["M"]
    if op in ("gated", "gated_train"):
        D, F = case["D"], case["F"]
        if op == "gated":
            return {"bytes": 2 * (M * D + 2 * F * D + M * F), "flops": 4 * M * D * F}
        return {"bytes": 2 * (2 * M * D + 4 * F * D + 2 * M * F), "flops": 12 * M * D * F}
    if op in ("xent", "xent_train"):
        D, V = case["D"], case["V"]
        if op == "xent":
            return {"bytes": 2 * (M * D + V * D) + 16 * M, "flops": 2 * M * D * V}
        return {"bytes": 4 * (M * D + V * D) + 20 * M, "flops": 6 * M * D * V}
    K, N = case["K"], case["N"]
    rows = 2 * N if op == "q4_gated" else N
    groups = -(-K // case["group"])
    return {"bytes": rows * (-(-K // 32) * 16) + rows * groups * (3 if case["zero"] else 2) + 2 * M * K + 2 * M * N,
            "flops": 2 * M * rows * K}


def exact(case, seed):
    """The definitions in 64 bits, with derivatives of the block by way of the tanh and logistic functions' own."""
    state = prepare(case, seed)
    op = case["op"]
    x = state["x"].double()

    def activation(g):  # value and derivative
        if case["act"] == "silu":
            s = 0.5 * (1.0 + torch.tanh(0.5 * g))
            return g * s, s + g * s * (1.0 - s)
        c = math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(2.0 * c * (g + 0.044715 * g ** 3))  # (1 + tanh(a)) / 2 = sigmoid(2 a)
        return g * s, s + g * s * (1.0 - s) * 2.0 * c * (1.0 + 0.134145 * g ** 2)

    if op in ("gated", "gated_train"):
        w = state["w"].double()
        gate, up = torch.chunk(torch.matmul(x, w.T), 2, dim=1)
        a, slope = activation(gate)
        out = {"h": a * up}
        if op == "gated_train":
            dh = state["dh"].double()
            d = torch.cat([slope.mul_(up).mul_(dh), a.mul_(dh)], dim=1)
            out["h"] = out["h"].clone()
            out["dx"] = torch.matmul(d, w)
            out["dw"] = torch.matmul(d.T.contiguous(), x)
        return out
    if op in ("xent", "xent_train"):
        w, target = state["w"].double(), state["target"]
        z = torch.matmul(x, w.T)
        lse = torch.logsumexp(z, dim=1)
        valid = torch.nonzero(target != IGNORE)[:, 0]
        loss = torch.zeros_like(lse)
        loss[valid] = lse[valid] - z[valid, target[valid]]
        out = {"loss": loss, "lse": lse}
        if op == "xent_train":
            z.sub_(lse[:, None]).exp_()
            z[valid, target[valid]] -= 1.0
            weight = torch.zeros_like(lse)
            weight[valid] = state["dloss"].double()[valid]
            z.mul_(weight[:, None])
            out["dx"] = torch.matmul(z, w)
            out["dw"] = torch.matmul(z.T.contiguous(), x)
        return out
    M, K, group = case["M"], case["K"], case["group"]
    rows = state["q"].shape[0]
    groups = -(-K // group)
    low, high = state["q"].long() % 16, state["q"].long() // 16
    v = torch.empty((rows, 2 * low.shape[1]), dtype=torch.float64, device=x.device)
    v[:, 0::2], v[:, 1::2] = low.double(), high.double()
    y = torch.zeros((M, rows), dtype=torch.float64, device=x.device)
    for k in range(groups):  # one group of every row after the other
        a, b = k * group, min(K, (k + 1) * group)
        zero = 8.0 if state["zero"] is None else state["zero"][:, k:k + 1].double()
        y += torch.matmul(x[:, a:b], (v[:, a:b] - zero).T) * state["scale"][:, k].double()
    if op == "q4_gated":
        gate, up = torch.chunk(y, 2, dim=1)
        y = activation(gate)[0] * up
    return {"y": y}
