"""Cases that measure the operators that serve a model's tokens: 8-bit products,
a mixture-of-experts layer, and the choice of the next token.

Weights are laid out as in the matrix products here (a row is an output
feature, the contraction runs along it):

* quant: rows of 16-bit values as 8-bit integers with a scale for each row;
* i8: products of 8-bit integers with a scale for each token and each weight
  row, plain or as the gated block; the tokens come as integers, or in 16 bits
  and are made integers on the way;
* moe: a router's choice of top_k experts for each token, the gated blocks of
  these experts, their second products, and the weighted sum;
* sample: one token for each row of logits, from a given random number, with
  temperature, top-k, top-p and min-p.

``run`` computes them in elementary torch operations in 32 bits (64 where a
value next to a border decides), rounded once at the end, or, where ``own`` is
true, through the library.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
TINY = 2.0 ** -126


def listed():
    return [
        # a projection's weights, quantized when a model is loaded: bound by memory
        {"name": "quant_weights", "op": "quant", "type": "bf16", "M": 12288, "K": 4096},
        # some prompts' tokens, rows that start on no alignment
        {"name": "quant_ragged", "op": "quant", "type": "f16", "M": 1021, "K": 1001},
        # a projection of a full batch of prompts: bound by the matrix units
        {"name": "i8_prompt_large", "op": "i8", "type": "bf16", "M": 8192, "N": 8192, "K": 8192, "given": False},
        # the smallest call: one token through a narrow projection, where latency counts
        {"name": "i8_token_small", "op": "i8", "type": "bf16", "M": 1, "N": 1024, "K": 1024, "given": False},
        # several sequences' tokens, already integers, with odd sizes
        {"name": "i8_batch_ragged", "op": "i8", "type": "f16", "M": 13, "N": 11001, "K": 4090, "given": True},
        # a prompt's gated block
        {"name": "i8_gated_prompt", "op": "i8_gated", "type": "f16", "act": "gelu", "M": 2048, "N": 8192, "K": 4096, "given": True},
        # one token through a gated block: bound by the weights' bytes
        {"name": "i8_gated_token", "op": "i8_gated", "type": "bf16", "act": "silu", "M": 1, "N": 12288, "K": 4096, "given": False},
        # the smallest mixture: one token, few narrow experts
        {"name": "moe_token_small", "op": "moe", "type": "bf16", "act": "silu", "M": 1, "D": 1024, "F": 512, "E": 8, "k": 2, "normalize": True},
        # one token, eight of many experts: bound by the chosen experts' bytes
        {"name": "moe_token", "op": "moe", "type": "bf16", "act": "silu", "M": 1, "D": 4096, "F": 1280, "E": 64, "k": 8, "normalize": True},
        # a batch of sequences' tokens that reaches nearly all experts, odd sizes
        {"name": "moe_batch_ragged", "op": "moe", "type": "f16", "act": "gelu", "M": 37, "D": 2050, "F": 1001, "E": 60, "k": 4, "normalize": False},
        # the next token of one sequence from a large vocabulary, where latency counts
        {"name": "sample_token", "op": "sample", "type": "bf16", "M": 1, "V": 131072},
        # a serving batch's next tokens, each sequence with settings of its own, an odd vocabulary
        {"name": "sample_batch", "op": "sample", "type": "f16", "M": 256, "V": 50021},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range; one in three is left odd or ragged."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 256 and rng.random() < 0.67:
        n = max(256, n // 64 * 64)
    return n


def draw(rng):
    op = rng.choice(["quant", "i8", "i8", "i8_gated", "i8_gated", "moe", "moe", "sample", "sample"])
    case = {"op": op, "type": rng.choice(["f16", "bf16"])}
    if op in ("i8_gated", "moe"):
        case["act"] = rng.choice(["silu", "gelu"])
    if op == "quant":
        case.update(M=_size(rng, 1, 8192), K=_size(rng, 64, 8192))
    elif op in ("i8", "i8_gated"):
        # a few sequences' tokens, or whole prompts
        M = _size(rng, 1, 64) if rng.random() < 0.5 else _size(rng, 64, 4096)
        case.update(M=M, N=_size(rng, 256, 8192), K=_size(rng, 128, 8192), given=rng.random() < 0.5)
    elif op == "moe":
        E = rng.choice([4, 8, 16, 60, 64])
        case.update(M=_size(rng, 1, 64), D=_size(rng, 256, 4096), F=_size(rng, 128, 1280), E=E, k=rng.choice([1, 2, min(E, 6), min(E, 8)]),
                    normalize=rng.random() < 0.5)
    else:
        case.update(M=_size(rng, 1, 256), V=_size(rng, 1000, 131072))
    return case


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["type"]]
    op, M = case["op"], case["M"]

    def normal(*shape, scale=1.0, to=torch.float32):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(to)

    def uniform(n, lo, hi):
        return torch.rand(n, generator=gen, device=dev) * (hi - lo) + lo

    def tokens(n):
        """Activations: some channels are several times as large as the others."""
        return (normal(M, n) * torch.exp(0.7 * normal(n))).to(dtype)

    state = {key: case.get(key) for key in ("op", "type", "act", "k", "normalize")}
    if op == "quant":
        state["x"] = tokens(case["K"])
    elif op in ("i8", "i8_gated"):
        K, rows = case["K"], case["N"] * (2 if op == "i8_gated" else 1)
        width = -(-K // 16) * 16  # a row's bytes, padded with zeros
        state["w"] = torch.zeros((rows, width), device=dev, dtype=torch.int8)
        state["w"][:, :K] = (normal(rows, K) * 36.0).round_().clamp_(-127, 127).to(torch.int8)
        state["ws"] = uniform(rows, 0.7, 1.3) * (K ** -0.5 / 36.0)
        state["x"], state["xs"] = tokens(K), None
        if case["given"]:
            q, state["xs"] = _plain_quant(state["x"])
            state["x"] = q
    elif op == "moe":
        D, F, E = case["D"], case["F"], case["E"]
        state["x"] = normal(M, D, to=dtype)
        state["router"] = normal(E, D, scale=1.5 * D ** -0.5, to=dtype)
        state["w"] = normal(E, 2 * F, D, scale=D ** -0.5, to=dtype)
        state["down"] = normal(E, D, F, scale=2.0 * F ** -0.5, to=dtype)
    else:
        V = case["V"]
        # a model's logits: most tokens improbable, a few that lead
        state["logits"] = (normal(M, V, scale=2.0) + 6.0 * (torch.rand((M, V), generator=gen, device=dev) < 20.0 / V)).to(dtype)
        state["u"] = torch.rand(M, generator=gen, device=dev)
        kind = torch.rand((4, M), generator=gen, device=dev)
        # one sequence in eight is greedy; of the others each setting is off for one in four
        state["temperature"] = torch.where(kind[0] < 0.125, torch.zeros_like(kind[0]), uniform(M, 0.5, 1.5))
        state["top_k"] = torch.where(kind[1] < 0.25, torch.zeros_like(kind[1]), uniform(M, 1, 200)).to(torch.int32)
        state["top_p"] = torch.where(kind[2] < 0.25, torch.ones_like(kind[2]), uniform(M, 0.5, 1.0))
        state["min_p"] = torch.where(kind[3] < 0.25, torch.zeros_like(kind[3]), uniform(M, 0.0, 0.1))
    return state


def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    t = torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t)


def _plain_quant(x):
    M, K = x.shape
    scale = (x.abs().amax(dim=1).double() / 127.0).clamp(min=TINY).float()
    q = torch.zeros((M, -(-K // 16) * 16), device=x.device, dtype=torch.int8)
    q[:, :K] = torch.round(x.double() / scale.double()[:, None]).to(torch.int8)
    return q, scale


def _plain_i8(state):
    q, scale = _plain_quant(state["x"]) if state["xs"] is None else (state["x"], state["xs"])
    y = (q.float() @ state["w"].float().t()) * scale[:, None] * state["ws"]
    if state["op"] == "i8_gated":
        N = y.shape[1] // 2
        y = _act(state["act"], y[:, :N]) * y[:, N:]
    return {"y": y.to(TYPES[state["type"]])}


def _plain_route(state):
    """The chosen experts of each token, the largest logit first and the lowest index where they are equal, and their weights."""
    logits = state["x"].double() @ state["router"].double().t()
    by, at = torch.sort(logits, dim=1, descending=True, stable=True)
    k = state["k"]
    e = torch.exp(by - by[:, :1])
    total = (e[:, :k] if state["normalize"] else e).sum(dim=1, keepdim=True)
    return at[:, :k], (e[:, :k] / total).float()


def _plain_moe(state):
    x, w, down, k = state["x"], state["w"], state["down"], state["k"]
    (M, D), (E, _, F) = x.shape, down.shape
    experts, weights = _plain_route(state)
    if M * k < E:  # the chosen experts' weights alone
        at = experts.reshape(-1)
        rows = x.float().repeat_interleave(k, 0)[:, :, None]
        y = torch.bmm(w[at].float(), rows)[:, :, 0]
        h = _act(state["act"], y[:, :F]) * y[:, F:]
        y = torch.bmm(down[at].float(), h[:, :, None])[:, :, 0].view(M, k, D)
        y = (y * weights[:, :, None]).sum(dim=1)
    else:  # every expert on every token, with a weight of zero where it is not chosen
        p = torch.zeros((M, E), device=x.device).scatter_(1, experts, weights)
        y = (x.float() @ w.view(-1, D).float().t()).view(M, E, 2 * F)
        h = _act(state["act"], y[:, :, :F]) * y[:, :, F:] * p[:, :, None]
        y = h.reshape(M, E * F) @ down.transpose(1, 2).reshape(E * F, D).float()
    return {"y": y.to(x.dtype), "experts": experts.to(torch.int32), "weights": weights}


def _plain_sample(state):
    z, V = state["logits"].double(), state["logits"].shape[1]
    by, at = torch.sort(z, dim=1, descending=True, stable=True)
    t = state["temperature"].double()[:, None]
    p = torch.exp((by - by[:, :1]) / torch.where(t > 0, t, torch.ones_like(t)))
    rank = torch.arange(V, device=z.device)
    k = state["top_k"].long()[:, None]
    keep = (rank < torch.where(k > 0, k, V)) & (p >= state["min_p"].double()[:, None])
    p = torch.where(rank < torch.where(k > 0, k, V), p, torch.zeros_like(p))
    run = p.cumsum(dim=1)
    top_p = state["top_p"].double()[:, None]
    keep &= (top_p >= 1) | (run - p < top_p * run[:, -1:])
    keep &= (t > 0) | (rank == 0)
    keep[:, 0] = True
    run = torch.where(keep, p, torch.zeros_like(p)).cumsum(dim=1)
    n = (run <= state["u"].double()[:, None] * run[:, -1:]).sum(dim=1)
    n = torch.minimum(n, keep.sum(dim=1) - 1)
    return {"token": at.gather(1, n[:, None])[:, 0]}


def _own(state):
    from software_pipelined_tiled_pipeline_amd import pgemm

    op, fmt = state["op"], state["type"]

    def call(name, *args, **more):
        return getattr(pgemm, f"pgemm_{fmt}_{name}")(*args, **more)

    if op == "quant":
        q, scale = call("quant_i8", state["x"])
        return {"q": q, "scale": scale}
    if op == "i8":
        return {"y": call("i8", state["x"], state["w"], state["ws"], xs=state["xs"])}
    if op == "i8_gated":
        return {"y": call("i8_gated", state["x"], state["w"], state["ws"], xs=state["xs"], act=state["act"])}
    if op == "moe":
        y, experts, weights = call("moe", state["x"], state["router"], state["w"], state["down"], state["k"], act=state["act"],
                                   normalize=state["normalize"], routing=True)
        return {"y": y, "experts": experts, "weights": weights}
    return {"token": call("sample", state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                          top_p=state["top_p"], min_p=state["min_p"])}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "quant":
        q, scale = _plain_quant(state["x"])
        return {"q": q, "scale": scale}
    if state["op"] == "moe":
        return _plain_moe(state)
    if state["op"] == "sample":
        return _plain_sample(state)
    return _plain_i8(state)


def work(case):
    """Inputs read once (of the experts those that so many choices reach on average), outputs written once, and the products."""
    op, M = case["op"], case["M"]
    if op == "quant":
        return {"bytes": 3 * M * case["K"] + 4 * M, "flops": 2 * M * case["K"]}
    if op in ("i8", "i8_gated"):
        N, K = case["N"], case["K"]
        rows = 2 * N if op == "i8_gated" else N
        return {"bytes": rows * (K + 4) + M * K * (1 if case["given"] else 2) + 2 * M * N, "flops": 2 * M * rows * K}
    if op == "moe":
        D, F, E, k = case["D"], case["F"], case["E"], case["k"]
        reached = E * (1.0 - (1.0 - k / E) ** M)
        return {"bytes": int(reached * 6 * F * D) + 2 * E * D + 4 * M * D + 8 * M * k, "flops": 2 * M * (3 * k * F * D + E * D)}
    return {"bytes": 2 * M * case["V"] + 28 * M, "flops": 4 * M * case["V"]}


def exact(case, seed):
    """The definitions in 64 bits, expert by expert and in blocks of weight rows."""
    state = prepare(case, seed)
    op, M = case["op"], case["M"]

    def activation(g):
        if case["act"] == "silu":
            return g * 0.5 * (1.0 + torch.tanh(0.5 * g))
        return g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))  # (1 + tanh(a)) / 2 = sigmoid(2 a)

    if op == "quant":
        top = state["x"].double().abs().max(dim=1).values
        return {"q": None, "scale": torch.maximum(top / 127.0, torch.full_like(top, TINY))}
    if op in ("i8", "i8_gated"):
        x = state["x"].double()
        if state["xs"] is None:
            # a rounded scale decides which integers its row gets
            scale = torch.maximum(x.abs().max(dim=1).values / 127.0, torch.full((M,), TINY, device=x.device, dtype=torch.float64)).float().double()
            x = torch.round(x / scale[:, None])
        else:
            scale = state["xs"].double()
        x = x[:, :case["K"]]
        y = torch.empty((M, state["w"].shape[0]), dtype=torch.float64, device=x.device)
        for n in range(0, y.shape[1], 4096):
            y[:, n:n + 4096] = torch.matmul(x, state["w"][n:n + 4096, :case["K"]].double().T)
        y = y * scale[:, None] * state["ws"].double()[None, :]
        if op == "i8_gated":
            gate, up = torch.chunk(y, 2, dim=1)
            y = activation(gate) * up
        return {"y": y}
    if op == "moe":
        x, F, k = state["x"].double(), case["F"], case["k"]
        logits = torch.matmul(x, state["router"].double().T)
        left, chosen = logits.clone(), []
        for _ in range(k):
            chosen.append(left.argmax(dim=1))
            left[torch.arange(M, device=x.device), chosen[-1]] = -math.inf
        chosen = torch.stack(chosen, dim=1)
        over = torch.logsumexp(logits.gather(1, chosen) if case["normalize"] else logits, dim=1)
        p = torch.exp(logits.gather(1, chosen) - over[:, None])
        y = torch.zeros_like(x)
        for e in range(case["E"]):
            row, place = torch.nonzero(chosen == e, as_tuple=True)
            if len(row) == 0:
                continue
            both = torch.matmul(x[row], state["w"][e].double().T)
            h = activation(both[:, :F]) * both[:, F:]
            y[row] += p[row, place][:, None] * torch.matmul(h, state["down"][e].double().T)
        return {"y": y, "experts": None, "weights": p}
    return None  # whole numbers
