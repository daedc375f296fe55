"""Trains a small next-token model on the fused operators, then serves it with 4-bit or 8-bit weights.

    python examples/gated_lm.py [--steps 60] [--vocab 4000] [--bits 8] [--temperature 0.7]

The model is an embedding, one gated feed-forward block and a vocabulary head:

    h = silu(e[token] Wg^T) * (e[token] Wu^T),   logits = h Wh^T

It learns a fixed successor of every token.  A training step runs the block
(pgemm_bf16_gated, keeping its projections), the loss over the vocabulary without
its logits (pgemm_bf16_xent) and both gradients; the optimizer keeps fp32 weights.
Serving quantizes the block and the head to 4 bits with a scale and a zero point
per group of 32 and decodes token by token with pgemm_bf16_q4_gated and
pgemm_bf16_q4; or to 8 bits with a scale per row (pgemm_bf16_quant_i8), for
pgemm_bf16_i8_gated and pgemm_bf16_i8.  pgemm_bf16_sample takes the next token:
the likeliest one at temperature 0.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from software_pipelined_tiled_pipeline_amd import pgemm  # noqa: E402

GROUP = 32


class GatedBlock(torch.autograd.Function):
    """h = silu(x Wg^T) * (x Wu^T) for w = [Wg; Wu]."""

    @staticmethod
    def forward(ctx, x, w):
        h, saved = pgemm.pgemm_bf16_gated(x, w, save=True)
        ctx.save_for_backward(x, w, saved)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, w, saved = ctx.saved_tensors
        return pgemm.pgemm_bf16_gated_bwd(dh.contiguous(), x, w, saved=saved)


class VocabularyLoss(torch.autograd.Function):
    """Cross entropy per token of the logits h w^T."""

    @staticmethod
    def forward(ctx, h, w, target):
        loss, lse = pgemm.pgemm_bf16_xent(h, w, target)
        ctx.save_for_backward(h, w, target, lse)
        return loss

    @staticmethod
    def backward(ctx, dloss):
        h, w, target, lse = ctx.saved_tensors
        dh, dw = pgemm.pgemm_bf16_xent_bwd(dloss, h, w, target, lse)
        return dh, dw, None


def quantize(w):
    """4-bit weights of w [N, K]: packed values, scales and zero points per group of a row."""
    N, K = w.shape
    g = w.float().view(N, K // GROUP, GROUP)
    low, high = g.amin(2).clamp(max=0), g.amax(2).clamp(min=0)
    scale = ((high - low) / 15).clamp(min=1e-8).bfloat16()
    zero = (-low / scale.float()).round().clamp(0, 15)
    values = (g / scale.float()[:, :, None] + zero[:, :, None]).round().clamp(0, 15)
    return pgemm.pack_q4(values.view(N, K).to(torch.uint8)), scale, zero.to(torch.uint8)


def train(vocab, width, hidden, tokens, steps, seed=0, report=10):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    successor = torch.randperm(vocab, generator=gen, device="cuda")

    def weight(n, k):
        return (torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5).requires_grad_()
    params = embed, block, head = weight(vocab, width), weight(2 * hidden, width), weight(vocab, hidden)
    with torch.no_grad():
        embed.mul_(width ** 0.5)
    adam = torch.optim.Adam(params, lr=3e-3)
    losses = []
    for step in range(steps):
        token = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        h = GatedBlock.apply(embed[token].bfloat16(), block.bfloat16())
        loss = VocabularyLoss.apply(h, head.bfloat16(), successor[token]).mean()
        adam.zero_grad()
        loss.backward()
        adam.step()
        losses.append(loss.detach())
        if report and step % report == 0:
            print(f"step {step}: loss {loss.item():.3f}", flush=True)
    return successor, embed, block, head, [x.item() for x in losses]


def serve(embed, block, head, first, count, bits=4, temperature=0.0, seed=0):
    """`count` tokens after each of `first`, the likeliest one every time at temperature 0."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.tensor(temperature, device="cuda")
    e = embed.bfloat16()
    if bits == 4:
        b, h = quantize(block), quantize(head)
    else:
        b, h = (pgemm.pgemm_bf16_quant_i8(w.bfloat16()) for w in (block, head))
    token, out = first, []
    for _ in range(count):
        if bits == 4:
            y = pgemm.pgemm_bf16_q4_gated(e[token], *b, group=GROUP)
            z = pgemm.pgemm_bf16_q4(y, *h, group=GROUP)
        else:
            y = pgemm.pgemm_bf16_i8_gated(e[token], *b)
            z = pgemm.pgemm_bf16_i8(y, *h)
        u = torch.rand(len(token), generator=gen, device="cuda")
        token = pgemm.pgemm_bf16_sample(z, u, temperature=t)
        out.append(token)
    return torch.stack(out, 1)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--vocab", type=int, default=4000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--bits", type=int, choices=(4, 8), default=4)
    ap.add_argument("--temperature", type=float, default=0.0)
    a = ap.parse_args(argv)
    successor, embed, block, head, losses = train(a.vocab, a.width, a.hidden, a.tokens, a.steps)
    first = torch.arange(8, device="cuda") * (a.vocab // 8)
    with torch.no_grad():
        got = serve(embed, block, head, first, 16, a.bits, a.temperature)
    want, token = [], first
    for _ in range(16):
        token = successor[token]
        want.append(token)
    right = (got == torch.stack(want, 1)).float().mean().item()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; {a.bits}-bit decoding: {100 * right:.0f} % of the tokens right")
    return losses, right


if __name__ == "__main__":
    main()
