"""A vocabulary head's life on one GPU: trained, stepped, quantised, served.

The head of a tiny language model, W (vocabulary x width), and the embedding
that feeds it learn a fixed next-token rule.  Each training step takes the
softmax cross entropy of H W^T and its gradient without the logits in memory
(``os2.XentFunction``) and one AdamW step over both tensors with 8-bit moments
(``os2.adamw``).  The trained head is then quantised to 8 bits, one scale an
output channel (``os2.quantize_rows``), and serves single tokens through the
8-bit product (``os2.i8linear``).

    python examples/vocab_head.py [--steps 200] [--vocab 1000] [--width 128]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rns_emulated_fp64_gb300 as os2  # noqa: E402

IGNORE = -100


class Tensor8bit:
    """A parameter in BF16 with its 8-bit moments."""

    def __init__(self, value):
        n = value.numel()
        blocks = -(-n // os2.ADAMW_BLOCK)
        self.p = value.bfloat16().requires_grad_(True)
        self.m = torch.zeros(value.shape, dtype=torch.int8, device=value.device)
        self.v = torch.zeros(value.shape, dtype=torch.uint8, device=value.device)
        self.m_scale = torch.zeros(blocks, device=value.device)
        self.v_scale = torch.zeros(blocks, device=value.device)


def step(tensors, number, lr):
    os2.adamw([t.p.detach() for t in tensors], [t.p.grad for t in tensors], [t.m for t in tensors],
              [t.v for t in tensors], step=number, lr=lr, beta1=0.9, beta2=0.95, weight_decay=0.01,
              exp_avg_scales=[t.m_scale for t in tensors],
              exp_avg_sq_scales=[t.v_scale for t in tensors])
    for t in tensors:
        t.p.grad = None


def train(steps=200, vocab=1000, width=128, batch=512, lr=1e-2, seed=0):
    """Returns (embedding, head, losses, the rule: token -> next token)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rule = torch.randperm(vocab, generator=g, device="cuda")
    emb = Tensor8bit(torch.randn(vocab, width, generator=g, device="cuda"))
    head = Tensor8bit(torch.randn(vocab, width, generator=g, device="cuda") * width ** -0.5)
    losses = []
    for i in range(1, steps + 1):
        tokens = torch.randint(0, vocab, (batch,), generator=g, device="cuda")
        labels = rule[tokens]
        labels[torch.rand(batch, generator=g, device="cuda") < 0.2] = IGNORE  # a prompt's positions
        h = torch.nn.functional.embedding(tokens, emb.p)
        loss = os2.XentFunction.apply(h, head.p, labels, IGNORE).sum() / (labels != IGNORE).sum()
        loss.backward()
        step([emb, head], i, lr)
        losses.append(loss.detach())
    return emb.p.detach(), head.p.detach(), torch.stack(losses).tolist(), rule


def serve(emb, head, tokens):
    """The next token of each, one at a time, through the 8-bit head."""
    q, scale = os2.quantize_rows(head)
    out = [os2.i8linear(emb[t:t + 1], q, scale, out_dtype=torch.float32).argmax(1) for t in tokens.tolist()]
    return torch.cat(out)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--width", type=int, default=128)
    a = ap.parse_args(argv)
    emb, head, losses, rule = train(a.steps, a.vocab, a.width)
    tokens = torch.arange(min(200, a.vocab), device="cuda")
    right = (serve(emb, head, tokens) == rule[tokens]).float().mean().item()
    status = os2.get_status()
    if status:
        raise SystemExit(f"device status {status}: {os2.status_string(status)}")
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; the 8-bit head serves {100 * right:.0f} % right")
    return losses, right


if __name__ == "__main__":
    main()
