#!/usr/bin/env python3
"""Trains the last part of a language model on synthetic tokens, then scores with it.

A step runs, on one handle and one stream:

    u = a @ proj^T                               the GEMM (a block's last projection)
    h = residual + dropout(u);  y = norm(h)      add_rms_norm
    loss = cross entropy of y @ head^T           linear_cross_entropy (a third of the tokens ignored)
    dy, dhead                                    linear_cross_entropy_backward
    du, dresidual, dnorm                         add_rms_norm_backward

and a plain gradient step on `head` and the norm's weight. Afterwards it scores single tokens
(without dropout) and writes the norm in 8 bits, as a server would.

    python examples/lm_head_step.py [--steps N] [--tokens T] [--hidden H] [--vocab V]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from async_pipelines_gb300 import gemm_ws  # noqa: E402

IGNORE = -100


class Head:
    """The weights, and the buffers of a step of `tokens` tokens."""

    def __init__(self, g, tokens, hidden, vocab, seed=0):
        self.g, self.tokens, self.hidden, self.vocab = g, tokens, hidden, vocab
        gen = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16()

        self.proj = normal(1, hidden, hidden, scale=hidden ** -0.5)
        self.head = normal(vocab, hidden, scale=0.02)
        self.norm = torch.ones(hidden, device="cuda", dtype=torch.bfloat16)
        # full-precision copies that the steps accumulate in
        self.head32, self.norm32 = self.head.float(), self.norm.float()
        bf16 = dict(device="cuda", dtype=torch.bfloat16)
        self.u = torch.empty(1, tokens, hidden, **bf16)
        self.h, self.y, self.dy, self.du, self.dresidual = (torch.empty(tokens, hidden, **bf16)
                                                            for _ in range(5))
        self.dhead, self.dnorm = torch.empty_like(self.head), torch.empty_like(self.norm)
        self.rstd, self.loss, self.lse = (torch.empty(tokens, device="cuda") for _ in range(3))
        self.mean = torch.empty(2, device="cuda")
        need = max(g.linear_cross_entropy_workspace(tokens, hidden, vocab, b) for b in (False, True))
        self.workspace = torch.empty(need, dtype=torch.uint8, device="cuda")

    def forward(self, a, residual, targets, p=0.0, rng=None):
        g = self.g
        g.run(a[None], self.proj, None, self.u)
        g.add_rms_norm(self.u[0], self.norm, self.y, residual=residual, h=self.h, rstd=self.rstd,
                       p=p, rng=rng)
        g.linear_cross_entropy(self.y, self.head, targets, self.loss, self.lse, mean=self.mean,
                               ignore_index=IGNORE, workspace=self.workspace)

    def backward(self, targets, p=0.0, rng=None):
        g = self.g
        g.linear_cross_entropy_backward(self.y, self.head, targets, self.lse, self.mean[1:],
                                        dx=self.dy, dweight=self.dhead, ignore_index=IGNORE,
                                        workspace=self.workspace)
        g.add_rms_norm_backward(self.dy, self.h, self.norm, self.rstd, self.du, self.dnorm,
                                dresidual=self.dresidual, p=p, rng=rng)

    def update(self, rate):
        self.head32 -= rate * self.dhead
        self.norm32 -= rate * self.dnorm
        self.head.copy_(self.head32)
        self.norm.copy_(self.norm32)


def train(steps=30, tokens=1024, hidden=512, vocab=5000, rate=20.0, p=0.1, seed=0):
    """Returns the mean losses of the steps, and what the scoring at the end found."""
    g = gemm_ws.GemmWS(0)
    m = Head(g, tokens, hidden, vocab, seed)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    targets = torch.randint(vocab, (tokens,), device="cuda", generator=gen)
    targets[torch.rand(tokens, device="cuda", generator=gen) < 1 / 3] = IGNORE
    a, residual = (torch.randn(tokens, hidden, device="cuda", generator=gen).bfloat16() for _ in range(2))
    rng = torch.tensor([seed + 7, 0], device="cuda")
    losses = []
    for _ in range(steps):
        m.forward(a, residual, targets, p, rng)
        m.backward(targets, p, rng)
        m.update(rate)
        rng[1] += tokens * ((hidden + 7) // 8)   # the next step's mask
        losses.append(float(m.mean[0]))

    # Scoring: all tokens at once, then some of them one by one.
    m.forward(a, residual, targets)
    batch = m.loss.clone()
    one = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    worst = 0.0
    for i in range(0, tokens, max(1, tokens // 16)):
        g.linear_cross_entropy(m.y[i:i + 1], m.head, targets[i:i + 1], *one, ignore_index=IGNORE)
        worst = max(worst, float((one[0] - batch[i]).abs()))
    # The norm in 8 bits, a scale for each 128 columns.
    y8 = torch.empty(tokens, hidden, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(tokens, (hidden + 127) // 128, device="cuda")
    g.add_rms_norm(m.u[0], m.norm, y8, residual=residual, scales=scales)
    back = y8.float() * scales.repeat_interleave(128, 1)[:, :hidden]
    off8 = float((back - m.y.float()).norm() / m.y.float().norm())
    assert g.query_status() == gemm_ws.OK
    g.close()
    return losses, {"single_token_difference": worst, "norm_8bit_relative_difference": off8}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=5000)
    a = ap.parse_args()
    losses, found = train(a.steps, a.tokens, a.hidden, a.vocab)
    print(f"ln(vocab) = {math.log(a.vocab):.4f}")
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.4f}")
    for k, v in found.items():
        print(f"{k} = {v:.3g}")


if __name__ == "__main__":
    main()
