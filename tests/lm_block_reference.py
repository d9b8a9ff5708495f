"""Plain implementations in 64 bits of the operators around a block and of serving in 8-bit integers, for the tests.

They follow the formulas of include/gemm_ws_lm.h and share no code with the library.
"""
from __future__ import annotations

import math

import torch


def _norm(v, eps):
    return 1.0 / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + eps)


def block_norm(x, residual, weight, post=None, gate=None, alpha=1.0, eps=1e-6):
    """h, y and the two inverse roots in 64 bits, and the sums of magnitudes that h's error goes by."""
    x, weight = x.double(), weight.double()
    r1 = torch.ones(len(x), 1, dtype=torch.float64) if post is None else _norm(x, eps)
    b = x * r1
    if post is not None:
        b = b * post.double()
    if gate is not None:
        b = b * gate.double()
    h = alpha * residual.double() + b
    r2 = _norm(h, eps)
    return h, h * r2 * weight, r1[:, 0], r2[:, 0], abs(alpha) * residual.double().abs() + b.abs()


def block_norm_backward(dy, x, h, weight, rstd, post=None, post_rstd=None, gate=None, alpha=1.0, dh=None):
    """Gradients by name, and by name the sums of magnitudes that their errors go by."""
    dy, x, h, weight = dy.double(), x.double(), h.double(), weight.double()
    one = torch.ones(1, 1, dtype=torch.float64)
    r2 = rstd.double()[:, None]
    r1 = one if post is None else post_rstd.double()[:, None]
    p = one if post is None else post.double()
    k = one if gate is None else gate.double().view(-1, x.shape[1])
    a, m, n = dy * weight, h * r2, x * r1
    g = r2 * (a - m * (a * m).mean(1, keepdim=True))
    sg = r2 * (a.abs() + m.abs() * (a * m).abs().mean(1, keepdim=True))
    if dh is not None:
        g, sg = g + dh.double(), sg + dh.double().abs()
    e, se = g * k, sg * k.abs()
    out = {"dresidual": alpha * g, "dweight": (dy * m).sum(0)}
    size = {"dresidual": abs(alpha) * sg, "dweight": (dy * m).abs().sum(0)}
    if post is None:
        out["dx"], size["dx"] = e, se
    else:
        ep, sp = e * p, se * p.abs()
        out["dx"] = r1 * (ep - n * (ep * n).mean(1, keepdim=True))
        size["dx"] = r1 * (sp + n.abs() * (sp * n.abs()).mean(1, keepdim=True))
        out["dpost_weight"], size["dpost_weight"] = (e * n).sum(0), (se * n.abs()).sum(0)
    if gate is not None:
        dg, sd = g * n * p, sg * (n * p).abs()
        out["dgate"], size["dgate"] = (dg, sd) if gate.dim() == 2 else (dg.sum(0), sd.sum(0))
    return out, size


def quantize_rows(x):
    """The integers and scales of x in 32 bits: single operations, so that each has one right result."""
    x = x.float()
    top = x.abs().amax(1)
    scale = (top / torch.full_like(top, 127.0)).clamp(min=2.0 ** -126)
    odd = ~torch.isfinite(top)
    scale[odd] = math.nan
    q = torch.round(x / scale[:, None])
    q[odd] = 0.0
    return q.to(torch.int8), scale


def int8_matmul(a, w, a_scales, w_scales, bias=None):
    """The sums as whole numbers, and d in 64 bits with the magnitudes that its error goes by."""
    sums = a.double() @ w.double().T   # whole numbers below 2^53
    d = sums * a_scales.double()[:, None] * w_scales.double()
    size = d.abs()
    if bias is not None:
        d, size = d + bias.double(), size + bias.double().abs()
    return sums, d, size


def adjust_logits(logits, tokens=None, lengths=None, prompts=None, repetition=None, frequency=None, presence=None,
                  bias_tokens=None, bias_values=None, allowed=None):
    """The adjusted logits in 64 bits and the magnitudes that their errors go by, token by token."""
    z = logits.double().clone()
    size = z.abs()
    rows, vocab = z.shape
    for r in range(rows):
        if tokens is not None:
            n = tokens.shape[1] if lengths is None else min(max(int(lengths[r]), 0), tokens.shape[1])
            p = 0 if prompts is None else int(prompts[r])
            count = {}
            for i in range(n):
                v = int(tokens[r, i])
                if 0 <= v < vocab:
                    count[v] = count.get(v, 0) + (1 if i >= p else 0)
            rep = 1.0 if repetition is None else float(repetition[r])
            for v, c in count.items():
                s = float(z[r, v])
                s = s / rep if s > 0 else s * rep
                mag = abs(s)
                if c > 0:
                    f = 0.0 if frequency is None else float(frequency[r]) * c
                    q = 0.0 if presence is None else float(presence[r])
                    s -= f + q
                    mag += abs(f) + abs(q)
                z[r, v], size[r, v] = s, mag
        if bias_tokens is not None:
            for v, b in zip(bias_tokens[r].tolist(), bias_values[r].tolist()):
                if 0 <= v < vocab:
                    z[r, v] += b
                    size[r, v] += abs(b)
        if allowed is not None:
            word = allowed[r].long() & 0xFFFFFFFF
            v = torch.arange(vocab)
            z[r, (word[v // 32] >> (v % 32)) & 1 == 0] = -math.inf
    return z, size
