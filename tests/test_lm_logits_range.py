"""Adjusted logits that pass the range of a 16-bit output, and the two ways in which a history is counted.

Values past the range are chosen at least 1 % from the border to an infinity, so each has one right result.
"""
from __future__ import annotations

import math

import pytest
import torch

from async_pipelines_gb300 import gemm_ws
from tests import lm_block_reference as ref

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    handle.close()


def past_the_range(dtype):
    """Logits, and what penalties and biases make of them: an infinity of each sign or a value just inside, by every operation."""
    top = torch.finfo(dtype).max
    rows, vocab = 3, 48
    z = torch.zeros(rows, vocab)
    z[:, 0:4] = 0.9 * top                # divided, multiplied, biased up and down
    z[:, 4:8] = -0.9 * top
    z[:, 8], z[:, 9] = top, -top         # as they are
    z[:, 10], z[:, 11] = math.inf, -math.inf
    z[:, 12:14] = 1.0
    tokens = torch.tensor([[0, 4, 8, 9, 12, 20]]).repeat(rows, 1)
    bias_tokens = torch.tensor([[1, 2, 5, 6, 13, 14, 15, 16]]).repeat(rows, 1)
    up = torch.tensor([0.5, -0.5, -0.5, 0.5, 3.0, -3.0, 0.95, -0.95]) * top
    return {"logits": z.to(dtype), "tokens": tokens, "repetition": torch.tensor([0.5, 2.0, 1.0]),
            "frequency": torch.tensor([0.25, -0.25, 0.0]) * top, "presence": torch.tensor([0.25, -3.0, 0.0]) * top,
            "bias_tokens": bias_tokens, "bias_values": up.repeat(rows, 1)}


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("place", [False, True])
def test_outputs_past_the_range(g, dtype, place):
    v = past_the_range(dtype)
    if dtype is torch.bfloat16:   # its range is that of the 32 bits that all is computed in: no step may pass it and come back
        v["frequency"][1] = v["presence"][1] = 0.0
        v["bias_values"] = v["bias_values"].clamp(-0.99 * torch.finfo(dtype).max, 0.99 * torch.finfo(dtype).max)
    want, size = ref.adjust_logits(**v)
    top = torch.finfo(dtype).max
    assert not bool(((want.abs() > 1.0001 * top) & (want.abs() < 1.01 * top)).any())
    assert int((want > 1.01 * top).sum()) >= 3 and int((want < -1.01 * top).sum()) >= 3
    dev = {k: t.cuda() for k, t in v.items()}
    logits = dev.pop("logits")
    out = logits if place else torch.empty_like(logits)
    g.adjust_logits(logits, out, **dev)
    got = out.cpu().double()
    right = want.clone()
    right[want > 1.01 * top], right[want < -1.01 * top] = math.inf, -math.inf
    assert torch.equal(got.isinf(), right.isinf()) and torch.equal(got[right.isinf()], right[right.isinf()])
    fine = ~right.isinf()
    # operations in 32 bits, 2^-24 each of the magnitudes, and the output's own rounding
    tol = torch.finfo(dtype).eps / 2 * right[fine].abs() + 2.0 ** -21 * size[fine].clamp(max=4.0 * top)
    assert bool(((got - right)[fine].abs() <= tol).all())


@gpu
@pytest.mark.parametrize("rows,vocab", [(2, 6000), (40, 8192), (40, 8193), (700, 30001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_hash_table_and_counts_by_place_are_the_same(g, rows, vocab, dtype):
    """Up to 4096 tokens of a history are counted in a hash table, more of them at their places in a slice of the vocabulary: one
    more token that counts for nothing changes the way, and no bit."""
    gen = torch.Generator("cuda").manual_seed(vocab)
    z = (3.0 * torch.randn(rows, vocab, device="cuda", generator=gen)).to(dtype)
    tokens = torch.randint(0, vocab, (rows, 4096), device="cuda", generator=gen)
    tokens[:, ::3] = torch.randint(0, 50, (rows, 1366), device="cuda", generator=gen)
    more = torch.cat([tokens, torch.full((rows, 1), -1, device="cuda")], 1)
    f = 0.25 + torch.rand(rows, device="cuda", generator=gen)
    b = torch.randint(0, vocab, (rows, 1024), device="cuda", generator=gen)
    value = torch.randn(rows, 1024, device="cuda", generator=gen)
    prompts = torch.full((rows,), 1000, dtype=torch.int32, device="cuda")
    kw = dict(prompt_lengths=prompts, repetition=f, frequency=f, presence=f, bias_tokens=b, bias_values=value)
    first, second = torch.empty_like(z), torch.empty_like(z)
    g.adjust_logits(z, first, tokens=tokens, **kw)
    g.adjust_logits(z, second, tokens=more, **kw)
    assert torch.equal(first, second) and not torch.equal(first, z)
