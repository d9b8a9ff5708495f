"""How a token's share of the loss enters the cross entropy's gradients.

(softmax - [target]) * g / s is rounded to bf16 on its way into both products, s, the largest |g|, is not: what
all tokens of the largest gradient have in common is not off by a common share. Of a head that
knows nothing yet their targets' terms are p - 1 with p about 1 / V, which rounds to -1: off by p. Everything
else is rounded independently, up to 2^-8 a value, so that over N values it averages to 2^-8 / sqrt(3 N).
"""
from __future__ import annotations

import math

import pytest
import torch

from async_pipelines_gb300 import gemm_ws

pytestmark = pytest.mark.gpu

IGNORE = -100


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


def untrained(T, H, V, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + T)
    w = (0.3 * torch.randn(V, H, device="cuda", generator=gen) / math.sqrt(H)).bfloat16()
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    return x, w, torch.randint(V, (T,), device="cuda", generator=gen)


def in_64_bits(x, w, t, grad):
    p = torch.softmax(x.double() @ w.double().T, 1)
    p[torch.arange(len(t), device="cuda"), t] -= 1.0
    p *= grad.double()[:, None]
    return p @ w.double(), p.T @ x.double()


def common(got, want):
    """The share by which `got` as a whole is larger than `want`, itself rounded as an output is: a row of
    dweight that one token names is -g times x, whose few significands are all rounded the same way."""
    want = want.to(got.dtype).double()
    return float((got.double() * want).sum() / (want * want).sum()) - 1.0


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def gradients(g, x, w, t, grad):
    loss, lse, mean = (torch.empty(n, device="cuda") for n in (len(t), len(t), 2))
    g.linear_cross_entropy(x, w, t, loss, lse, mean=mean, ignore_index=IGNORE)
    dx, dw = torch.full_like(x, 3.0), torch.full_like(w, 3.0)
    g.linear_cross_entropy_backward(x, w, t, lse, mean[1:] if grad is None else grad, dx=dx, dweight=dw,
                                    ignore_index=IGNORE)
    return dx, dw


# 1 / T rounded to bf16 is off by 3.4e-3 to 3.9e-3 of it, one way or the other
@pytest.mark.parametrize("T", [255, 253, 510, 491, 480])
@pytest.mark.parametrize("each", [False, True])
def test_the_mean_of_any_number_of_tokens(g, T, each):
    H, V = 64, 20000
    x, w, t = untrained(T, H, V)
    grad = torch.full((T,), 1.0 / T, device="cuda")
    dx, dw = gradients(g, x, w, t, grad if each else None)
    want = in_64_bits(x, w, t, grad)
    bound = 4.0 / V + 4 * 2.0 ** -8 / math.sqrt(3 * T * H)      # p is e^(0.3 z) / V; four deviations
    for got, exact in zip((dx, dw), want):
        assert abs(common(got, exact)) < bound
        # an output's own rounding: 2^-8 at most, 2^-8 / sqrt(3) of the smallest significands on average
        assert off(got, exact) < 2.0 ** -8 / math.sqrt(3) + bound


def test_one_gradient_for_all_and_the_same_for_each(g):
    x, w, t = untrained(700, 264, 5001)
    one = gradients(g, x, w, t, torch.full((1,), 0.0137, device="cuda"))
    each = gradients(g, x, w, t, torch.full((700,), 0.0137, device="cuda"))
    for a, b in zip(one, each):
        assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [1.0, 1e-30, 1e30])
def test_classes_of_weights(g, scale):
    """Tokens of weight 1, 0.3, -0.7 and 1e-4, some of weight 0. The smaller weights' share of the largest is
    rounded, by up to 2^-8 of it."""
    T, H, V = 900, 128, 20000
    x, w, t = untrained(T, H, V, 5)
    weights = torch.tensor([1.0, 0.3, -0.7, 1e-4, 0.0], device="cuda")
    which = torch.arange(T, device="cuda") % 5
    grad = weights[which] * scale
    dx, dw = gradients(g, x, w, t, grad)
    want = in_64_bits(x, w, t, grad)
    for k in range(4):
        mine = which == k
        bound = (0.0 if k == 0 else 2.0 ** -8) + 4.0 / V + 4 * 2.0 ** -8 / math.sqrt(3 * int(mine.sum()) * H)
        assert abs(common(dx[mine], want[0][mine])) < bound
        assert off(dx[mine], want[0][mine]) < 2.0 ** -8 / math.sqrt(3) + bound
    assert not dx[which == 4].any()
    assert off(dw, want[1]) < 2.0 ** -8 / math.sqrt(3) + 2.0 ** -8


@pytest.mark.parametrize("T", [40, 600])
@pytest.mark.parametrize("each", [False, True])
def test_rows_without_a_gradient_may_hold_anything(g, T, each):
    """Targets outside the vocabulary, and tokens of gradient 0: no part in dweight, dx 0."""
    x, w, t = untrained(T, 72, 900, 9)
    without = torch.arange(T, device="cuda") % 7 == 3
    t = torch.where(without, 900 + 5, t)
    grad = torch.full((T,), 0.25, device="cuda")
    clean = gradients(g, x, w, t, grad if each else grad[:1].clone())
    dirty = x.clone()
    dirty[without] = float("nan")
    got = gradients(g, dirty, w, t, grad if each else grad[:1].clone())
    for a, b in zip(got, clean):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    assert not got[0][without].any()
    if each:
        t2 = torch.where(without, 1, t)
        got = gradients(g, dirty, w, t2, torch.where(without, 0.0, grad))
        for a, b in zip(got, clean):
            assert torch.equal(a, b)
    nothing = gradients(g, dirty, w, t, torch.zeros(T if each else 1, device="cuda"))
    assert not nothing[0].any() and not nothing[1].any()
