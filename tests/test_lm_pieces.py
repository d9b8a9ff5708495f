"""The cross entropy's gradients over several pieces of the vocabulary.

A piece of G takes at most 256 MB, so these sizes take two to four of them: dx is added to by the
later ones, dweight's rows and the targets lie in each, the last is shorter and odd. Tolerances as
in tests/test_lm_loss.py; the reference is computed on the GPU in 64 bits.
"""
from __future__ import annotations

import math

import pytest
import torch

from async_pipelines_gb300 import gemm_ws

pytestmark = pytest.mark.gpu

IGNORE = -100
PIECE_BYTES = 256 << 20


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


def g_rows(T):
    """G's rows: whole tiles."""
    return 128 if T <= 128 else -(-T // 256) * 256


def make(T, H, V, ignored):
    gen = torch.Generator("cuda").manual_seed(T + H + V)
    w = (torch.randn(V, H, device="cuda", generator=gen) * 1.5 / math.sqrt(H)).bfloat16()
    t = torch.randint(V, (T,), device="cuda", generator=gen)
    edges = [V - 1, 0, V // 2, V // 3, 2 * V // 3, V // 4, 3 * V // 4, V - 300]
    n = min(T, len(edges))
    t[:n] = torch.tensor(edges[:n], device="cuda")
    up = torch.rand(T, 1, device="cuda", generator=gen) * 5.0
    x = (torch.randn(T, H, device="cuda", generator=gen) + up * w[t].float()).bfloat16()
    skip = torch.rand(T, device="cuda", generator=gen) < ignored
    skip[:n] = False
    return x, w, torch.where(skip, IGNORE, t)


def check(name, got, want, size):
    u = 2.0 ** -8
    got = got.double()
    bad = ~((got - want).abs() <= u * want.abs() + (u + 2.0 ** -14) * size + 2.0 ** -120)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off"
    assert float((got - want).norm()) <= 4e-3 * float(want.norm()), name


@pytest.mark.parametrize("T,H,V,ignored", [
    (4100, 64, 70001, 0.3),        # three pieces, CTA pairs
    (1030, 256, 140001, 0.0),      # two, with dx's sums cut along the vocabulary
    (40000, 64, 9001, 0.2),        # the least piece, 4096 words
    (300, 72, 600001, 0.4),
    (100, 128, 2200001, 0.3),      # up to 128 tokens: single CTAs
    (1, 64, 3200001, 0.0),
])
def test_gradients(g, T, H, V, ignored):
    x, w, t = make(T, H, V, ignored)
    need = g.linear_cross_entropy_workspace(T, H, V, True)
    assert need < 2 * g_rows(T) * V          # G of all of the vocabulary would not fit it
    loss, lse, mean = (torch.empty(n, device="cuda") for n in (T, T, 2))
    g.linear_cross_entropy(x, w, t, loss, lse, mean=mean, ignore_index=IGNORE)
    counted = t != IGNORE
    xd, wd = torch.where(counted[:, None], x.double(), 0.0), w.double()
    p = xd @ wd.T
    want_lse = torch.logsumexp(p, 1)
    tol = math.sqrt(H) * 2.0 ** -23 * float(xd.abs().sum(1).max() * wd.abs().max()) + 2.0 ** -20 * 20
    assert torch.all((lse - torch.where(counted, want_lse, 0.0)).abs() <= tol)
    at = torch.where(counted, t, 0)
    p = torch.exp(p - want_lse[:, None])
    p[torch.arange(T, device="cuda"), at] -= 1.0
    grad = torch.rand(T, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) + 0.5
    p *= torch.where(counted, grad.double(), 0.0)[:, None]
    want_dx, want_dw = p @ wd, p.T @ xd
    p.abs_()
    size_dx, size_dw = p @ wd.abs(), p.T @ xd.abs()
    del p
    dx, dw = torch.full_like(x, 3.0), torch.full_like(w, 3.0)
    g.linear_cross_entropy_backward(x, w, t, lse, grad, dx=dx, dweight=dw, ignore_index=IGNORE)
    check("dx", dx, want_dx, size_dx)
    check("dweight", dw, want_dw, size_dw)
    dx, dw = torch.full_like(x, 3.0), torch.full_like(w, 3.0)
    g.linear_cross_entropy_backward(x, w, t, lse, grad, dx=dx, ignore_index=IGNORE)
    g.linear_cross_entropy_backward(x, w, t, lse, grad, dweight=dw, ignore_index=IGNORE)
    check("dx alone", dx, want_dx, size_dx)
    check("dweight alone", dw, want_dw, size_dw)


@pytest.mark.parametrize("T", [1, 60, 128, 129, 300, 1030, 5000])
def test_a_piece_keeps_to_its_bytes(g, T):
    """G's rows are rounded up to whole tiles, which counts where there are few tokens."""
    H, V = 64, 1 << 24
    need = g.linear_cross_entropy_workspace(T, H, V, True)
    beside = 2 * g_rows(T) * H + 16 * T + 16 * T * H * 4 + (1 << 16)     # x packed, a row's numbers, dx's sums
    assert need <= PIECE_BYTES + beside
