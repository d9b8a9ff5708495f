"""The language-model operators' waits, tested without faulting the GPU.

The debug build's fault 3 leaves copies out, so that the waits for them can only run out. The call
must end on its own, report GEMM_WS_ERR_TIMEOUT through the status query, and leave the handle fit: the
next call returns the bits of a handle that never gave up.
"""
from __future__ import annotations

import time

import pytest
import torch

from async_pipelines_gb300 import gemm_ws
from tests.debug_helpers import configure, debug_handle
from tests.test_lm_norm import rng_words, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = debug_handle(timeout_ms=200)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


def gives_up_and_recovers(g, call, outs):
    """`call` normally, with the fault, and normally again."""
    call()
    assert g.query_status() == gemm_ws.OK
    want = [v.clone() for v in outs]
    configure(g, fault=3)
    start = time.perf_counter()
    call()
    status = g.query_status()
    took = time.perf_counter() - start
    configure(g, fault=0)
    assert status == gemm_ws.ERR_TIMEOUT, gemm_ws.status_string(status)
    assert took < 20.0
    assert g.query_status() == gemm_ws.OK          # reading cleared the word
    for v in outs:
        v.fill_(float("nan"))
    call()
    assert g.query_status() == gemm_ws.OK
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,V", [(5, 3000), (100, 70000), (300, 5000), (2000, 20000)])
@pytest.mark.parametrize("backward", [False, True])
def test_cross_entropy(g, T, V, backward):
    """In one launch, with single CTAs, rows as they lie or packed, and with CTA pairs."""
    H = 512
    gen = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    w = (torch.randn(V, H, device="cuda", generator=gen) / 20).bfloat16()
    t = torch.randint(V, (T,), device="cuda", generator=gen)
    loss, lse, mean = (torch.empty(n, device="cuda") for n in (T, T, 2))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    g.linear_cross_entropy(x, w, t, loss, lse, mean=mean)
    if backward:
        gives_up_and_recovers(g, lambda: g.linear_cross_entropy_backward(x, w, t, lse, mean[1:], dx, dw),
                              (dx, dw))
    else:
        gives_up_and_recovers(g, lambda: g.linear_cross_entropy(x, w, t, loss, lse, mean=mean),
                              (loss, lse, mean))


@pytest.mark.parametrize("T,H,dtype", [(6000, 1024, torch.bfloat16), (2000, 8192, torch.float16),
                                       (2000, 8192, torch.float32)])
@pytest.mark.parametrize("dropout", [False, True])
def test_norm_rings(g, T, H, dtype, dropout):
    """Teams of one warp and of many; forward only with dropout of 16-bit types, which takes a ring."""
    gen = torch.Generator().manual_seed(T)
    x, res, dy = (rows(T, H, dtype, gen) for _ in range(3))
    w = rows(1, H, dtype, gen)[0]
    kw = dict(p=0.25, rng=rng_words(5, 9)) if dropout else {}
    h, y, dx, dres = (torch.empty_like(x) for _ in range(4))
    dw, rstd = torch.empty_like(w), torch.empty(T, device="cuda")

    def forward():
        g.add_rms_norm(x, w, y, residual=res, h=h, rstd=rstd, **kw)

    forward()
    if dropout and dtype != torch.float32:
        gives_up_and_recovers(g, forward, (y, h, rstd))
    gives_up_and_recovers(
        g, lambda: g.add_rms_norm_backward(dy, h, w, rstd, dx, dw, dh=res, dresidual=dres, **kw),
        (dx, dres, dw))
