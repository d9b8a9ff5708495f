"""A ring of the block norms that gives up waits for the copies that are under way, and for no others.

By the debug build: each team gives up a row that has come, as if its wait had run out. All copies that it had called for are
there or about to be, so that the call ends at once; a copy that was never called for would be waited for for 100 ms.
"""
from __future__ import annotations

import time

import pytest
import torch

from async_pipelines_gb300 import gemm_ws
from tests.debug_helpers import configure, debug_handle
from tests.test_lm_block import block_inputs, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = debug_handle(timeout_ms=1000)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


def ends_at_once(g, call, outs):
    call()
    assert g.query_status() == gemm_ws.OK
    want = [v.clone() for v in outs]
    configure(g, fault=5)
    torch.cuda.synchronize()
    start = time.perf_counter()
    call()
    status = g.query_status()
    took = time.perf_counter() - start
    configure(g, fault=0)
    assert status == gemm_ws.ERR_TIMEOUT
    assert took < 0.09, f"{1e3 * took:.0f} ms"
    for v in outs:
        v.fill_(float("nan"))
    call()
    assert g.query_status() == gemm_ws.OK
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


# more rows for each team than its part of the ring holds
SHAPES = [(8000, 1024, torch.bfloat16), (1500, 8192, torch.bfloat16), (1500, 4096, torch.float32)]


@pytest.mark.parametrize("T,H,dtype", [(1500, 8448, torch.bfloat16), (8000, 1024, torch.float32), (1500, 8192, torch.float32)])
@pytest.mark.parametrize("post", [True, False])
def test_forward(g, T, H, dtype, post):
    v, _ = block_inputs(T, H, dtype, "cols", post, 1)
    y, h = torch.empty_like(v["x"]), torch.empty_like(v["x"])
    ends_at_once(g, lambda: g.block_norm(v["x"], v["residual"], v["weight"], y, post_weight=v["post"], gate=v["gate"], h=h),
                 (y, h))


@pytest.mark.parametrize("T,H,dtype", SHAPES)
@pytest.mark.parametrize("gate", ["none", "rows"])
@pytest.mark.parametrize("post", [True, False])
def test_gradient(g, T, H, dtype, gate, post):
    v, gen = block_inputs(T, H, dtype, gate, post, 2)
    dy, dh = rows(T, H, dtype, gen), rows(T, H, dtype, gen)
    y, h, dx, dres = (torch.empty_like(v["x"]) for _ in range(4))
    r1, r2 = torch.empty(T, device="cuda") if post else None, torch.empty(T, device="cuda")
    g.block_norm(v["x"], v["residual"], v["weight"], y, post_weight=v["post"], gate=v["gate"], h=h, post_rstd=r1, rstd=r2)
    dw = torch.empty_like(v["weight"])
    dg = torch.empty_like(v["x"]) if gate == "rows" else None
    ends_at_once(
        g, lambda: g.block_norm_backward(dy, v["x"], h, v["weight"], r2, dx, dres, post_weight=v["post"], post_rstd=r1,
                                         gate=v["gate"], dh=dh, dweight=dw, dgate=dg),
        [t for t in (dx, dres, dw, dg) if t is not None])
