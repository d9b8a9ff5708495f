"""The waits of the block norms' rings and of the 8-bit product, run out without faulting the GPU, by the debug build's
fault 3 as in test_lm_watchdog.py: the call ends, reports a timeout, and the next one has the bits of an untroubled handle.
"""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import gemm_ws
from tests.debug_helpers import debug_handle
from tests.test_lm_block import block_inputs, rows
from tests.test_lm_int8 import integers, scales
from tests.test_lm_watchdog import gives_up_and_recovers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = debug_handle(timeout_ms=200)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


@pytest.mark.parametrize("M,N,K", [(20, 600, 4096), (700, 3000, 640), (2000, 9000, 1500)])
def test_int8_product(g, M, N, K):
    """K cut between pairs, one tile a pair, and several."""
    gen = torch.Generator().manual_seed(M)
    a, w, sa, sw = integers(M, K, gen), integers(N, K, gen, (K + 15) // 16 * 16), scales(M, gen), scales(N, gen)
    d = torch.empty(M, N, device="cuda")
    gives_up_and_recovers(g, lambda: g.int8_matmul(a, w, sa, sw, d), (d,))


# more rows than the rings hold, so that the fault leaves some out
@pytest.mark.parametrize("T,H,dtype", [(1500, 8448, torch.bfloat16), (8000, 1024, torch.float32), (700, 8192, torch.float32)])
@pytest.mark.parametrize("post", [True, False])
def test_forward_ring(g, T, H, dtype, post):
    v, _ = block_inputs(T, H, dtype, "cols", post, 1)
    y, h = torch.empty_like(v["x"]), torch.empty_like(v["x"])
    gives_up_and_recovers(g, lambda: g.block_norm(v["x"], v["residual"], v["weight"], y, post_weight=v["post"],
                                                  gate=v["gate"], h=h), (y, h))


@pytest.mark.parametrize("T,H,dtype", [(6000, 1024, torch.float16), (1500, 8192, torch.bfloat16), (1500, 4096, torch.float32)])
@pytest.mark.parametrize("gate,post", [("cols", True), ("rows", True), ("none", False)])
def test_gradient_ring(g, T, H, dtype, gate, post):
    v, gen = block_inputs(T, H, dtype, gate, post, 2)
    dy, dh = rows(T, H, dtype, gen), rows(T, H, dtype, gen)
    y, h, dx, dres = (torch.empty_like(v["x"]) for _ in range(4))
    r1, r2 = torch.empty(T, device="cuda") if post else None, torch.empty(T, device="cuda")
    g.block_norm(v["x"], v["residual"], v["weight"], y, post_weight=v["post"], gate=v["gate"], h=h, post_rstd=r1, rstd=r2)
    dw = torch.empty_like(v["weight"])
    dp = torch.empty_like(dw) if post else None
    dg = torch.empty_like(v["gate"]) if gate != "none" else None
    gives_up_and_recovers(
        g, lambda: g.block_norm_backward(dy, v["x"], h, v["weight"], r2, dx, dres, post_weight=v["post"], post_rstd=r1,
                                         gate=v["gate"], dh=dh, dweight=dw, dpost_weight=dp, dgate=dg),
        [t for t in (dx, dres, dw, dp, dg) if t is not None])
