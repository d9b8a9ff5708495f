"""Rows off 16-byte boundaries: what they may cost against aligned ones."""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import gemm_ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


def time_of(call, n=10):
    best = float("inf")
    call()
    for _ in range(5):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        for _ in range(n):
            call()
        end.record()
        torch.cuda.synchronize()
        best = min(best, start.elapsed_time(end) / n)
    return best


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_forward_of_odd_rows_keeps_two_of_them_on_an_sm(g, dtype):
    """8192 x 8191 against 8192 x 8192: about twice the time, three and a half times with one row an SM."""
    took = []
    for cols in (8191, 8192):
        x, res, h, y = (torch.zeros(8192, cols, dtype=dtype, device="cuda") for _ in range(4))
        w, rstd = torch.ones(cols, dtype=dtype, device="cuda"), torch.empty(8192, device="cuda")
        took.append(time_of(lambda: g.add_rms_norm(x, w, y, residual=res, h=h, rstd=rstd)))
    assert took[0] < 2.8 * took[1]
