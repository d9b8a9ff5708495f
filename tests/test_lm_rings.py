"""The norm's kernels that bring rows through shared memory: teams of one warp, calls in place.

Tolerances as in tests/test_lm_norm.py: an output's one rounding, and F32 of the terms' magnitudes.
"""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import gemm_ws
from tests import lm_reference as ref
from tests.test_lm_norm import EPS, F32, rng_words, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


def near(got, want, dtype, size, slack=F32):
    tol = ref.UNIT[dtype] * want.abs() + slack * size + ref.TINY[dtype]
    assert torch.all((got.double() - want).abs() <= tol)


def mask(g, T, H, p, words):
    """The mask of a plain call on ones, which its own test checks."""
    keep = torch.empty(T, H, device="cuda")
    g.dropout(torch.ones_like(keep), keep, p, words)
    return keep.double()


@pytest.mark.parametrize("T,H,dtype", [(19457, 1024, torch.bfloat16), (20001, 256, torch.float16),
                                       (16000, 512, torch.float32), (17000, 8, torch.bfloat16)])
@pytest.mark.parametrize("dropout", [False, True])
def test_gradients_of_one_warp_teams(g, T, H, dtype, dropout):
    """A stage is filled again as soon as one lane says so: the others have read it by then."""
    gen = torch.Generator().manual_seed(T)
    dy, h, dh = (rows(T, H, dtype, gen, 0, 0, s) for s in (1.0, 2.0, 0.5))
    w = rows(1, H, dtype, gen)[0]
    rstd = (0.1 + torch.rand(T, generator=gen)).cuda()
    p, words = (0.25, rng_words(7, 11)) if dropout else (0.0, None)
    runs = []
    for _ in range(4):
        dx, dres, dw = torch.full_like(dy, 9.0), torch.full_like(dy, 9.0), torch.full_like(w, 9.0)
        g.add_rms_norm_backward(dy, h, w, rstd, dx, dw, dh=dh, dresidual=dres, p=p, rng=words)
        runs.append((dx, dres, dw))
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)
    dx, dres, dw = runs[0]
    want = ref.add_rms_norm_backward(dy, h, w, rstd, dh)
    near(dres, want[1], dtype, want[3])
    near(dw, want[2], dtype, want[4])
    near(dx, ref.apply_keep(want[1], mask(g, T, H, p, words)) if dropout else want[1], dtype, want[3] * 2)


@pytest.mark.parametrize("T,H,dtype", [(5000, 264, torch.bfloat16), (900, 8192, torch.bfloat16),
                                       (1300, 2048, torch.float16), (700, 8192, torch.float32)])
@pytest.mark.parametrize("dropout", [False, True])
def test_in_place(g, T, H, dtype, dropout):
    """Outputs over the inputs that they may replace: the same bits, forward and backward."""
    gen = torch.Generator().manual_seed(T + H)
    x, res, dy, dh = (rows(T, H, dtype, gen, 8, 0, s) for s in (1.0, 3.0, 1.0, 0.5))
    w = rows(1, H, dtype, gen)[0]
    kw = dict(p=0.25, rng=rng_words(5, 9)) if dropout else {}
    h, y, dx, dres = (torch.empty(T, H, dtype=dtype, device="cuda") for _ in range(4))
    dw, rstd = torch.empty_like(w), torch.empty(T, device="cuda")
    g.add_rms_norm(x, w, y, residual=res, h=h, rstd=rstd, eps=EPS, **kw)
    g.add_rms_norm_backward(dy, h, w, rstd, dx, dw, dh=dh, dresidual=dres, **kw)

    def copy_of(m):
        out = rows(T, H, dtype, gen, 8)
        out.copy_(m)
        return out

    for y_over_x in (True, False):
        a, b = copy_of(x), copy_of(res)
        if y_over_x:
            g.add_rms_norm(a, w, a, residual=b, h=b, eps=EPS, **kw)
            assert torch.equal(a, y) and torch.equal(b, h)
        else:
            c = torch.empty_like(y)
            g.add_rms_norm(a, w, c, residual=b, h=a, eps=EPS, **kw)
            assert torch.equal(a, h) and torch.equal(c, y) and torch.equal(b, res)
    for dx_over_dy in (True, False):
        a, b, dw2 = copy_of(dy), copy_of(dh), torch.empty_like(dw)
        over, other = (a, b) if dx_over_dy else (b, a)
        g.add_rms_norm_backward(a, h, w, rstd, over, dw2, dh=b, dresidual=other, **kw)
        assert torch.equal(over, dx) and torch.equal(other, dres) and torch.equal(dw2, dw)
