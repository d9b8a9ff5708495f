"""The language-model operators at the limits of their sizes.

On the CPU the debug build runs the kernels' own index arithmetic, for extents close to 2^31, against
Python's integers. On the GPU the largest extents that are accepted run with what lies around their
outputs watched.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from async_pipelines_gb300 import build, gemm_ws
from tests import lm_reference as ref


@pytest.fixture(scope="module")
def dbg():
    build.ensure_built()
    return gemm_ws.load_debug_library()


# ------------------------------------------------------------------ on the CPU

@pytest.mark.parametrize("cols", [1, 7, 8, 9, 2047, 2048, 2049, 2 ** 31 - 2049, 2 ** 31 - 2048, 2 ** 31 - 2047,
                                  2147483548, 2 ** 31 - 17, 2 ** 31 - 9, 2 ** 31 - 8, 2 ** 31 - 7, 2 ** 31 - 1])
def test_columns_of_a_row(dbg, cols):
    """The last steps of a row's threads, those that have no group among them: columns in the row or at
    its end, and no group that is said to be whole without being so."""
    groups = -(-cols // 8)
    first = max(0, groups - 300)
    count = groups - first + 256
    rows = np.zeros((count, 3), dtype=np.int32)
    assert dbg.gemm_ws_debug_row_columns(cols, first, count, rows.ctypes.data) == gemm_ws.OK
    for i, (c, whole, next_whole) in enumerate(rows.tolist()):
        g = first + i
        assert c == 8 * g if g < groups else c >= cols
        assert whole == (c + 8 <= cols)
        assert next_whole == (c + 16 <= cols)


LARGEST = 2 ** 31 - 4096      # of an extent of the cross entropy


@pytest.mark.parametrize("cg,bn", [(1, 256), (1, 96), (2, 256)])
@pytest.mark.parametrize("extent", [LARGEST - 1, LARGEST, 2 ** 31 - 256, 2 ** 31 - 255, 2 ** 31 - 1])
def test_units_of_the_largest_extents(dbg, cg, bn, extent):
    """A vocabulary, a hidden size or a count of tokens of almost 2^31: all of its tiles are walked."""
    for count, n, k, tiles in ((1, extent, 8, -(-extent // bn)), (1, 8, extent, 1),
                               (extent, 8, 8, -(-extent // (128 * cg)))):
        jobs = (ctypes.c_int * 4)(-1, n, k, 1)
        rows, total = np.zeros((1, 8), dtype=np.int32), ctypes.c_int64()
        assert dbg.gemm_ws_debug_ce_units(cg, 7, bn, count, jobs, 1, rows.ctypes.data, 1,
                                          ctypes.byref(total)) == gemm_ws.OK
        assert total.value == tiles
        assert tuple(rows[0, 6:]) == (0, -(-k // (64 * cg)))


# ------------------------------------------------------------------ on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


@gpu
@pytest.mark.parametrize("cols", [2147483548, 2 ** 31 - 1])
def test_dropout_of_the_longest_rows(g, cols):
    """One row off any boundary, of almost 2^31 columns: nothing below or behind it is written."""
    before, behind = 2 ** 31 + 1, 4096
    buf = torch.full((before + cols + behind,), 5.0, dtype=torch.bfloat16, device="cuda")
    row = buf[before:before + cols].view(1, cols)
    row.fill_(1.0)
    seed, first = 41, 2 ** 40
    g.dropout(row, row, 0.5, torch.tensor([seed, first], device="cuda"))
    assert torch.all(buf[:before] == 5.0) and torch.all(buf[before + cols:] == 5.0)
    last = cols // 8 - 500
    for group, n in ((0, 4096), (last, cols - 8 * last)):
        keep = ref.keep_factor(1, n, 0.5, (seed, first + group))
        assert torch.equal(row[:, 8 * group:8 * group + n].cpu().double(), keep)
    share = float((row[0, ::1024] == 0).float().mean())
    assert abs(share - 0.5) < 2e-3      # two million samples: a deviation of 3.5e-4
    del buf, row
    torch.cuda.empty_cache()


@gpu
def test_extents_past_the_largest_are_refused(g):
    for sizes in ((LARGEST + 1, 8, 8), (1, LARGEST + 8, 8), (1, 8, LARGEST + 1), (2 ** 31 - 1, 8, 1),
                  (1, 8, 2 ** 31 - 255), (2 ** 31, 8, 1)):
        for backward in (False, True):
            with pytest.raises(gemm_ws.GemmWSError) as e:
                g.linear_cross_entropy_workspace(*sizes, backward)
            assert e.value.status == gemm_ws.ERR_INVALID_ARG
    assert g.linear_cross_entropy_workspace(1, 8, LARGEST) > 0
    assert g.linear_cross_entropy_workspace(1, LARGEST, 8) > 0


@gpu
def test_the_largest_vocabulary(g):
    """2^31 - 4096 words. A part of a row's sum is added to 2e5 times, each time off by up to 2^-24 of
    it: by about sqrt(2e5) of that, 3e-5, at the most."""
    T, H, V, step = 3, 8, LARGEST, 2 ** 24
    gen = torch.Generator("cuda").manual_seed(5)
    w = torch.empty(V, H, device="cuda", dtype=torch.bfloat16)
    for a in range(0, V, step):
        w[a:a + step] = torch.randn(min(step, V - a), H, device="cuda", generator=gen) / 2
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    t = torch.tensor([V - 1, 0, V // 2], device="cuda")
    loss, lse, mean = (torch.empty(n, device="cuda") for n in (T, T, 2))
    g.linear_cross_entropy(x, w, t, loss, lse, mean=mean)
    parts = [torch.logsumexp(x.double() @ w[a:a + step].double().T, 1) for a in range(0, V, step)]
    want = torch.logsumexp(torch.stack(parts), 0)
    assert torch.all((lse - want).abs() <= 1e-4)
    at = (x.double() * w[t].double()).sum(1)
    assert torch.all((loss - (want - at)).abs() <= 1e-4)
    assert abs(float(mean[0]) - float((want - at).mean())) <= 1e-4
    # the gradients, in 2048 pieces; the last rows of dweight
    dx, dw = torch.full_like(x, 3.0), torch.full_like(w, 3.0)
    g.linear_cross_entropy_backward(x, w, t, lse, mean[1:], dx=dx, dweight=dw)
    want_dx = -w[t].double()
    for a in range(0, V, step):
        part = w[a:a + step].double()
        want_dx += torch.exp(x.double() @ part.T - want[:, None]) @ part
    want_dx /= T
    assert float((dx.double() - want_dx).norm()) <= 4e-3 * float(want_dx.norm())
    for a in (0, V // 2 - 500, V - 1000):
        rows = torch.arange(a, a + 1000, device="cuda")
        p = torch.exp(x.double() @ w[a:a + 1000].double().T - want[:, None])
        p -= (t[:, None] == rows).double()
        tail = p.T @ x.double() / T
        assert float((dw[a:a + 1000].double() - tail).norm()) <= 4e-3 * float(tail.norm())
        rest = ~torch.isin(rows, t)
        assert float((dw[a:a + 1000][rest].double() - tail[rest]).norm()) <= 4e-3 * float(tail[rest].norm())
    del w, dw
    torch.cuda.empty_cache()
