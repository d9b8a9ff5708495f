"""The language-model operators at the limits of their sizes.

On the CPU the debug build runs the kernels' own index arithmetic, for extents close to 2^31, against
Python's integers. On the GPU the largest extents that are accepted run with what lies around their
outputs watched.
"""
from __future__ import annotations

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
