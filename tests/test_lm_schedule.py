"""CPU checks of the language-model operators' boundary and of the cross entropy's schedule.

The debug build lists the units that the product kernel's clusters walk, by the kernel's own
functions: every tile of every job (and every cut of its K) once, the cuts a partition of K, and
the clusters' loads even.
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest

from async_pipelines_gb300 import build, gemm_ws, lm_ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dbg():
    build.ensure_built()
    return gemm_ws.load_debug_library()


def test_every_declared_operator_is_exported_and_bound(dbg):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gemm_ws_lm.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(gemm_ws_\w+)\s*\(", text))
    assert names == set(lm_ops.EXPORTS)
    for lib in (gemm_ws.load_library(), dbg):
        for name in names:
            assert hasattr(lib, name)


def units(dbg, cg, clusters, bn, count, jobs):
    flat = (ctypes.c_int * (4 * len(jobs)))(*[v for j in jobs for v in j])
    n = ctypes.c_int64()
    args = (cg, clusters, bn, count, flat, len(jobs))
    assert dbg.gemm_ws_debug_ce_units(*args, None, 0, ctypes.byref(n)) == gemm_ws.OK
    rows = np.zeros((n.value, 8), dtype=np.int32)
    assert dbg.gemm_ws_debug_ce_units(*args, rows.ctypes.data, n.value, ctypes.byref(n)) == gemm_ws.OK
    return rows


def check_cover(rows, cg, bn, count, jobs):
    for j, (m, n, k, cuts) in enumerate(jobs):
        m, k = (count if v < 0 else v for v in (m, k))
        mine = rows[rows[:, 2] == j]
        tiles = {(a, b) for a in range(0, m, 128 * cg) for b in range(0, n, bn)}
        seen = [tuple(r) for r in mine[:, 3:6]]
        assert len(seen) == len(set(seen)) == len(tiles) * cuts
        assert {s[:2] for s in seen} == tiles
        stages = -(-k // (64 * cg))
        edges = [c * stages // cuts for c in range(cuts + 1)]
        for _, _, cut, s0, s1 in mine[:, 3:8]:
            assert (s0, s1) == (edges[cut], edges[cut + 1])


@pytest.mark.parametrize("cg,clusters,bn", [(1, 152, 256), (1, 152, 96), (2, 76, 256), (2, 74, 256), (1, 7, 64)])
@pytest.mark.parametrize("count", [0, 1, 127, 300, 4500])
def test_logits_cover(dbg, cg, clusters, bn, count):
    for n, k in ((1, 8), (1000, 256), (50001, 3000)):
        jobs = [(-1, n, k, 1)]
        check_cover(units(dbg, cg, clusters, bn, count, jobs), cg, bn, count, jobs)


@pytest.mark.parametrize("cg,clusters", [(1, 152), (2, 76), (2, 74), (1, 5)])
@pytest.mark.parametrize("count", [0, 1, 64, 129, 1000, 4096])
@pytest.mark.parametrize("piece,hidden,cuts", [(256, 64, 1), (25001, 3000, 1), (32768, 4096, 1),
                                               (8192, 2048, 4), (131072, 256, 16)])
def test_gradients_cover(dbg, cg, clusters, count, piece, hidden, cuts):
    jobs = [(-1, hidden, piece, cuts), (piece, hidden, -1, 1)]
    check_cover(units(dbg, cg, clusters, 256, count, jobs), cg, 256, count, jobs)


@pytest.mark.parametrize("count,piece,hidden", [(4096, 32768, 4096), (4500, 25088, 3000), (2048, 32768, 2048)])
def test_gradients_are_balanced(dbg, count, piece, hidden):
    """dx's long units leave the clusters uneven; dweight's short ones fill the gaps, up to one
    short unit and what is left of a long one over whole short ones."""
    rows = units(dbg, 2, 76, 256, count, [(-1, hidden, piece, 1), (piece, hidden, -1, 1)])
    load = np.zeros(76)
    np.add.at(load, rows[:, 0], rows[:, 7] - rows[:, 6])
    short = -(-count // 128)
    long_over_short = -(-piece // 128) % short
    assert load.max() - load.min() <= short + long_over_short
