"""The norm's 8-bit output: the e4m3 rounding of y / scale, exactly, and with dropout before it."""
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


def quotients(x, rstd, w, scales):
    """(x * rstd * w) / scale in 32 bits, each operation rounded, as the operator is defined."""
    y = x * rstd[:, None] * w
    groups = scales.shape[1]
    size = x.shape[1] if groups == 1 else 128
    return y / scales.repeat_interleave(size, 1)[:, :x.shape[1]]


@pytest.mark.parametrize("T,H,groups", [(6000, 4096, 1), (6000, 4096, 32), (4001, 1000, 8), (1, 8192, 1)])
def test_values_are_the_roundings_of_the_quotients(g, T, H, groups):
    gen = torch.Generator("cuda").manual_seed(T + H)
    x = torch.randn(T, H, device="cuda", generator=gen)
    w = torch.randn(H, device="cuda", generator=gen)
    y = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    scales, rstd = torch.empty(T, groups, device="cuda"), torch.empty(T, device="cuda")
    g.add_rms_norm(x, w, y, rstd=rstd, scales=scales, eps=EPS)
    want = quotients(x, rstd, w, scales).to(torch.float8_e4m3fn)
    assert torch.equal(y.float(), want.float())


@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("scale", [7, 13, 14, 49])
def test_quotients_between_two_values_go_to_the_even_one(g, groups, scale):
    """Columns whose quotient is exactly half-way: 25 between 24 and 26, 29 between 28 and 30, 50 and 58.
    The rest of the row makes the mean square a power of 4, so that the norm scales by a power of 2."""
    H = 256
    row = [448 * scale, 25 * scale, 29 * scale, 50 * scale, 58 * scale, -25 * scale]
    row = row + [0] * (128 - len(row)) + row if groups == 2 else row
    total = sum(v * v for v in row)
    mean = 1
    while mean * H < total + 4 * H:
        mean *= 4
    left = mean * H - total
    while left > 0 and len(row) < H:
        v = min(int(left ** 0.5), 448 * scale)      # the largest square that is left
        while v * v > left:
            v -= 1
        row.append(v)
        left -= v * v
    assert left == 0 and len(row) <= H
    x = torch.zeros(1, H, device="cuda")
    x[0, :len(row)] = torch.tensor(row, dtype=torch.float32)
    y = torch.empty(1, H, dtype=torch.float8_e4m3fn, device="cuda")
    scales, rstd = torch.empty(1, groups, device="cuda"), torch.empty(1, device="cuda")
    w = torch.ones(H, device="cuda")
    g.add_rms_norm(x, w, y, rstd=rstd, scales=scales, eps=0.0)
    want = quotients(x, rstd, w, scales)
    assert torch.equal(y.float(), want.to(torch.float8_e4m3fn).float())
    if float(rstd) == mean ** -0.5:                 # the root is exact, as it need not be
        assert y[0, :6].float().tolist() == [448, 24, 28, 48, 56, -24]


@pytest.mark.parametrize("T,H", [(1, 8), (3, 200), (40, 1001), (9, 4096), (700, 2056), (1300, 1024), (2, 32768)])
@pytest.mark.parametrize("form", ["row", "group"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_with_dropout(g, T, H, form, dtype):
    gen = torch.Generator().manual_seed(T * 5 + H)
    x, res = rows(T, H, dtype, gen), rows(T, H, dtype, gen, scale=4.0)
    w = rows(1, H, dtype, gen)[0]
    words = rng_words(3, 2 ** 35)
    size = H if form == "row" else 128
    groups = -(-H // size)
    y = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    scales, h, rstd = torch.empty(T, groups, device="cuda"), torch.empty_like(x), torch.empty(T, device="cuda")
    g.add_rms_norm(x, w, y, residual=res, h=h, rstd=rstd, scales=scales, eps=EPS, p=0.3, rng=words)
    keep = torch.empty(T, H, device="cuda")       # the mask of a plain call on ones, which its own test checks
    g.dropout(torch.ones_like(keep), keep, 0.3, words)
    want_h, want_r, want = ref.add_rms_norm(x, res, w, EPS, keep.double())
    sizes = 2 * x.double().abs() + res.double().abs()
    tol = ref.UNIT[dtype] * want_h.abs() + 2.0 ** -22 * sizes + ref.TINY[dtype]
    assert torch.all((h.double() - want_h).abs() <= tol)
    assert torch.all((rstd.double() - want_r).abs() <= F32 * want_r)
    padded = torch.zeros(T, groups * size, dtype=torch.float64, device="cuda")
    padded[:, :H] = want
    top = (padded.view(T, groups, size).abs().amax(2) / ref.E4M3_MAX).clamp(min=2.0 ** -126)
    slack = F32 * 8   # the sum that is normalised may cancel
    assert torch.all((scales.double() - top).abs() <= slack * top)
    v = want / top.repeat_interleave(size, 1)[:, :H]
    off = (y.double() - v).abs()
    assert torch.all(off <= (ref.E4M3_UNIT + slack) * v.abs() + ref.E4M3_TINY + slack)
