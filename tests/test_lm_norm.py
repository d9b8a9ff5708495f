"""Dropout, add + RMS norm and its gradients, against plain implementations in 64 bits.

Tolerances, fixed before the first run: an output is rounded once to its type (UNIT of its
value, or TINY), and the 32-bit arithmetic before that is a sum of at most a few hundred terms a
thread and tree, each operation off by 2^-24: within F32 = 2^-16 of the terms' magnitudes.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

from async_pipelines_gb300 import build, gemm_ws
from tests import lm_reference as ref

F32 = 2.0 ** -16
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6


# ------------------------------------------------------------------ on the CPU

def test_reference_generator_known_answers():
    """Known answers published with the generator (Random123's kat_vectors, philox4x32 10)."""
    assert ref.philox(0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox(2 ** 128 - 1, 2 ** 64 - 1) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_reference_gradient_against_differences():
    g = torch.Generator().manual_seed(3)
    x, res, dy, dh, v = (torch.randn(4, 10, generator=g, dtype=torch.float64) for _ in range(5))
    w = torch.randn(10, generator=g, dtype=torch.float64)
    keep = ref.keep_factor(4, 10, 0.3, (5, 9))

    def value(x_, w_):
        h, _, y = ref.add_rms_norm(x_, res, w_, EPS, keep)
        return float((y * dy).sum() + (h * dh).sum())

    h, rstd, _ = ref.add_rms_norm(x, res, w, EPS, keep)
    dx, _, dw, _, _ = ref.add_rms_norm_backward(dy, h, w, rstd, dh, keep)
    e = 1e-5
    assert abs((value(x + e * v, w) - value(x - e * v, w)) / (2 * e) - float((dx * v).sum())) < 1e-7
    u = torch.randn(10, generator=g, dtype=torch.float64)
    assert abs((value(x, w + e * u) - value(x, w - e * u)) / (2 * e) - float((dw * u).sum())) < 1e-7


def test_null_handle_is_refused_without_a_gpu():
    build.ensure_built()
    lib = gemm_ws.load_library()
    bad = gemm_ws.ERR_INVALID_ARG
    assert lib.gemm_ws_dropout(None, 0, None, 8, None, 8, 1, 8, 0.1, None, None) == bad
    assert lib.gemm_ws_add_rms_norm(None, 0, None, 8, None, 8, None, None, 8, None, 8, 0, None, None,
                                    1, 8, EPS, 0.0, None, None) == bad
    assert lib.gemm_ws_add_rms_norm_backward(None, 0, None, 8, None, 8, None, 8, None, None, None, 8,
                                             None, 8, None, 1, 8, 0.0, None, None) == bad


# ------------------------------------------------------------------ on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    handle.close()


def rows(T, H, dtype, gen, pad=0, shift=0, scale=1.0):
    """T x H on the GPU, `pad` elements between rows, `shift` elements past an aligned address."""
    buf = (scale * torch.randn(T * (H + pad) + shift, generator=gen)).to(dtype).cuda()
    return buf[shift:].view(T, H + pad)[:, :H]


def rng_words(seed, first):
    return torch.tensor([seed, first], dtype=torch.int64, device="cuda")


def close(got, want, dtype, size=None, slack=F32, what=""):
    got = got.detach().cpu().double()
    size = want.abs() if size is None else size
    tol = ref.UNIT[dtype] * want.abs() + slack * size + ref.TINY[dtype]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / tol).max()):.3g} of the tolerance")


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 1000), (7, 1024), (3, 1032), (2, 4096), (1, 8192),
          (2, 8191), (1, 32768), (1300, 40), (700, 2048), (331, 1001)]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 8), (3, 13), (40, 64), (9, 1001), (300, 129)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_dropout(g, dtype, T, H, pad, shift):
    gen = torch.Generator().manual_seed(T * H + pad)
    x = rows(T, H, dtype, gen, pad, shift)
    y = torch.full((T, H), 7.0, dtype=dtype, device="cuda")
    words = (2 ** 40 + 17, 2 ** 64 - 3 - 2 ** 64)      # the counter passes 2^64
    g.dropout(x, y, 0.25, rng_words(*words))
    keep = ref.keep_factor(T, H, 0.25, words)
    close(y, ref.apply_keep(x.cpu().double(), keep), dtype, slack=2.0 ** -22, what="y")
    assert torch.equal(y.cpu() == 0, (keep == 0) | (x.cpu() == 0))


@gpu
def test_dropout_edges(g):
    x = torch.tensor([[float("inf"), float("nan"), 1.0, -2.0] * 64] * 8, device="cuda")
    words = (11, 5)
    y = torch.empty_like(x)
    g.dropout(x, y, 0.5, rng_words(*words))
    dropped = ref.keep_factor(8, 256, 0.5, words) == 0
    assert torch.all(y.cpu()[dropped] == 0)
    assert torch.equal(torch.isfinite(y.cpu())[~dropped], torch.isfinite(x.cpu())[~dropped])
    g.dropout(x, y, 1.0, rng_words(*words))
    assert torch.all(y == 0)
    g.dropout(x, y, 0.0, None)
    assert torch.equal(y.isnan(), x.isnan()) and torch.equal(y[~y.isnan()], x[~x.isnan()])
    z = torch.randn(8, 256, device="cuda")
    want = torch.empty_like(z)
    g.dropout(z, want, 0.5, rng_words(*words))
    g.dropout(z, z, 0.5, rng_words(*words))            # in place
    assert torch.equal(z, want)
    g.dropout(z[:0], want[:0], 0.5, rng_words(*words))  # empty


@gpu
def test_dropout_past_32_bits(g):
    """Elements beyond 2^32 of one call: the last rows of a tall matrix."""
    T, H = 2 ** 19 + 3, 8200
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    g.dropout(x, x, 0.5, rng_words(99, 1))
    groups = H // 8
    n = T - 2
    keep = ref.keep_factor(2, H, 0.5, (99, 1 + n * groups))
    assert torch.equal(x[n:].cpu().double(), keep)
    share = float((x[::64] == 0).float().mean())
    assert abs(share - 0.5) < 1e-3
    del x
    torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("form", ["plain", "strided", "dropout"])
def test_norm_and_gradients(g, dtype, T, H, form):
    if form == "dropout" and T * H > 40000:
        pytest.skip("the reference's mask is slow")
    gen = torch.Generator().manual_seed(T + H)
    pad, shift = {"plain": (0, 0), "strided": (5, 1), "dropout": (8, 0)}[form]
    x, res, dy, dh = (rows(T, H, dtype, gen, pad, shift, s) for s in (1.0, 3.0, 1.0, 0.5))
    w = rows(1, H, dtype, gen)[0]
    p, words, keep = 0.0, None, None
    if form == "dropout":
        p, words = 0.3, (123, 2 ** 33)
        keep = ref.keep_factor(T, H, p, words)
        words = rng_words(*words)
    h, y = torch.empty(T, H, dtype=dtype, device="cuda"), rows(T, H, dtype, gen, pad, shift)
    rstd = torch.empty(T, device="cuda")
    g.add_rms_norm(x, w, y, residual=res, h=h, rstd=rstd, eps=EPS, p=p, rng=words)
    want_h, want_r, want_y = ref.add_rms_norm(x.cpu(), res.cpu(), w.cpu(), EPS, keep)
    sizes = x.cpu().double().abs() * 2 + res.cpu().double().abs()
    close(h, want_h, dtype, sizes, 2.0 ** -22, "h")
    close(rstd, want_r, torch.float32, what="rstd")
    close(y, want_y, dtype, sizes * want_r[:, None] * w.cpu().double().abs(), what="y")

    dx, dres = torch.empty_like(h), torch.empty_like(h)
    dw = torch.empty_like(w)
    g.add_rms_norm_backward(dy, h, w, rstd, dx, dw, dh=dh, dresidual=dres if p else None, p=p,
                            rng=words)
    want = ref.add_rms_norm_backward(dy.cpu(), h.cpu(), w.cpu(), rstd.cpu(), dh.cpu(), keep)
    close(dx, want[0], dtype, want[3] * 2, what="dx")
    close(dw, want[2], dtype, want[4], what="dw")
    if p:
        close(dres, want[1], dtype, want[3], what="dres")


@gpu
@pytest.mark.parametrize("T,H,dtype", [
    (608, 8, torch.bfloat16), (650, 8192, torch.bfloat16), (700, 4104, torch.float16),
    (1400, 2048, torch.float32), (615, 16384, torch.bfloat16), (640, 8192, torch.float32),
    (620, 16384, torch.float32), (609, 10008, torch.float16), (4000, 264, torch.bfloat16)])
@pytest.mark.parametrize("dropout", [False, True])
def test_gradients_of_many_rows(g, T, H, dtype, dropout):
    """Enough rows for several on each SM; strides between rows, with and without dh."""
    gen = torch.Generator().manual_seed(T + H)
    dy, h, dh = (rows(T, H, dtype, gen, 8, 0, s) for s in (1.0, 2.0, 0.5))
    w = rows(1, H, dtype, gen)[0]
    rstd = (0.1 + torch.rand(T, generator=gen)).cuda()
    p, words = (0.25, rng_words(7, 11)) if dropout else (0.0, None)
    dx, dres, dw = (torch.empty(T, H, dtype=dtype, device="cuda"), rows(T, H, dtype, gen, 16),
                    torch.empty_like(w))
    for given in (dh, None):
        g.add_rms_norm_backward(dy, h, w, rstd, dx, dw, dh=given, dresidual=dres, p=p, rng=words)
        want = ref.add_rms_norm_backward(dy.cpu(), h.cpu(), w.cpu(), rstd.cpu(),
                                         None if given is None else given.cpu())
        close(dres, want[1], dtype, want[3], what="dres")
        close(dw, want[2], dtype, want[4], what="dw")
        if dropout:
            # the mask of a plain call on ones, which its own test checks
            keep = torch.empty(T, H, device="cuda")
            g.dropout(torch.ones_like(keep), keep, p, words)
            keep = keep.cpu().double()
            close(dx, ref.apply_keep(want[1], keep), dtype, want[3] * 2, what="dx")
        else:
            assert torch.equal(dx, dres)


@gpu
@pytest.mark.parametrize("T", [1, 40, 151, 153, 303, 305, 607])
@pytest.mark.parametrize("H,dtype", [
    (256, torch.bfloat16), (264, torch.float16), (512, torch.float32), (776, torch.bfloat16),
    (1024, torch.float32), (1032, torch.bfloat16), (2048, torch.float16), (4104, torch.bfloat16)])
@pytest.mark.parametrize("dropout", [False, True])
def test_gradients_from_one_row_to_some_of_each_sm(g, T, H, dtype, dropout):
    """Where a warp, a block and the rows in shared memory take over from each other."""
    test_gradients_of_many_rows(g, T, H, dtype, dropout)


@gpu
@pytest.mark.parametrize("T,H,dtype", [(3, 12288, torch.bfloat16), (153, 12288, torch.float32),
                                       (160, 16392, torch.float16), (170, 32768, torch.bfloat16)])
@pytest.mark.parametrize("dropout", [False, True])
def test_gradients_of_long_rows(g, T, H, dtype, dropout):
    test_gradients_of_many_rows(g, T, H, dtype, dropout)


@gpu
@pytest.mark.parametrize("T,H,dtype", [
    (608, 8, torch.bfloat16), (650, 8192, torch.bfloat16), (700, 4104, torch.float16),
    (1400, 2048, torch.float32), (615, 16384, torch.bfloat16), (640, 8192, torch.float32),
    (620, 16384, torch.float32), (4000, 264, torch.bfloat16)])
@pytest.mark.parametrize("given", [True, False])
def test_norm_with_dropout_of_many_rows(g, T, H, dtype, given):
    """Enough rows for several on each SM; strides between rows, with and without a residual."""
    gen = torch.Generator().manual_seed(T + H)
    x, res = (rows(T, H, dtype, gen, 8, 0, s) for s in (1.0, 3.0))
    w = rows(1, H, dtype, gen)[0]
    p, words = 0.25, rng_words(7, 11)
    h, y = torch.empty(T, H, dtype=dtype, device="cuda"), rows(T, H, dtype, gen, 16)
    rstd = torch.empty(T, device="cuda")
    g.add_rms_norm(x, w, y, residual=res if given else None, h=h, rstd=rstd, eps=EPS, p=p, rng=words)
    # the mask of a plain call on ones, which its own test checks
    keep = torch.empty(T, H, device="cuda")
    g.dropout(torch.ones_like(keep), keep, p, words)
    want_h, want_r, want_y = ref.add_rms_norm(x.cpu(), res.cpu() if given else None, w.cpu(), EPS,
                                              keep.cpu().double())
    sizes = x.cpu().double().abs() * 2 + (res.cpu().double().abs() if given else 0.0)
    close(h, want_h, dtype, sizes, 2.0 ** -22, "h")
    close(rstd, want_r, torch.float32, what="rstd")
    close(y, want_y, dtype, sizes * want_r[:, None] * w.cpu().double().abs(), what="y")


@gpu
def test_norm_without_residual_and_in_place(g):
    gen = torch.Generator().manual_seed(8)
    x, res = rows(33, 520, torch.bfloat16, gen), rows(33, 520, torch.bfloat16, gen)
    w = rows(1, 520, torch.bfloat16, gen)[0]
    y = torch.empty_like(x)
    g.add_rms_norm(x, w, y)                                 # no residual, h not written
    close(y, ref.add_rms_norm(x.cpu(), None, w.cpu(), EPS)[2], torch.bfloat16, what="y")
    h = torch.empty_like(x)
    g.add_rms_norm(x, w, y, residual=res, h=h)
    x2, res2 = x.clone(), res.clone()
    g.add_rms_norm(x2, w, x2, residual=res2, h=res2)        # y over x, h over the residual
    assert torch.equal(x2, y) and torch.equal(res2, h)
    rstd = torch.empty(33, device="cuda")
    g.add_rms_norm(x, w, y, residual=res, h=h, rstd=rstd)
    dy, dh = rows(33, 520, torch.bfloat16, gen), rows(33, 520, torch.bfloat16, gen)
    dx, dr, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    g.add_rms_norm_backward(dy, h, w, rstd, dx, dw, dh=dh, dresidual=dr)
    assert torch.equal(dx, dr)                              # no dropout: the same
    dh2 = dh.clone()
    g.add_rms_norm_backward(dy, h, w, rstd, dh2, dh=dh2)    # dx over dh, no dweight
    assert torch.equal(dh2, dx)


@gpu
@pytest.mark.parametrize("T,H", [(1, 8), (3, 100), (5, 128), (4, 1000), (2, 1001), (9, 4096),
                                 (700, 2056), (1, 32768)])
@pytest.mark.parametrize("form", ["row", "group"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_in_8_bits(g, T, H, form, dtype):
    gen = torch.Generator().manual_seed(T * 3 + H)
    x, res = rows(T, H, dtype, gen), rows(T, H, dtype, gen, scale=4.0)
    if T > 1:
        x[0], res[0] = 0, 0                                 # a row of zeros
    w = rows(1, H, dtype, gen)[0]
    size = H if form == "row" else 128
    groups = -(-H // size)
    y = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(T, groups, device="cuda") if groups > 1 else torch.empty(T, device="cuda")
    h = torch.empty_like(x)
    g.add_rms_norm(x, w, y, residual=res, h=h, scales=scales)
    want_h, _, want = ref.add_rms_norm(x.cpu(), res.cpu(), w.cpu(), EPS)
    close(h, want_h, dtype, x.cpu().double().abs() + res.cpu().double().abs(), 2.0 ** -22, "h")
    padded = torch.zeros(T, groups * size, dtype=torch.float64)
    padded[:, :H] = want
    top = (padded.view(T, groups, size).abs().amax(2) / ref.E4M3_MAX).clamp(min=2.0 ** -126)
    slack = F32 * 8   # the sum that is normalised may cancel
    assert torch.all((scales.cpu().double().view(T, groups) - top).abs() <= slack * top)
    v = want / top.repeat_interleave(size, 1)[:, :H]
    off = (y.cpu().double() - v).abs()
    assert torch.all(off <= (ref.E4M3_UNIT + slack) * v.abs() + ref.E4M3_TINY + slack)
    if T > 1:
        assert torch.all(y[0].float() == 0)


@gpu
def test_norm_past_32_bits(g):
    """More than 2^32 elements: the last rows, forward and backward, with dropout."""
    T, H, dt = 2 ** 19 + 5, 8200, torch.bfloat16
    gen = torch.Generator().manual_seed(77)
    one = rows(1, H, dt, gen)
    x = one.repeat(T, 1)
    x[-3:] = rows(3, H, dt, gen)
    w = rows(1, H, dt, gen)[0]
    y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda")
    words = (3, 2 ** 34)
    g.add_rms_norm(x, w, y, h=h, rstd=rstd, eps=EPS, p=0.2, rng=rng_words(*words))
    groups = H // 8
    keep = ref.keep_factor(3, H, 0.2, (words[0], words[1] + (T - 3) * groups))
    tail = x[-3:].cpu()
    want_h, want_r, want_y = ref.add_rms_norm(tail, None, w.cpu(), EPS, keep)
    close(h[-3:], want_h, dt, what="h")
    close(y[-3:], want_y, dt, what="y")
    dx, dw = y, torch.empty_like(w)
    g.add_rms_norm_backward(x, h, w, rstd, dx, dw, p=0.2, rng=rng_words(*words))
    want = ref.add_rms_norm_backward(tail, h[-3:].cpu(), w.cpu(), rstd[-3:].cpu(), None, keep)
    close(dx[-3:], want[0], dt, want[3] * 2, what="dx")
    total = torch.zeros(H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(total)
    for a in range(0, T, 2 ** 15):
        part = x[a:a + 2 ** 15].double() * h[a:a + 2 ** 15].double() * rstd[a:a + 2 ** 15, None].double()
        total += part.sum(0)
        size += part.abs().sum(0)
    # sums of thousands of rows in 32 bits: 2^-24 for each of the about 2^12 additions of a column
    close(dw, total.cpu(), dt, size.cpu(), 2.0 ** -12, what="dw")
    del x, y, h, dx
    torch.cuda.empty_cache()


@gpu
def test_norm_of_infinities_and_nan(g):
    x = torch.randn(4, 512, device="cuda")
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    w, y = torch.ones(512, device="cuda"), torch.empty(4, 512, device="cuda")
    g.add_rms_norm(x, w, y)
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    assert y[1, 3].isnan() and torch.all(y[1, 4:] == 0) and y[2].isnan().all()
    for groups in (1, 4):
        q = torch.empty(4, 512, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(4, groups, device="cuda")
        g.add_rms_norm(x, w, q, scales=s)
        assert torch.isfinite(s[0]).all() and torch.isfinite(s[3]).all()
        assert s[1, 0].isnan() and s[2].isnan().all()
        assert q[2].float().isnan().all() and torch.isfinite(q[3].float()).all()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", [(1, 9), (5, 33), (3, 257), (40, 1001), (2, 8195), (1300, 77)])
@pytest.mark.parametrize("pad,shift", [(1, 1), (6, 3), (0, 7), (13, 5)])
def test_rows_off_any_boundary_leave_the_rest_alone(g, dtype, T, H, pad, shift):
    """Unaligned inputs and outputs: right values, in place too, and no element between rows written."""
    gen = torch.Generator().manual_seed(T + H + pad)

    def room(kind=dtype):
        """An output of canaries: (buffer, its T x H window, the mask of what lies outside)."""
        buf = torch.full((T * (H + pad) + shift + 16,), 5.0, device="cuda").to(kind)
        outside = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
        outside[shift:shift + T * (H + pad)].view(T, H + pad)[:, :H] = False
        return buf, buf[shift:shift + T * (H + pad)].view(T, H + pad)[:, :H], outside

    def untouched(*rooms):
        for buf, _, outside in rooms:
            assert torch.all(buf.float()[outside] == 5.0)

    x, res, dy = (rows(T, H, dtype, gen, pad, 8 - shift) for _ in range(3))
    w = rows(1, H, dtype, gen, 0, 1)[0]
    ry, rh, rx, rd = (room() for _ in range(4))
    rstd = torch.empty(T, device="cuda")
    g.add_rms_norm(x, w, ry[1], residual=res, h=rh[1], rstd=rstd, eps=EPS)
    want_h, want_r, want_y = ref.add_rms_norm(x.cpu(), res.cpu(), w.cpu(), EPS)
    sizes = x.cpu().double().abs() + res.cpu().double().abs()
    close(rh[1], want_h, dtype, sizes, 2.0 ** -22, "h")
    close(ry[1], want_y, dtype, sizes * want_r[:, None] * w.cpu().double().abs(), what="y")
    dw = torch.empty(H + 1, dtype=dtype, device="cuda")[1:]
    g.add_rms_norm_backward(dy, rh[1], w, rstd, rx[1], dw, dresidual=rd[1])
    want = ref.add_rms_norm_backward(dy.cpu(), rh[1].cpu(), w.cpu(), rstd.cpu())
    close(rx[1], want[0], dtype, want[3], what="dx")
    close(dw, want[2], dtype, want[4], what="dw")
    assert torch.equal(rx[1], rd[1])
    untouched(ry, rh, rx, rd)

    r8 = room(torch.float8_e4m3fn)
    scales = torch.empty(T, -(-H // 128), device="cuda")
    g.add_rms_norm(x, w, r8[1], residual=res, scales=scales)
    v = want_y / scales.cpu().double().repeat_interleave(128, 1)[:, :H]
    off = (r8[1].float().cpu().double() - v).abs()
    assert torch.all(off <= (ref.E4M3_UNIT + 8 * F32) * v.abs() + ref.E4M3_TINY + 8 * F32)
    untouched(r8)

    y, h = ry[1].clone(), rh[1].clone()
    rx[1].copy_(x)
    rd[1].copy_(res)
    g.add_rms_norm(rx[1], w, rx[1], residual=rd[1], h=rd[1], eps=EPS)     # in place
    assert torch.equal(rx[1], y) and torch.equal(rd[1], h)
    words = rng_words(9, 2)
    g.dropout(x, ry[1], 0.4, words)
    rx[1].copy_(x)
    g.dropout(rx[1], rx[1], 0.4, words)
    keep = ref.keep_factor(T, H, 0.4, (9, 2)) if T * H < 50000 else None
    assert torch.equal(rx[1], ry[1])
    if keep is not None:
        close(ry[1], ref.apply_keep(x.cpu().double(), keep), dtype, slack=2.0 ** -22, what="dropout")
    untouched(rx, rd, ry)


@gpu
def test_empty_and_no_rows(g):
    w = torch.randn(64, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    r = torch.empty(0, device="cuda")
    g.add_rms_norm(none, w, none, rstd=r)
    dw = torch.full_like(w, 3.0)
    g.add_rms_norm_backward(none, none, w, r, none, dw)
    torch.cuda.synchronize()
    assert torch.all(dw == 0)


@gpu
def test_same_bits_on_another_stream_and_in_a_graph(g):
    gen = torch.Generator().manual_seed(21)
    T, H, dt = 2000, 1536, torch.bfloat16
    x, res, dy = (rows(T, H, dt, gen) for _ in range(3))
    w = rows(1, H, dt, gen)[0]
    words = rng_words(4, 10)
    out = {k: torch.empty_like(x) for k in ("h", "y", "dx", "dr")}
    rstd, dw = torch.empty(T, device="cuda"), torch.empty_like(w)

    def both(stream=None):
        g.add_rms_norm(x, w, out["y"], residual=res, h=out["h"], rstd=rstd, p=0.1, rng=words,
                       stream=stream)
        g.add_rms_norm_backward(dy, out["h"], w, rstd, out["dx"], dw, dresidual=out["dr"], p=0.1,
                                rng=words, stream=stream)

    def snapshot():
        torch.cuda.synchronize()
        got = {**{k: v.clone() for k, v in out.items()}, "rstd": rstd.clone(), "dw": dw.clone()}
        for v in (*out.values(), rstd, dw):
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        return got

    both()
    first = snapshot()
    s = torch.cuda.Stream()
    both(s)
    second = snapshot()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    graph.replay()
    third = snapshot()
    for k in first:
        assert torch.equal(first[k], second[k]) and torch.equal(first[k], third[k]), k
    words[1] += T * H // 8          # the replay draws another mask
    graph.replay()
    fourth = snapshot()
    assert not torch.equal(fourth["dx"] == 0, third["dx"] == 0)
    both()
    assert torch.equal(fourth["dx"], out["dx"])


@gpu
def test_refusals(g):
    dt = torch.bfloat16
    x, w, y = torch.randn(4, 64, device="cuda").to(dt), torch.ones(64, device="cuda", dtype=dt), \
        torch.full((4, 64), 9.0, device="cuda", dtype=dt)
    r = torch.empty(4, device="cuda")
    words = rng_words(1, 2)
    for call in (
        lambda: g.dropout(x, y[:3], 0.1, words),                       # another shape
        lambda: g.dropout(x, y.float(), 0.1, words),                   # another type
        lambda: g.dropout(x, y, 0.1, None),                            # no generator
        lambda: g.dropout(x, y, 1.5, words),                           # p out of range
        lambda: g.dropout(x, y, float("nan"), words),
        lambda: g.dropout(x.cpu(), y, 0.1, words),                     # on the host
        lambda: g.dropout(x.t(), y.t(), 0.1, words),                   # columns apart
        lambda: g.dropout(x[0], y[0], 0.1, words),                     # one dimension
        lambda: g.add_rms_norm(x, w[:63], y),
        lambda: g.add_rms_norm(x, w.float(), y),
        lambda: g.add_rms_norm(x, w, y, rstd=r[:2]),
        lambda: g.add_rms_norm(x, w, y, scales=r),                     # scales, and y not in 8 bits
        lambda: g.add_rms_norm(x.double(), w.double(), y.double()),
        lambda: g.add_rms_norm(x[:1].expand(4, 64), w, y),             # rows that overlap
    ):
        with pytest.raises(ValueError):
            call()
    buf = torch.randn(5 * 64, device="cuda").to(dt)
    a, b = buf[:256].view(4, 64), buf[64:].view(4, 64)
    wide = torch.zeros(1, 32776, device="cuda", dtype=dt)
    for call in (
        lambda: g.dropout(a, b, 0.1, words),                           # overlapping rows
        lambda: g.add_rms_norm(a, w, y, h=b),
        lambda: g.add_rms_norm(x, w, y, h=y),                          # both outputs in one place
        lambda: g.add_rms_norm(x, w, y, residual=y),                   # y over the residual
        lambda: g.add_rms_norm(x, w, y, eps=-1.0),
        lambda: g.add_rms_norm(wide, wide[0], torch.empty_like(wide)),  # beyond 32768 columns
        lambda: g.add_rms_norm_backward(y, x, w, r, x),                # dx over h
        lambda: g.add_rms_norm_backward(y, x, w, r, y, dresidual=y),
    ):
        with pytest.raises(gemm_ws.GemmWSError) as e:
            call()
        assert e.value.status == gemm_ws.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.all(y == 9.0)
    lib, vp = g.lib, ctypes.c_void_p
    assert lib.gemm_ws_dropout(g.handle, 7, x.data_ptr(), 64, y.data_ptr(), 64, 4, 64, 0.0, None,
                               vp(0)) == gemm_ws.ERR_INVALID_ARG
    assert lib.gemm_ws_dropout(g.handle, 0, None, 64, y.data_ptr(), 64, 4, 64, 0.0, None,
                               vp(0)) == gemm_ws.ERR_INVALID_ARG
    assert lib.gemm_ws_dropout(g.handle, 0, x.data_ptr(), 63, y.data_ptr(), 64, 4, 64, 0.0, None,
                               vp(0)) == gemm_ws.ERR_INVALID_ARG
