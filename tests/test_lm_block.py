"""The norms around a block with gate and scaled residual, their gradients, and rows in 8-bit integers, against plain
implementations in 64 bits.

Tolerances, fixed before the first run: an output is rounded once to its type (UNIT of its value, or TINY), and the
32-bit arithmetic before that is within F32 = 2^-16 of the magnitudes that it adds: products of up to eight factors, each
off by 2^-24 (a root by 2^-22), and sums in trees and chains of at most a few hundred terms a thread.
"""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import build, gemm_ws
from tests import lm_block_reference as ref
from tests.lm_reference import E4M3_MAX, E4M3_TINY, E4M3_UNIT, TINY, UNIT

F32 = 2.0 ** -16
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-6
gpu = pytest.mark.gpu


# ------------------------------------------------------------------ on the CPU

@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "cols", "rows"])
def test_reference_gradient_against_differences(post, gate):
    gen = torch.Generator().manual_seed(11)
    T, H, alpha = 4, 10, 0.7
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    at = {"x": rand(T, H), "residual": rand(T, H), "weight": rand(H)}
    if post:
        at["post"] = rand(H)
    if gate != "none":
        at["gate"] = rand(H) if gate == "cols" else rand(T, H)
    dy, dh = rand(T, H), rand(T, H)

    def value(v):
        h, y = ref.block_norm(alpha=alpha, eps=EPS, **v)[:2]
        return float((y * dy).sum() + (h * dh).sum())

    h, _, r1, r2, _ = ref.block_norm(alpha=alpha, eps=EPS, **at)
    grads, _ = ref.block_norm_backward(dy, at["x"], h, at["weight"], r2, at.get("post"), r1, at.get("gate"), alpha, dh)
    names = {"x": "dx", "residual": "dresidual", "weight": "dweight", "post": "dpost_weight", "gate": "dgate"}
    e = 1e-5
    for k, v in at.items():
        step = rand(*v.shape)
        slope = (value({**at, k: v + e * step}) - value({**at, k: v - e * step})) / (2 * e)
        assert abs(slope - float((grads[names[k]] * step).sum())) < 1e-6, k


def test_null_handle_is_refused_without_a_gpu():
    build.ensure_built()
    lib = gemm_ws.load_library()
    bad = gemm_ws.ERR_INVALID_ARG
    assert lib.gemm_ws_block_norm(None, 0, None, 8, None, 8, None, 0, None, None, None, 8, None, 8, 0, None, None, None,
                                  1, 8, 1.0, EPS, None) == bad
    assert lib.gemm_ws_block_norm_backward(None, 0, None, 8, None, 8, None, 8, None, 8, None, 0, None, None, None, None,
                                           None, 8, None, 8, None, 0, None, None, 1, 8, 1.0, None) == bad
    assert lib.gemm_ws_quantize_rows(None, 0, None, 8, None, 8, None, 1, 8, None) == bad


# ------------------------------------------------------------------ on the GPU

@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    handle.close()


def rows(T, H, dtype, gen, pad=0, shift=0, scale=1.0):
    """T x H on the GPU, `pad` elements between rows, `shift` elements past an aligned address."""
    buf = (scale * torch.randn(T * (H + pad) + shift, generator=gen)).to(dtype).cuda()
    return buf[shift:].view(T, H + pad)[:, :H]


def output(T, H, dtype, pad=0, shift=0):
    """Like rows, and the buffer around it, all of 7."""
    buf = torch.full((T * (H + pad) + shift,), 7, dtype=torch.float32).to(dtype).cuda()
    return buf[shift:].view(T, H + pad)[:, :H], buf


def untouched(buf, view, H):
    """What lies between the rows is still 7."""
    around = torch.ones_like(buf, dtype=torch.bool)
    mask = around.as_strided(view.shape, view.stride(), view.storage_offset())
    mask[:] = False
    return bool((buf.float()[around] == 7).all())


def close(got, want, dtype, size=None, slack=F32, what=""):
    got = got.detach().cpu().double()
    size = want.abs() if size is None else size
    tol = UNIT[dtype] * want.abs() + slack * size + TINY[dtype]
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / tol).max()):.3g} of the tolerance")


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (2, 1000), (7, 1024), (3, 1032), (2, 4096), (1, 8192), (3, 8191), (2, 16384),
          (1300, 40), (700, 2048), (331, 1001), (310, 520), (2500, 136)]


def block_inputs(T, H, dtype, gate, post, seed, pad=0, shift=0):
    gen = torch.Generator().manual_seed(seed)
    vec = lambda s: (s + 0.2 * torch.randn(H, generator=gen)).to(dtype).cuda()  # noqa: E731
    v = {"x": rows(T, H, dtype, gen, pad, shift, 2.0), "residual": rows(T, H, dtype, gen, pad, shift, 3.0),
         "weight": vec(1.0), "post": vec(1.0) if post else None, "gate": None}
    if gate == "cols":
        v["gate"] = vec(0.5)
    elif gate == "rows":
        v["gate"] = rows(T, H, dtype, gen, pad, shift)
    return v, gen


def on_cpu(v):
    return {k: None if t is None else t.cpu() for k, t in v.items()}


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate,post,alpha,pad,shift", [("none", True, 1.0, 0, 0), ("cols", True, 0.9, 8, 0),
                                                       ("rows", False, 2.5, 0, 0), ("rows", True, 1.0, 3, 1),
                                                       ("cols", False, 1.0, 5, 3), ("none", False, 0.5, 0, 0)])
def test_block_norm_and_gradients(g, dtype, T, H, gate, post, alpha, pad, shift):
    v, gen = block_inputs(T, H, dtype, gate, post, T + H, pad, shift)
    c = on_cpu(v)
    y, ybuf = output(T, H, dtype, pad, shift)
    h, hbuf = output(T, H, dtype, pad, shift)
    r1 = torch.full((T,), 7.0, device="cuda") if post else None
    r2 = torch.full((T,), 7.0, device="cuda")
    g.block_norm(v["x"], v["residual"], v["weight"], y, post_weight=v["post"], gate=v["gate"], alpha=alpha, h=h,
                 post_rstd=r1, rstd=r2, eps=EPS)
    wh, wy, w1, w2, size = ref.block_norm(alpha=alpha, eps=EPS, **c)
    close(h, wh, dtype, size, what="h")
    spread = (size.norm(dim=1) / wh.norm(dim=1).clamp(min=1e-30))[:, None]
    scale_y = size * w2[:, None] * c["weight"].double().abs()
    close(y, wy, dtype, scale_y + wy.abs() * (1 + spread), what="y")
    assert bool(((r2.cpu().double() - w2).abs() <= F32 * w2 * (1 + spread[:, 0])).all())
    if post:
        assert bool(((r1.cpu().double() - w1).abs() <= F32 * w1).all())
    assert untouched(ybuf, y, H) and untouched(hbuf, h, H)

    dy, dh = rows(T, H, dtype, gen, pad, shift), rows(T, H, dtype, gen, pad, shift, 0.5)
    dx, dxbuf = output(T, H, dtype, pad, shift)
    dres, dresbuf = output(T, H, dtype, pad, shift)
    outs = {"dx": dx, "dresidual": dres, "dweight": torch.full((H,), 7.0, dtype=dtype, device="cuda")}
    if post:
        outs["dpost_weight"] = torch.full((H,), 7.0, dtype=dtype, device="cuda")
    if gate == "cols":
        outs["dgate"] = torch.full((H,), 7.0, dtype=dtype, device="cuda")
    elif gate == "rows":
        outs["dgate"], gbuf = output(T, H, dtype, pad, shift)
    g.block_norm_backward(dy, v["x"], h, v["weight"], r2, post_weight=v["post"], post_rstd=r1, gate=v["gate"],
                          alpha=alpha, dh=dh, **outs)
    want, sizes = ref.block_norm_backward(dy.cpu(), c["x"], h.cpu(), c["weight"], r2.cpu(), c["post"],
                                          None if r1 is None else r1.cpu(), c["gate"], alpha, dh.cpu())
    assert set(want) == set(outs)
    for k in want:
        close(outs[k], want[k], dtype, sizes[k], what=k)
    assert untouched(dxbuf, dx, H) and untouched(dresbuf, dres, H)
    if gate == "rows":
        assert untouched(gbuf, outs["dgate"], H)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,pad", [(1, 1, 0), (3, 100, 0), (2, 128, 0), (5, 1000, 8), (4, 4104, 0), (2, 8191, 1),
                                     (700, 256, 0), (1, 16384, 0), (331, 1001, 2)])
@pytest.mark.parametrize("kind", ["row", "group", "int8"])
def test_block_norm_in_8_bits(g, dtype, T, H, pad, kind):
    v, _ = block_inputs(T, H, dtype, "cols", True, T * H, pad)
    c = on_cpu(v)
    groups = (H + 127) // 128 if kind == "group" else 1
    scales = torch.full((T, groups), 7.0, device="cuda")
    h, _ = output(T, H, dtype, pad)
    q_type = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    y, ybuf = output(T, H, q_type, pad)
    g.block_norm(v["x"], v["residual"], v["weight"], y, post_weight=v["post"], gate=v["gate"], h=h, scales=scales, eps=EPS)
    wh, wy, _, w2, size = ref.block_norm(alpha=1.0, eps=EPS, **c)
    close(h, wh, dtype, size, what="h")
    if kind == "group" and groups == 1:
        kind = "row"   # the same thing
    spread = (size.norm(dim=1) / wh.norm(dim=1))[:, None]
    err = F32 * (size * w2[:, None] * c["weight"].double().abs() + wy.abs() * (1 + spread))   # of y in 32 bits
    width = 128 if kind == "group" else H
    most = 127.0 if kind == "int8" else E4M3_MAX
    got, s = y.cpu().float().double(), scales.cpu().double()
    for k in range(groups):
        part = slice(k * width, min(H, (k + 1) * width))
        top = wy[:, part].abs().amax(1)
        assert bool(((s[:, k] - top / most).abs() <= err[:, part].amax(1) / most + 2.0 ** -23 * top / most).all())
        back = got[:, part] * s[:, k:k + 1]
        if kind == "int8":
            tol = s[:, k:k + 1] / 2 * (1 + 2.0 ** -16) + err[:, part]   # half a step
        else:
            tol = E4M3_UNIT * wy[:, part].abs() * (1 + 2.0 ** -16) + E4M3_TINY * s[:, k:k + 1] + err[:, part]
        assert bool(((back - wy[:, part]).abs() <= tol).all())
    assert untouched(ybuf.float() if kind == "int8" else ybuf, y, H)


@gpu
def test_block_norm_8_bits_are_roundings_of_its_own_row(g):
    """Each integer is the rounding of its fp32 quotient: rows whose norm is exact in 32 bits show it."""
    T, H = 40, 256
    gen = torch.Generator().manual_seed(5)
    x = torch.zeros(T, H, device="cuda")
    res = torch.randint(-2000, 2000, (T, H), generator=gen).float()
    res[:, 0] = 2032.0
    # y = h * rstd * weight: whole numbers times one factor
    y = torch.empty(T, H, dtype=torch.int8, device="cuda")
    scales, r2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    one = torch.ones(H, device="cuda")
    g.block_norm(x, res.cuda(), one, y, rstd=r2, scales=scales)
    v = res * r2.cpu()[:, None]
    want = torch.round(v / scales.cpu()[:, None])
    assert torch.equal(y.cpu().float(), want)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,pad,shift", [(1, 1, 0, 0), (3, 7, 0, 0), (5, 64, 0, 0), (9, 1001, 3, 1), (2, 8192, 0, 0),
                                           (300, 129, 0, 0), (2, 32768, 0, 0), (1, 32767, 0, 0), (2000, 256, 0, 0),
                                           (400, 8192, 0, 0), (64, 2056, 8, 0)])
def test_quantize_rows(g, dtype, T, H, pad, shift):
    gen = torch.Generator().manual_seed(T + H)
    x = rows(T, H, dtype, gen, pad, shift)
    x *= torch.exp(2.0 * torch.randn(T, 1, generator=gen)).to(dtype).cuda()
    x[T // 2] = 0   # a row of zeros has the smallest scale
    y, buf = output(T, H, torch.int8, pad, shift)
    scales = torch.full((T,), 7.0, device="cuda")
    g.quantize_rows(x, y, scales)
    q, s = ref.quantize_rows(x.cpu())
    assert torch.equal(scales.cpu(), s) and torch.equal(y.cpu(), q)
    assert untouched(buf.float(), y, H)


@gpu
def test_quantize_rows_ties_and_edges(g):
    """Quotients on and next to the middle of two integers; denormals; infinities and NaN."""
    base = torch.arange(-127, 128, dtype=torch.float32)
    half = torch.arange(-126, 127, dtype=torch.float32) + 0.5
    near = torch.cat([torch.nextafter(half, half + 1), torch.nextafter(half, half - 1)])
    line = torch.cat([base, half, near])
    line = torch.cat([line, torch.zeros(1024 - len(line))])
    x = torch.stack([line * s for s in (1.0, 3.0, 7.0, 0.3, 1e-30, 1e30, 2.0 ** -140)] +
                    [line.clone() for _ in range(3)])
    x[7, 5], x[8, 6], x[9, 1023] = float("inf"), float("nan"), float("-inf")
    y = torch.full(x.shape, 7, dtype=torch.int8, device="cuda")
    scales = torch.empty(len(x), device="cuda")
    g.quantize_rows(x.cuda(), y, scales)
    q, s = ref.quantize_rows(x)
    assert torch.equal(torch.nan_to_num(scales.cpu(), nan=-1.0), torch.nan_to_num(s, nan=-1.0))
    assert torch.equal(y.cpu(), q)


@gpu
@pytest.mark.parametrize("H", [64, 1001])
def test_rows_of_infinities_and_nan_stay_their_own(g, H):
    """A NaN or an infinity in one row leaves the other rows as they are, in every output form."""
    v, gen = block_inputs(6, H, torch.bfloat16, "rows", True, 3)
    bad = v["x"].clone()
    bad[1, 3], bad[3, H - 1] = float("nan"), float("inf")
    for q_type in (torch.bfloat16, torch.int8):
        got = []
        for x in (v["x"], bad):
            y = torch.zeros(6, H, dtype=q_type, device="cuda")
            scales = torch.zeros(6, device="cuda") if q_type is torch.int8 else None
            g.block_norm(x, v["residual"], v["weight"], y, post_weight=v["post"], gate=v["gate"], scales=scales)
            got.append((y.float().cpu(), None if scales is None else scales.cpu()))
        for r in (0, 2, 4, 5):
            assert torch.equal(got[0][0][r], got[1][0][r])
        if q_type is torch.int8:
            assert bool(torch.isnan(got[1][1][1])) and not got[1][0][1].any()
        else:
            assert bool(torch.isnan(got[1][0][1]).all())


@gpu
@pytest.mark.parametrize("H", [512, 515])
@pytest.mark.parametrize("T", [3, 700])
def test_in_place(g, T, H):
    """h over x or the residual, y over x; dx and dresidual over dy and dh."""
    v, gen = block_inputs(T, H, torch.bfloat16, "cols", True, 9)
    new = lambda: torch.empty(T, H, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y, h, r1, r2 = new(), new(), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    kw = dict(post_weight=v["post"], gate=v["gate"], alpha=0.8)
    g.block_norm(v["x"], v["residual"], v["weight"], y, h=h, post_rstd=r1, rstd=r2, **kw)
    x, res = v["x"].clone(), v["residual"].clone()
    g.block_norm(x, res, v["weight"], x, h=res, **kw)
    assert torch.equal(x, y) and torch.equal(res, h)
    x2, y2 = v["x"].clone(), new()
    g.block_norm(x2, v["residual"], v["weight"], y2, h=x2, **kw)
    assert torch.equal(x2, h) and torch.equal(y2, y)
    dy, dh = rows(T, H, torch.bfloat16, gen), rows(T, H, torch.bfloat16, gen)
    dx, dres = new(), new()
    bw = dict(post_weight=v["post"], post_rstd=r1, gate=v["gate"], alpha=0.8)
    g.block_norm_backward(dy, v["x"], h, v["weight"], r2, dx, dres, dh=dh, **bw)
    for first in (True, False):
        a, b = dy.clone(), dh.clone()
        out = (a, b) if first else (b, a)
        g.block_norm_backward(a, v["x"], h, v["weight"], r2, out[0], out[1], dh=b, **bw)
        assert torch.equal(out[0], dx) and torch.equal(out[1], dres)


@gpu
def test_same_bits_on_every_run_and_in_a_graph(g):
    T, H = 1500, 1024
    v, gen = block_inputs(T, H, torch.bfloat16, "cols", True, 21)
    dy = rows(T, H, torch.bfloat16, gen)
    new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    r1, r2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")

    def step(out):
        g.block_norm(v["x"], v["residual"], v["weight"], out["y"], post_weight=v["post"], gate=v["gate"], h=out["h"],
                     post_rstd=r1, rstd=r2)
        g.block_norm_backward(dy, v["x"], out["h"], v["weight"], r2, out["dx"], out["dres"], post_weight=v["post"],
                              post_rstd=r1, gate=v["gate"], dweight=out["dw"], dpost_weight=out["dp"], dgate=out["dg"])

    def fresh():
        return {k: new(T, H) for k in ("y", "h", "dx", "dres")} | {k: new(H) for k in ("dw", "dp", "dg")}

    first, second, third = fresh(), fresh(), fresh()
    step(first)
    step(second)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(third)
    for _ in range(3):
        for t in third.values():
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], second[k]) and torch.equal(first[k], third[k]), k
    assert g.query_status() == gemm_ws.OK


@gpu
def test_gradients_of_nothing_are_zero(g):
    H = 40
    e = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, device="cuda")
    dw, dp, dg = (torch.full((H,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    g.block_norm(e, e, w, e, post_weight=w, gate=w)
    g.block_norm_backward(e, e, e, w, none, e, post_weight=w, post_rstd=none, gate=w, dweight=dw, dpost_weight=dp,
                          dgate=dg)
    assert not dw.any() and not dp.any() and not dg.any()
    g.quantize_rows(e, torch.empty(0, H, dtype=torch.int8, device="cuda"), none)


@gpu
def test_only_what_is_asked_for(g):
    """Each gradient alone has the bits that it has with the others."""
    T, H = 333, 264
    v, gen = block_inputs(T, H, torch.bfloat16, "cols", True, 2)
    dy = rows(T, H, torch.bfloat16, gen)
    new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    h, y, r1, r2 = new(T, H), new(T, H), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    g.block_norm(v["x"], v["residual"], v["weight"], y, post_weight=v["post"], gate=v["gate"], h=h, post_rstd=r1, rstd=r2)
    kw = dict(post_weight=v["post"], post_rstd=r1, gate=v["gate"])
    full = {"dweight": new(H), "dpost_weight": new(H), "dgate": new(H)}
    dx = new(T, H)
    g.block_norm_backward(dy, v["x"], h, v["weight"], r2, dx, **full, **kw)
    for k in full:
        one, dx1 = new(H), new(T, H)
        g.block_norm_backward(dy, v["x"], h, v["weight"], r2, dx1, **{k: one}, **kw)
        assert torch.equal(one, full[k]) and torch.equal(dx1, dx), k


@gpu
def test_refusals(g):
    T, H = 4, 64
    v, _ = block_inputs(T, H, torch.bfloat16, "cols", True, 1)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(T, device="cuda")
    x, res, w = v["x"], v["residual"], v["weight"]

    def refused(error, fn, *a, **k):
        with pytest.raises(error):
            fn(*a, **k)

    for bad in (float("nan"), float("inf")):
        refused(gemm_ws.GemmWSError, g.block_norm, x, res, w, y, alpha=bad)
    refused(gemm_ws.GemmWSError, g.block_norm, x, res, w, y, eps=-1.0)
    refused(gemm_ws.GemmWSError, g.block_norm, x, res, w, y, post_rstd=f)          # no norm after the block
    refused(gemm_ws.GemmWSError, g.block_norm, x, res, w, res)                     # y over the residual
    refused(gemm_ws.GemmWSError, g.block_norm, x, res, w, y, h=y)
    refused(ValueError, g.block_norm, x, None, w, y)
    refused(ValueError, g.block_norm, x, res, w, y, gate=w[:32])
    refused(ValueError, g.block_norm, x, res, w, y.float())
    refused(ValueError, g.block_norm, x, res, w, torch.empty(T, H, dtype=torch.int8, device="cuda"))   # no scales
    refused(ValueError, g.block_norm, x, res, w, y.t().contiguous().t())
    refused(ValueError, g.block_norm, x.cpu(), res, w, y)
    wide = torch.empty(1, 16385, dtype=torch.bfloat16, device="cuda")
    ww = torch.empty(16385, dtype=torch.bfloat16, device="cuda")
    refused(gemm_ws.GemmWSError, g.block_norm, wide, wide, ww, torch.empty_like(wide))
    # gradients
    refused(gemm_ws.GemmWSError, g.block_norm_backward, y, x, res, w, f, x)        # dx over x
    refused(gemm_ws.GemmWSError, g.block_norm_backward, y, x, res, w, f, torch.empty_like(y), post_weight=w)
    refused(gemm_ws.GemmWSError, g.block_norm_backward, y, x, res, w, f, torch.empty_like(y), dpost_weight=torch.empty_like(w))
    refused(ValueError, g.block_norm_backward, y, x, res, w, f, torch.empty_like(y), dgate=torch.empty_like(w))
    refused(ValueError, g.block_norm_backward, y, x, res, w, f, torch.empty_like(y), gate=w, dgate=torch.empty_like(y))
    refused(gemm_ws.GemmWSError, g.block_norm_backward, y, x, res, w, f, torch.empty_like(y), dweight=w)
    # rows in 8-bit integers
    q = torch.empty(T, H, dtype=torch.int8, device="cuda")
    refused(ValueError, g.quantize_rows, x, y, f)
    refused(ValueError, g.quantize_rows, x, q, f[:2])
    refused(ValueError, g.quantize_rows, q, q, f)
    refused(gemm_ws.GemmWSError, g.quantize_rows, torch.empty(1, 32769, device="cuda"),
            torch.empty(1, 32769, dtype=torch.int8, device="cuda"), f[:1])
    lib = g.lib
    assert lib.gemm_ws_quantize_rows(g.handle, 0, x.data_ptr(), H, x.data_ptr(), H, f.data_ptr(), T, H, None) == \
        gemm_ws.ERR_INVALID_ARG   # over its input
    assert lib.gemm_ws_quantize_rows(g.handle, 3, x.data_ptr(), H, q.data_ptr(), H, f.data_ptr(), T, H, None) == \
        gemm_ws.ERR_INVALID_ARG
    assert g.query_status() == gemm_ws.OK
