"""The linear cross entropy and its gradients, against plain implementations in 64 bits.

Tolerances, fixed before the first run. Logits: bf16 products are exact in fp32 and their sums
over `hidden` are off by at most hidden * 2^-24 of the terms' magnitudes (far less in practice;
sqrt(hidden) of them is allowed for). exp and log add a few 2^-22. Gradients: the logits'
gradient is rounded to bf16 once (2^-8 of each term of the sums; the test allows that of the
terms' magnitudes, though roundings average out), and the output once more.
"""
from __future__ import annotations

import math

import pytest
import torch

from async_pipelines_gb300 import build, gemm_ws
from tests import lm_reference as ref

IGNORE = -100


# ------------------------------------------------------------------ on the CPU

def test_reference_gradient_against_differences():
    gen = torch.Generator().manual_seed(5)
    x, v = (torch.randn(6, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    w, u = (torch.randn(11, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    t = torch.tensor([3, IGNORE, 0, 10, 3, IGNORE])
    grad = torch.rand(6, generator=gen, dtype=torch.float64)

    def value(x_, w_):
        return float((ref.linear_cross_entropy(x_, w_, t, IGNORE)[0] * grad).sum())

    dx, dw, _, _ = ref.linear_cross_entropy_backward(x, w, t, grad, IGNORE)
    e = 1e-5
    assert abs((value(x + e * v, w) - value(x - e * v, w)) / (2 * e) - float((dx * v).sum())) < 1e-7
    assert abs((value(x, w + e * u) - value(x, w - e * u)) / (2 * e) - float((dw * u).sum())) < 1e-7


def test_null_handle_is_refused_without_a_gpu():
    build.ensure_built()
    lib = gemm_ws.load_library()
    bad = gemm_ws.ERR_INVALID_ARG
    assert lib.gemm_ws_linear_ce(None, None, 8, None, 8, None, 8, IGNORE, None, None, None, 1, 8, 8,
                                 None, 0, None) == bad
    assert lib.gemm_ws_linear_ce_backward(None, None, 8, None, 8, None, 8, IGNORE, None, None, 0,
                                          None, 8, None, 8, 1, 8, 8, None, 0, None) == bad
    assert lib.gemm_ws_linear_ce_workspace(None, 1, 8, 8, 0) == -bad


# ------------------------------------------------------------------ on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


def make(T, H, V, seed, ignored=0.0, pad=0, shift=0, int32=False):
    """x, weight, targets on the CPU; x's logits are a few units wide, some targets likely."""
    gen = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, H, generator=gen) * 1.5 / math.sqrt(H)).bfloat16()
    t = torch.randint(V, (T,), generator=gen)
    up = torch.rand(T, 1, generator=gen) * 5.0
    x = (torch.randn(T, H, generator=gen) + up * w[t].float()).bfloat16()
    t = torch.where(torch.rand(T, generator=gen) < ignored, IGNORE, t)
    return x, w, t.int() if int32 else t


def on_gpu(m, pad=0, shift=0):
    """The matrix on the GPU, `pad` elements between rows, `shift` past an aligned address."""
    T, H = m.shape
    buf = torch.full((T * (H + pad) + shift,), float("nan"), dtype=m.dtype, device="cuda")
    out = buf[shift:].view(T, H + pad)[:, :H]
    out.copy_(m)
    return out


def forward(g, x, w, t, **kw):
    T = x.shape[0]
    loss, lse, mean = (torch.full((n,), 5.0, device="cuda") for n in (T, T, 2))
    g.linear_cross_entropy(x, w, t, loss, lse, mean=mean, **kw)
    return loss, lse, mean


def check_forward(got, x, w, t):
    loss, lse, mean = (v.cpu().double() for v in got)
    t = t.long()
    want = ref.linear_cross_entropy(x, w, t, IGNORE)
    H = x.shape[1]
    size = (x.double().abs() @ w.double().abs().T).amax(1)    # a logit's terms' magnitudes
    tol = math.sqrt(H) * 2.0 ** -23 * size + 2.0 ** -20 * (1 + want[1].abs())
    assert torch.all((lse - want[1]).abs() <= tol)
    assert torch.all((loss - want[0]).abs() <= 2 * tol)
    assert abs(mean[0] - want[2]) <= float(2 * tol.max()) + 2.0 ** -20 * abs(want[2])
    n = int((t != IGNORE).sum())
    assert abs(mean[1] - (1.0 / n if n else 0.0)) <= 2.0 ** -24


def check_backward(dx, dw, x, w, t, grad):
    want = ref.linear_cross_entropy_backward(x, w, t.long(), grad, IGNORE)
    u = 2.0 ** -8
    for name, got, i in (("dx", dx, 0), ("dw", dw, 1)):
        got = got.cpu().double()
        # the exponent's error is the logit's, a few 2^-20; it counts like a rounding
        tol = u * want[i].abs() + (u + 2.0 ** -14) * want[2 + i] + 2.0 ** -120
        bad = ~((got - want[i]).abs() <= tol)
        assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off"
        # and over all elements the roundings average out
        off = float((got - want[i]).norm()), float(want[i].norm())
        assert off[0] <= 4e-3 * off[1], f"{name}: relative error {off[0] / max(off[1], 1e-300):.3g}"


CASES = [
    (1, 8, 1), (1, 8, 9), (2, 64, 100), (1, 4096, 5000), (7, 72, 1003), (61, 256, 2000),
    (128, 512, 256), (129, 136, 777), (200, 1000, 4097), (256, 256, 1000), (300, 64, 40000),
    (1000, 200, 30001), (2500, 512, 8191), (640, 2048, 6000),
]


@gpu
@pytest.mark.parametrize("T,H,V", CASES)
@pytest.mark.parametrize("ignored", [0.0, 0.4])
def test_loss_and_gradients(g, T, H, V, ignored):
    x, w, t = make(T, H, V, T + H + V, ignored, int32=T % 2 == 1)
    xd, wd, td = x.cuda(), w.cuda(), t.cuda()
    got = forward(g, xd, wd, td)
    check_forward(got, x, w, t)
    dx, dw = torch.full_like(xd, 3.0), torch.full_like(wd, 3.0)
    g.linear_cross_entropy_backward(xd, wd, td, got[1], got[2][1:], dx=dx, dweight=dw)
    check_backward(dx, dw, x, w, t, torch.full((T,), float(got[2][1])))


@gpu
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 9, 32, 33, 100, 128])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("V", [37, 70000])
def test_few_tokens(g, T, shift, V):
    """Rows read where they lie (or packed, when they are not aligned), joined in one launch or two."""
    x, w, t = make(T, 520, V, T + shift, 0.3 if T > 2 else 0.0, int32=shift == 1)
    if T > 3:
        t[2] = V      # outside the vocabulary: NaN, which the mean shows too
    got = forward(g, on_gpu(x, 0 if shift else 8, shift), w.cuda(), t.cuda())
    loss, lse, mean = got
    if T > 3:
        assert loss[2].isnan() and torch.isfinite(lse[2]) and mean[0].isnan()
        keep = torch.arange(T) != 2
        n = int((t != IGNORE).sum())
        assert abs(float(mean[1]) - 1.0 / n) <= 2.0 ** -24
        want = ref.linear_cross_entropy(x[keep], w, t[keep].long(), IGNORE)
        tol = math.sqrt(520) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T).amax(1) + \
            2.0 ** -20 * 20
        assert torch.all((loss.cpu().double()[keep] - want[0]).abs() <= 2 * tol[keep])
        assert torch.all((lse.cpu().double()[keep] - want[1]).abs() <= tol[keep])
    else:
        check_forward(got, x, w, t)


@gpu
def test_strides_grad_of_each_token_and_one_gradient_only(g):
    T, H, V = 333, 264, 3001
    x, w, t = make(T, H, V, 9, 0.2)
    xd, wd, td = on_gpu(x, 5, 1), on_gpu(w, 16), t.cuda()
    got = forward(g, xd, wd, td)
    check_forward(got, x, w, t)
    grad = torch.randn(T, generator=torch.Generator().manual_seed(1))
    grad[::7] = 0.0
    dx, dw = on_gpu(torch.zeros(T, H).bfloat16(), 8), on_gpu(torch.zeros(V, H).bfloat16(), 24)
    g.linear_cross_entropy_backward(xd, wd, td, got[1], grad.cuda(), dx=dx, dweight=dw)
    check_backward(dx, dw, x, w, t, grad)
    dx1, dw1 = torch.empty_like(x, device="cuda"), torch.empty_like(w, device="cuda")
    g.linear_cross_entropy_backward(xd, wd, td, got[1], grad.cuda(), dx=dx1)
    g.linear_cross_entropy_backward(xd, wd, td, got[1], grad.cuda(), dweight=dw1)
    torch.testing.assert_close(dx1, dx, rtol=2.0 ** -7, atol=1e-6)
    torch.testing.assert_close(dw1, dw, rtol=2.0 ** -7, atol=1e-6)


@gpu
@pytest.mark.parametrize("T", [5, 300])
def test_uncounted_rows_are_not_read(g, T):
    H, V = 128, 900
    x, w, t = make(T, H, V, 4, 0.5)
    t[0], t[-1] = IGNORE, IGNORE
    clean = forward(g, x.cuda(), w.cuda(), t.cuda())
    dx, dw = torch.empty_like(x, device="cuda"), torch.empty_like(w, device="cuda")
    g.linear_cross_entropy_backward(x.cuda(), w.cuda(), t.cuda(), clean[1], clean[2][1:], dx, dw)
    dirty = x.clone()
    dirty[t == IGNORE] = float("nan")
    dirty[0] = float("inf")
    got = forward(g, dirty.cuda(), w.cuda(), t.cuda())
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    g.linear_cross_entropy_backward(dirty.cuda(), w.cuda(), t.cuda(), got[1], got[2][1:], dx2, dw2)
    for a, b in zip((*clean, dx, dw), (*got, dx2, dw2)):
        assert torch.equal(a, b)
    assert torch.all(dx[(t == IGNORE).cuda()] == 0)


@gpu
@pytest.mark.parametrize("T", [1, 8, 100, 300])
def test_infinite_logits(g, T):
    """Words of logit -inf, more than a tile of them, count as nothing; +inf and NaN make NaN."""
    H, V, shut, inf = 256, 5000, 1000, float("inf")
    gen = torch.Generator().manual_seed(T)
    x = (torch.rand(T, H, generator=gen) + 0.1).bfloat16()
    w = (torch.randn(V, H, generator=gen) / 16).bfloat16()
    t = torch.randint(shut, V, (T,), generator=gen)
    w[:shut] = -inf
    got = forward(g, x.cuda(), w.cuda(), t.cuda())
    check_forward(got, x, w[shut:], t - shut)
    dw = torch.full_like(w, 3.0, device="cuda")
    g.linear_cross_entropy_backward(x.cuda(), w.cuda(), t.cuda(), got[1], got[2][1:], dweight=dw)
    dx = torch.empty_like(x, device="cuda")
    open_ = w[shut:].cuda()
    g.linear_cross_entropy_backward(x.cuda(), open_, (t - shut).cuda(), got[1], got[2][1:], dx=dx)
    assert not dw[:shut].any()
    check_backward(dx, dw[shut:], x, w[shut:], t - shut, torch.full((T,), float(got[2][1])))

    t[0] = 3
    loss, lse, mean = forward(g, x.cuda(), w.cuda(), t.cuda())
    assert loss[0] == inf and mean[0] == inf and torch.equal(lse, got[1]) and torch.equal(loss[1:], got[0][1:])
    for value in (inf, float("nan")):
        w[shut + 7] = value
        loss, lse, _ = forward(g, x.cuda(), w.cuda(), t.cuda())
        assert lse.isnan().all() and loss.isnan().all()


@gpu
def test_no_counted_token_and_no_token(g):
    x, w, t = make(130, 64, 500, 2)
    t[:] = IGNORE
    loss, lse, mean = forward(g, x.cuda(), w.cuda(), t.cuda())
    assert not loss.any() and not lse.any() and not mean.any()
    dx, dw = torch.ones_like(x, device="cuda"), torch.ones_like(w, device="cuda")
    g.linear_cross_entropy_backward(x.cuda(), w.cuda(), t.cuda(), lse, mean[1:], dx, dw)
    assert not dx.any() and not dw.any()
    loss, lse, mean = forward(g, x[:0].cuda(), w.cuda(), t[:0].cuda())
    assert not mean.any()
    dw.fill_(1.0)
    g.linear_cross_entropy_backward(x[:0].cuda(), w.cuda(), t[:0].cuda(), lse, mean[1:], dx[:0], dw)
    assert not dw.any()


@gpu
def test_target_outside_the_vocabulary(g):
    x, w, t = make(40, 64, 300, 6)
    t[3], t[30] = 300, -7
    loss, lse, mean = forward(g, x.cuda(), w.cuda(), t.cuda())
    wrong = torch.zeros(40, dtype=torch.bool)
    wrong[3] = wrong[30] = True
    assert torch.equal(loss.isnan().cpu(), wrong) and mean[0].isnan()
    assert torch.isfinite(lse).all()
    dx, dw = torch.empty_like(x, device="cuda"), torch.empty_like(w, device="cuda")
    g.linear_cross_entropy_backward(x.cuda(), w.cuda(), t.cuda(), lse, mean[1:], dx, dw)
    assert not dx[wrong.cuda()].any() and torch.isfinite(dw).all() and dw.any()


@gpu
def test_large_logits_and_a_row_of_nan(g):
    """Logits of thousands: the running maximum keeps the sum finite; a NaN stays in its row."""
    x, w, t = make(150, 64, 700, 8)
    x = (x.float() * 500).bfloat16()
    x[7, 3] = float("nan")
    loss, lse, _ = forward(g, x.cuda(), w.cuda(), t.cuda())
    keep = torch.arange(150) != 7
    assert loss[7].isnan() and lse[7].isnan()
    assert torch.isfinite(loss.cpu()[keep]).all()
    want = ref.linear_cross_entropy(x[keep], w, t[keep], IGNORE)
    assert torch.all((lse.cpu()[keep].double() - want[1]).abs() <= 2.0 ** -18 * want[1].abs() + 1e-4)


@gpu
def test_same_bits_on_another_stream_in_a_graph_and_after_other_sizes(g):
    T, H, V = 700, 520, 9001
    x, w, t = make(T, H, V, 3, 0.1)
    x, w, t = x.cuda(), w.cuda(), t.cuda()
    loss, lse, mean = (torch.empty(n, device="cuda") for n in (T, T, 2))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    need = max(g.linear_cross_entropy_workspace(T, H, V, b) for b in (False, True))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def both(workspace=None, stream=None):
        g.linear_cross_entropy(x, w, t, loss, lse, mean=mean, workspace=workspace, stream=stream)
        g.linear_cross_entropy_backward(x, w, t, lse, mean[1:], dx, dw, workspace=workspace,
                                        stream=stream)

    def snapshot():
        torch.cuda.synchronize()
        got = [v.clone() for v in (loss, lse, mean, dx, dw)]
        for v in (loss, lse, mean, dx, dw):
            v.fill_(float("nan"))
        ws.fill_(0xFF)          # NaN patterns: nothing is left over from one call to the next
        torch.cuda.synchronize()
        return got

    runs = []
    both()
    runs.append(snapshot())
    both(ws, torch.cuda.Stream())
    runs.append(snapshot())
    both(None, torch.cuda.Stream())
    runs.append(snapshot())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(ws)
    graph.replay()
    runs.append(snapshot())
    forward(g, x[:3], w[:50], t[:3].clamp(max=49))
    graph.replay()
    runs.append(snapshot())
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


@gpu
def test_weight_past_32_bits(g):
    """A weight of more than 2^32 elements: the last rows of the vocabulary count and get theirs."""
    T, H, V = 5, 32776, 131100
    gen = torch.Generator("cuda").manual_seed(12)
    w = torch.randn(V, H, device="cuda", dtype=torch.bfloat16, generator=gen)
    w *= 1.5 / math.sqrt(H)
    t = torch.tensor([V - 1, 0, V - 300, IGNORE, V - 1], device="cuda")
    x = (torch.randn(T, H, device="cuda", generator=gen) + 3.0 * w[t.clamp(min=0)].float()).bfloat16()
    loss, lse, mean = forward(g, x, w, t)
    z = torch.cat([x.double() @ w[a:a + 8192].double().T for a in range(0, V, 8192)], 1)
    counted = t != IGNORE
    want = torch.logsumexp(z, 1)
    at = t.clamp(min=0)
    rows = torch.arange(T, device="cuda")
    assert torch.all((lse - want)[counted].abs() <= 1e-4)
    assert torch.all((loss - (want - z[rows, at]))[counted].abs() <= 2e-4)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    g.linear_cross_entropy_backward(x, w, t, lse, mean[1:], dx, dw)
    p = torch.softmax(z, 1)
    p[rows, at] -= 1.0
    p = torch.where(counted[:, None], p / 4, 0.0)
    last = V - 400
    tail = p[:, last:].T @ x.double()
    assert float((dw[last:].double() - tail).norm() / tail.norm()) < 4e-3
    head = p[:, :400].T @ x.double()
    assert float((dw[:400].double() - head).norm() / head.norm()) < 4e-3
    want_dx = sum(p[:, a:a + 8192] @ w[a:a + 8192].double() for a in range(0, V, 8192))
    assert float((dx.double() - want_dx).norm() / want_dx.norm()) < 4e-3
    del w, dw, z, p
    torch.cuda.empty_cache()


@gpu
def test_refusals(g):
    x, w, t = (v.cuda() for v in make(16, 64, 100, 1))
    loss, lse, mean = (torch.full((n,), 7.0, device="cuda") for n in (16, 16, 2))
    dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    for call in (
        lambda: g.linear_cross_entropy(x, w[:, :56], t, loss, lse),
        lambda: g.linear_cross_entropy(x.float(), w, t, loss, lse),
        lambda: g.linear_cross_entropy(x.half(), w.half(), t, loss, lse),
        lambda: g.linear_cross_entropy(x, w, t.float(), loss, lse),
        lambda: g.linear_cross_entropy(x, w, t[:5], loss, lse),
        lambda: g.linear_cross_entropy(x, w, t.cpu(), loss, lse),
        lambda: g.linear_cross_entropy(x, w, t, loss[:5], lse),
        lambda: g.linear_cross_entropy(x, w, t, loss, lse, mean=mean[:1]),
        lambda: g.linear_cross_entropy(x, w, t, loss, lse, workspace=loss),
        lambda: g.linear_cross_entropy_backward(x, w, t, lse, loss[:3], dx, dw),
        lambda: g.linear_cross_entropy_backward(x, w, t, lse, loss, dx[:, :8], dw),
    ):
        with pytest.raises(ValueError):
            call()
    bad, align = gemm_ws.ERR_INVALID_ARG, gemm_ws.ERR_ALIGNMENT
    ws = torch.empty(1024, dtype=torch.uint8, device="cuda")
    big = torch.empty(g.linear_cross_entropy_workspace(16, 64, 100, True) + 1, dtype=torch.uint8,
                      device="cuda")
    off = on_gpu(w.cpu(), 0, 1)
    for status, call in (
        (bad, lambda: g.linear_cross_entropy(x, w, t, loss, lse, workspace=ws)),
        (bad, lambda: g.linear_cross_entropy(x, w, t, loss, loss)),
        (bad, lambda: g.linear_cross_entropy_backward(x, w, t, lse, loss, x, dw)),
        (bad, lambda: g.linear_cross_entropy_backward(x, w, t, lse, loss, dx, w)),
        (align, lambda: g.linear_cross_entropy(x[:, :60], w[:, :60], t, loss, lse)),
        (align, lambda: g.linear_cross_entropy(x, off, t, loss, lse)),
        (align, lambda: g.linear_cross_entropy(x, on_gpu(w.cpu(), 4), t, loss, lse)),
        (align, lambda: g.linear_cross_entropy_backward(x, w, t, lse, loss, dx, off)),
        (align, lambda: g.linear_cross_entropy_backward(x, w, t, lse, loss, dx, dw,
                                                        workspace=big[1:])),
    ):
        with pytest.raises(gemm_ws.GemmWSError) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()
    for v in (loss, lse, dx, dw):
        assert torch.all(v == 7.0)
