"""Ways to call the block norms, the 8-bit product and the logits' adjustments that are allowed but out of the ordinary:
first calls inside a capture, two streams at once, inputs written by the kernel just before, outputs over inputs on the
paths for many rows, and plans of the product that cut only some tiles.

No tolerances: the results are those of the same calls made one by one, bit for bit, or exact whole numbers.
"""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import gemm_ws

gpu = pytest.mark.gpu
F32, I8, BF16 = torch.float32, torch.int8, torch.bfloat16


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    handle.close()


def values(gen, *shape, dtype=BF16):
    return torch.randn(*shape, generator=gen).to(dtype).cuda()


def integers(gen, *shape):
    return torch.randint(-128, 128, shape, generator=gen, dtype=I8).cuda()


def steps(g, T, H, V, seed):
    """Every operator once, with its own buffers: a call that runs them, and the outputs."""
    gen = torch.Generator().manual_seed(seed)
    x, res, dy, dh = (values(gen, T, H) for _ in range(4))
    w, post, gate = (values(gen, H) for _ in range(3))
    w8, sw = integers(gen, V, (H + 15) // 16 * 16)[:, :H], (1e-3 * torch.rand(V, generator=gen)).cuda()
    tokens = torch.randint(0, V, (T, 40), generator=gen).cuda()
    rep = torch.full((T,), 1.25, device="cuda")
    y, h, dx, dres = (torch.zeros_like(x) for _ in range(4))
    r1, r2, sx = (torch.zeros(T, device="cuda") for _ in range(3))
    dw, dpost, dgate = (torch.zeros_like(w) for _ in range(3))
    y8 = torch.zeros(T, H, dtype=I8, device="cuda")
    logits = torch.zeros(T, V, device="cuda")
    ws = torch.zeros(max(g.int8_matmul_workspace(T, V, H), 1), dtype=torch.uint8, device="cuda")

    def run(handle=g, stream=None):
        handle.block_norm(x, res, w, y, post_weight=post, gate=gate, alpha=0.9, h=h, post_rstd=r1, rstd=r2, stream=stream)
        handle.block_norm_backward(dy, x, h, w, r2, dx, dresidual=dres, post_weight=post, post_rstd=r1, gate=gate,
                                   alpha=0.9, dh=dh, dweight=dw, dpost_weight=dpost, dgate=dgate, stream=stream)
        handle.quantize_rows(y, y8, sx, stream=stream)
        handle.int8_matmul(y8, w8, sx, sw, logits, workspace=ws, stream=stream)
        handle.adjust_logits(logits, logits, tokens=tokens, repetition=rep, stream=stream)

    return run, (y, h, dx, dres, dw, dpost, dgate, y8, sx, logits)


def wanted(run, outputs):
    run()
    torch.cuda.synchronize()
    kept = [t.clone() for t in outputs]
    for t in outputs:
        t.zero_()
    return kept


def same(outputs, kept):
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(outputs, kept)):
        assert torch.equal(a, b), f"output {i}"


@gpu
@pytest.mark.parametrize("T,H,V", [(2, 512, 1000), (400, 1032, 1500)])
def test_first_calls_of_a_handle_inside_a_capture(g, T, H, V):
    run, outputs = steps(g, T, H, V, 1)
    kept = wanted(run, outputs)
    handle = gemm_ws.GemmWS(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(handle)
    for _ in range(2):
        for t in outputs:
            t.zero_()
        graph.replay()
        same(outputs, kept)
    assert handle.query_status() == gemm_ws.OK
    del graph
    handle.close()


@gpu
def test_two_handles_on_two_streams(g):
    other = gemm_ws.GemmWS(0)
    runs = [steps(g, 300, 1024, 2000, 2), steps(g, 96, 4096, 3000, 3)]
    kept = [wanted(*r) for r in runs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for (run, _), stream, handle in zip(runs, streams, (g, other)):
            run(handle, stream)
    for (_, outputs), k in zip(runs, kept):
        same(outputs, k)
    assert g.query_status() == gemm_ws.OK and other.query_status() == gemm_ws.OK
    other.close()


@gpu
@pytest.mark.parametrize("M,N,K", [(12, 2048, 1024), (200, 1000, 2000), (700, 9000, 512)])
def test_products_of_what_the_kernel_before_wrote(g, M, N, K):
    """Weights and tokens quantised on the stream just before, into the same buffers every time, with one workspace."""
    gen = torch.Generator().manual_seed(4)
    K16 = (K + 15) // 16 * 16
    a8, sa = torch.empty(M, K, dtype=I8, device="cuda"), torch.empty(M, device="cuda")
    w8, sw = torch.empty(N, K16, dtype=I8, device="cuda")[:, :K], torch.empty(N, device="cuda")
    ws = torch.empty(max(g.int8_matmul_workspace(M, N, K), 1), dtype=torch.uint8, device="cuda")
    inputs = [(values(gen, M, K), values(gen, N, K)) for _ in range(3)]
    want = []
    for a, w in inputs:
        g.quantize_rows(a, a8, sa)
        g.quantize_rows(w, w8, sw)
        torch.cuda.synchronize()
        d = torch.empty(M, N, device="cuda")
        g.int8_matmul(a8, w8, sa, sw, d, workspace=ws)
        torch.cuda.synchronize()
        want.append(d)
        sums = a8.double() @ w8.double().t()
        exact = sums * sa.double()[:, None] * sw.double()
        # the sum to 32 bits, and two products: 2^-24 each
        assert bool(((d.double() - exact).abs() <= 2.0 ** -22 * exact.abs() + 1e-30).all())
    got = [torch.empty(M, N, device="cuda") for _ in range(30)]
    for i, d in enumerate(got):
        a, w = inputs[i % 3]
        g.quantize_rows(a, a8, sa)
        g.quantize_rows(w, w8, sw)   # the kernel just before the product's two
        g.int8_matmul(a8, w8, sa, sw, d, workspace=ws)
    torch.cuda.synchronize()
    for i, d in enumerate(got):
        assert torch.equal(d, want[i % 3]), i
    assert g.query_status() == gemm_ws.OK


@gpu
@pytest.mark.parametrize("M,N,K", [(2600, 5200, 1300), (1500, 4096, 520), (170, 20000, 2100), (9, 40000, 777)])
def test_plans_that_cut_some_tiles(g, M, N, K):
    gen = torch.Generator().manual_seed(5)
    K16 = (K + 15) // 16 * 16
    a, w = integers(gen, M, K), integers(gen, N, K16)[:, :K]
    one_m, one_n = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    d = torch.empty(M, N, device="cuda")
    g.int8_matmul(a, w, one_m, one_n, d)
    want = a.double() @ w.double().t()
    assert torch.equal(d, want.float())   # one rounding of a whole number


def alias_case(T, H, dtype, gate, seed=6):
    gen = torch.Generator().manual_seed(seed)
    x, res, dy, dh = (values(gen, T, H, dtype=dtype) for _ in range(4))
    w, post = values(gen, H, dtype=dtype), values(gen, H, dtype=dtype)
    gates = values(gen, H, dtype=dtype) if gate == "cols" else values(gen, T, H, dtype=dtype)
    return x, res, dy, dh, w, post, gates


@gpu
@pytest.mark.parametrize("T,H,dtype", [(1300, 8448, BF16), (1300, 1024, F32), (1300, 1001, F32)])
@pytest.mark.parametrize("gate", ["cols", "rows"])
def test_forward_over_its_inputs(g, T, H, dtype, gate):
    x, res, _, _, w, post, gates = alias_case(T, H, dtype, gate)
    y, h = torch.empty_like(x), torch.empty_like(x)
    g.block_norm(x, res, w, y, post_weight=post, gate=gates, h=h)
    x1, res1 = x.clone(), res.clone()
    g.block_norm(x1, res1, w, x1, post_weight=post, gate=gates, h=res1)     # y over x, h over the residual
    x2 = x.clone()
    y2 = torch.empty_like(x)
    g.block_norm(x2, res, w, y2, post_weight=post, gate=gates, h=x2)        # h over x
    x3 = x.clone()
    h3 = torch.empty_like(x)
    g.block_norm(x3, x3, w, y2.zero_(), post_weight=post, gate=gates, h=x3)   # one matrix as x, residual and h
    g.block_norm(x, x, w, h3, post_weight=post, gate=gates)
    assert torch.equal(x1, y) and torch.equal(res1, h) and torch.equal(x2, h) and torch.equal(y2, h3)
    assert g.query_status() == gemm_ws.OK


@gpu
@pytest.mark.parametrize("T,H,dtype", [(1300, 2048, BF16), (1300, 1024, F32), (1300, 1001, F32), (1300, 512, BF16)])
@pytest.mark.parametrize("gate", ["cols", "rows"])
def test_gradients_over_their_inputs(g, T, H, dtype, gate):
    x, res, dy, dh, w, post, gates = alias_case(T, H, dtype, gate)
    y, h, dx, dres = (torch.empty_like(x) for _ in range(4))
    r1, r2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    g.block_norm(x, res, w, y, post_weight=post, gate=gates, h=h, post_rstd=r1, rstd=r2)

    def grads(dy_, dh_, dx_, dres_):
        sums = [torch.empty_like(w), torch.empty_like(post), torch.empty_like(gates)]
        g.block_norm_backward(dy_, x, h, w, r2, dx_, dresidual=dres_, post_weight=post, post_rstd=r1, gate=gates, dh=dh_,
                              dweight=sums[0], dpost_weight=sums[1], dgate=sums[2])
        return sums

    want = grads(dy, dh, dx, dres)
    for swap in (False, True):
        dy1, dh1 = dy.clone(), dh.clone()
        to = (dh1, dy1) if swap else (dy1, dh1)
        got = grads(dy1, dh1, *to)
        assert torch.equal(to[0], dx) and torch.equal(to[1], dres)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    dy1 = dy.clone()
    got = grads(dy1, dy1, dy1, dres.zero_())   # one matrix as dy, dh and dx
    dx2, dres2 = torch.empty_like(dx), torch.empty_like(dx)
    want = grads(dy, dy, dx2, dres2)
    assert torch.equal(dy1, dx2) and torch.equal(dres, dres2)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert g.query_status() == gemm_ws.OK


@gpu
@pytest.mark.parametrize("rows,vocab", [(3, 5000), (3, 5001), (700, 20000)])
def test_one_matrix_of_lists_for_all_rows_and_odd_lengths(g, rows, vocab):
    """Lengths and prompts below zero, above the history and above the length count as what is there."""
    gen = torch.Generator().manual_seed(7)
    logits = values(gen, rows, vocab, dtype=F32)
    tokens = torch.randint(-5, vocab + 5, (rows, 300), generator=gen).cuda()
    tokens[:, 0] = 1 << 40
    tokens[:, 1] = -(1 << 40)
    freq = torch.rand(rows, generator=gen).cuda()
    lengths = torch.tensor([-7, 1 << 30, 100] * rows, dtype=torch.int32)[:rows].cuda()
    prompts = torch.tensor([5, -3, 1 << 30] * rows, dtype=torch.int32)[:rows].cuda()
    out, want = torch.empty_like(logits), torch.empty_like(logits)
    g.adjust_logits(logits, out, tokens=tokens, lengths=lengths, prompt_lengths=prompts, frequency=freq, presence=freq)
    plain_l, plain_p = lengths.clamp(0, 300), prompts.clamp(0, 300)
    g.adjust_logits(logits, want, tokens=tokens, lengths=plain_l, prompt_lengths=plain_p, frequency=freq, presence=freq)
    assert torch.equal(out, want)
    assert torch.equal(out[0], logits[0]) and torch.equal(out[2], logits[2])   # nothing counts, and all is prompt
    assert not torch.equal(out[1], logits[1])
    # int32 tokens, and the same token in every place
    g.adjust_logits(logits, out, tokens=torch.full((rows, 300), 3, dtype=torch.int32, device="cuda"), frequency=freq)
    plain = logits.clone()
    plain[:, 3] = (logits[:, 3].double() - 300.0 * freq.double()).float()
    off = (out - plain).abs()
    off[:, 3] -= 2.0 ** -22 * (logits[:, 3].abs() + 300.0 * freq)   # two roundings of at most 2^-24 each
    assert float(off.max()) <= 0.0


@gpu
@pytest.mark.parametrize("dtype,out_type", [(F32, F32), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,vocab,history,biases", [(400, 20000, 4096, 1024), (2, 6000, 4096, 1024), (700, 70001, 4096, 1024),
                                                       (700, 30000, 4097, 1024), (700, 30000, 0, 1024), (900, 16400, 31, 1)])
def test_the_fullest_tables(g, dtype, out_type, rows, vocab, history, biases):
    """All tokens of the history and all with biases different."""
    gen = torch.Generator().manual_seed(8)
    logits = values(gen, rows, vocab, dtype=dtype)
    order = torch.randperm(vocab, generator=gen)
    order = order.repeat(1 + (history + biases) // vocab)[:history + biases].repeat(rows, 1)
    order = ((order + torch.arange(rows)[:, None]) % vocab).cuda()
    tokens, at = order[:, :history], order[:, history:]
    value = torch.randn(rows, biases, generator=gen).cuda()
    rep, freq = 0.5 + torch.rand(rows, generator=gen).cuda(), torch.rand(rows, generator=gen).cuda()
    out = torch.empty(rows, vocab, dtype=out_type, device="cuda")
    penalties = dict(tokens=tokens, repetition=rep, frequency=freq) if history else {}
    g.adjust_logits(logits, out, bias_tokens=at, bias_values=value, **penalties)
    z = logits.double()
    size = z.abs()
    if history:
        count = torch.zeros(rows, vocab, device="cuda").scatter_add_(1, tokens, torch.ones(rows, history, device="cuda"))
        r64 = rep.double()[:, None]
        z = torch.where(count > 0, torch.where(z > 0, z / r64, z * r64), z)
        z = z - freq.double()[:, None] * count
        size = size * torch.clamp(torch.maximum(r64, 1 / r64), min=1.0) + freq.double()[:, None] * count
    plus = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda").scatter_add_(1, at, value.double())
    most = torch.zeros(rows, vocab, dtype=torch.float64, device="cuda").scatter_add_(1, at, value.double().abs())
    z = z + plus
    # five roundings to 32 bits of at most 2^-24 of the magnitudes, and the output's own
    unit = {F32: 2.0 ** -24, BF16: 2.0 ** -8}[out_type]
    tol = unit * z.abs() + 2.0 ** -21 * (size + most) + 1e-30
    off = (out.double() - z).abs()
    assert bool((off <= tol).all()), f"worst {float((off / tol).max()):.3g} of the tolerance"
    inplace = logits.clone()
    if out_type is dtype:
        g.adjust_logits(inplace, inplace, bias_tokens=at, bias_values=value, **penalties)
        assert torch.equal(inplace, out)
    assert g.query_status() == gemm_ws.OK
