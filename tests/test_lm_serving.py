"""The operators around a block run together, as a decoding step and as a training step use them."""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import gemm_ws
from tests import lm_block_reference as ref
from tests.test_lm_block import block_inputs
from tests.test_lm_int8 import close as close_product
from tests.test_lm_logits import close as close_logits, words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    handle.close()


@pytest.mark.parametrize("T", [1, 5, 40])
def test_decoding_step(g, T):
    """Two projections in 8-bit integers with the norms around them, then a head and its logits' adjustments, in one graph."""
    H, F, V = 512, 1408, 5003
    gen = torch.Generator().manual_seed(T)
    v, _ = block_inputs(T, H, torch.bfloat16, "cols", True, T)

    def weights(n, k):
        w = torch.randn(n, k, generator=gen) / k ** 0.5
        q, s = ref.quantize_rows(w)
        return q.cuda(), s.cuda()

    up, down, head = weights(F, H), weights(H, F), weights(V, H)
    t = torch.randint(0, V, (T, 30), generator=gen).cuda()
    n = torch.full((T,), 30, dtype=torch.int32, device="cuda")
    rep, freq = torch.full((T,), 1.2, device="cuda"), torch.full((T,), 0.1, device="cuda")
    allowed = words(T, V, gen, 0.5).cuda()
    b16 = dict(dtype=torch.bfloat16, device="cuda")
    a8, f8 = (torch.empty(T, k, dtype=torch.int8, device="cuda") for k in (H, F))
    sa, sf = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    h, h2, mid, out = torch.empty(T, H, **b16), torch.empty(T, H, **b16), torch.empty(T, F, **b16), torch.empty(T, H, **b16)
    z, last = torch.empty(T, V, device="cuda"), torch.empty(T, V, device="cuda")
    keep = {}

    def step(keep=None):
        g.block_norm(v["x"], v["residual"], v["weight"], a8, post_weight=v["post"], gate=v["gate"], h=h, scales=sa)
        if keep is not None:
            keep["a8"], keep["sa"] = a8.clone(), sa.clone()
        g.int8_matmul(a8, up[0], sa, up[1], mid)
        g.quantize_rows(mid, f8, sf)
        g.int8_matmul(f8, down[0], sf, down[1], out)
        g.block_norm(out, h, v["weight"], a8, post_weight=v["post"], h=h2, scales=sa)
        g.int8_matmul(a8, head[0], sa, head[1], z)
        g.adjust_logits(z, last, tokens=t, lengths=n, repetition=rep, frequency=freq, allowed=allowed)

    step(keep)
    cpu = lambda *ts: [x.cpu() for x in ts]  # noqa: E731
    _, d, size = ref.int8_matmul(*cpu(keep["a8"], up[0], keep["sa"], up[1]))
    close_product(mid, d, torch.bfloat16, size)
    q, s = ref.quantize_rows(mid.cpu())
    assert torch.equal(f8.cpu(), q) and torch.equal(sf.cpu(), s)
    _, d, size = ref.int8_matmul(*cpu(f8, down[0], sf, down[1]))
    close_product(out, d, torch.bfloat16, size)
    wh, wy, _, w2, size = ref.block_norm(*cpu(out, h, v["weight"]), post=v["post"].cpu())
    err = 2.0 ** -16 * (size * w2[:, None] * v["weight"].cpu().double().abs() +
                        wy.abs() * (1 + (size.norm(dim=1) / wh.norm(dim=1))[:, None]))
    step_size = sa.cpu().double()[:, None]
    assert bool(((a8.cpu().double() * step_size - wy).abs() <= step_size / 2 * (1 + 2.0 ** -16) + err).all())
    _, d, size = ref.int8_matmul(*cpu(a8, head[0], sa, head[1]))
    close_product(z, d, torch.float32, size)
    want, size = ref.adjust_logits(z.cpu(), t.cpu(), n.cpu(), None, rep.cpu(), freq.cpu(), None, allowed=allowed.cpu())
    close_logits(last, want, torch.float32, size)
    first = last.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    last.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(last, first) and g.query_status() == gemm_ws.OK


def test_training_step(g):
    """Norms around a block, the head's cross entropy and its gradients, and back: against gradients in 64 bits. In 16 bits
    lie y, the cross entropy's gradient before its products, dy and the results: each is off by at most 2^-8 of itself, so that
    the gradients are within 2^-6 of theirs in the norm."""
    T, H, V = 200, 256, 700
    v, gen = block_inputs(T, H, torch.bfloat16, "cols", True, 3)
    head = (torch.randn(V, H, generator=gen) / 16).bfloat16().cuda()
    target = torch.randint(0, V, (T,), generator=gen).cuda()
    new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f32 = lambda n: torch.empty(n, device="cuda")  # noqa: E731
    y, h, dy, dx, dres, dhead = new(T, H), new(T, H), new(T, H), new(T, H), new(T, H), new(V, H)
    r1, r2, loss, lse, mean = f32(T), f32(T), f32(T), f32(T), f32(2)
    grads = {"dweight": new(H), "dpost_weight": new(H), "dgate": new(H)}
    kw = dict(post_weight=v["post"], gate=v["gate"], alpha=0.9)
    g.block_norm(v["x"], v["residual"], v["weight"], y, h=h, post_rstd=r1, rstd=r2, **kw)
    g.linear_cross_entropy(y, head, target, loss, lse, mean=mean)
    g.linear_cross_entropy_backward(y, head, target, lse, mean[1:], dx=dy, dweight=dhead)
    g.block_norm_backward(dy, v["x"], h, v["weight"], r2, dx, dres, post_rstd=r1, **kw, **grads)
    leaves = {k: v[k].cpu().double().requires_grad_() for k in ("x", "residual", "weight", "post", "gate")}
    _, wy, _, _, _ = ref.block_norm(alpha=0.9, **leaves)
    torch.nn.functional.cross_entropy(wy @ head.cpu().double().T, target.cpu()).backward()
    got = {"x": dx, "residual": dres, "weight": grads["dweight"], "post": grads["dpost_weight"], "gate": grads["dgate"]}
    for k, t in got.items():
        want = leaves[k].grad
        assert float((t.cpu().double() - want).norm()) <= 2.0 ** -6 * float(want.norm()), k
