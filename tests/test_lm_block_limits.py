"""Offsets past 32 bits, extents close to their limits, and the lengths where one variant takes over from another."""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import gemm_ws
from tests import lm_block_reference as ref
from tests.lm_reference import UNIT
from tests.test_lm_block import block_inputs, close, on_cpu, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    handle.close()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H", [512, 515])
def test_rows_far_apart(g, H):
    """Rows 2^24 + 8 elements apart: the last ones begin past 2^32 elements."""
    T, pitch = 270, 2 ** 24 + 8
    v, gen = block_inputs(T, H, torch.bfloat16, "rows", True, 7)

    def far(t):
        buf = torch.empty((T - 1) * pitch + H, dtype=t.dtype, device="cuda")
        out = buf.as_strided((T, H), (pitch, 1))
        out.copy_(t)
        return out

    new = lambda: torch.empty(T, H, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y, h, dx, dg = new(), new(), new(), new()
    r1, r2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dy = rows(T, H, torch.bfloat16, gen)
    kw = dict(post_weight=v["post"])
    g.block_norm(v["x"], v["residual"], v["weight"], y, gate=v["gate"], h=h, post_rstd=r1, rstd=r2, **kw)
    g.block_norm_backward(dy, v["x"], h, v["weight"], r2, dx, gate=v["gate"], post_rstd=r1, dgate=dg, **kw)
    x, res, gate, y2, h2 = far(v["x"]), far(v["residual"]), far(v["gate"]), far(y), far(h)
    y2.zero_(), h2.zero_()
    g.block_norm(x, res, v["weight"], y2, gate=gate, h=h2, **kw)
    assert torch.equal(y2, y) and torch.equal(h2, h)
    del res, y2
    dx2, dg2, dy2 = far(dx), far(dg), far(dy)
    dx2.zero_(), dg2.zero_()
    g.block_norm_backward(dy2, x, h2, v["weight"], r2, dx2, gate=gate, post_rstd=r1, dgate=dg2, **kw)
    assert torch.equal(dx2, dx) and torch.equal(dg2, dg)
    q, s = torch.zeros(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    g.quantize_rows(x, q, s)
    want, ws = ref.quantize_rows(v["x"].cpu())
    assert torch.equal(q.cpu(), want) and torch.equal(s.cpu(), ws)
    del x, gate, h2, dx2, dg2, dy2
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [1, 7, 24, 200])
def test_weights_of_more_than_4_gb(g, M):
    N, K = 70000, 65552
    gen = torch.Generator("cuda").manual_seed(M)
    w = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=gen)
    a = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=gen)
    sa, sw = torch.rand(M, device="cuda", generator=gen), torch.rand(N, device="cuda", generator=gen)
    d = torch.empty(M, N, device="cuda")
    g.int8_matmul(a, w, sa, sw, d)
    for part in (slice(0, 300), slice(N // 2, N // 2 + 300), slice(N - 300, N)):
        want = (a.double() @ w[part].double().T) * sa.double()[:, None] * sw[part].double()
        assert bool(((d[:, part].double() - want).abs() <= 2.0 ** -22 * want.abs() + 2.0 ** -140).all())
    assert g.query_status() == gemm_ws.OK
    del w
    torch.cuda.empty_cache()


def test_logits_past_32_bits(g):
    rows_, vocab = 33000, 131072 + 8
    z = torch.zeros(rows_, vocab, dtype=torch.float16, device="cuda")
    z[-1].fill_(2.0)
    z[0].fill_(-2.0)
    tokens = torch.full((rows_, 3), vocab - 1, dtype=torch.int32, device="cuda")
    one = torch.ones(rows_, device="cuda")
    g.adjust_logits(z, z, tokens=tokens, repetition=2.0 * one, frequency=one)
    assert float(z[-1, -1]) == 1.0 - 3.0 and float(z[-1, -2]) == 2.0
    assert float(z[0, -1]) == -4.0 - 3.0 and float(z[0, 0]) == -2.0
    assert float(z[5, -1]) == -3.0 and not bool(z[5, :-1].any())
    del z
    torch.cuda.empty_cache()


def test_a_large_vocabulary(g):
    """2^31 - 4097 words, more than a block's lists of slices cover, in place."""
    vocab = 2 ** 31 - 1 - 4096
    z = torch.zeros(1, vocab, dtype=torch.float16, device="cuda")
    where = torch.tensor([[0, 8191, 8192, vocab // 2, vocab - 8192, vocab - 1, -1, vocab]], device="cuda")
    g.adjust_logits(z, z, tokens=where, presence=torch.ones(1, device="cuda"), bias_tokens=where,
                    bias_values=torch.full((1, 8), 0.5, device="cuda"))
    found = torch.nonzero(z[0])[:, 0].cpu()
    assert torch.equal(found, where[0, :6].cpu()) and bool((z[0, found.cuda()] == -0.5).all())
    too_large = torch.empty(1, vocab + 1, dtype=torch.float16, device="cuda")
    with pytest.raises(gemm_ws.GemmWSError):
        g.adjust_logits(too_large, too_large)
    del z, too_large
    torch.cuda.empty_cache()


# Rows and lengths on both sides of each choice: teams of a warp and of a block, one, two and four groups a
# thread, the rings, and the general path.
@pytest.mark.parametrize("dtype,T,H", [
    (torch.bfloat16, 607, 1016), (torch.bfloat16, 608, 1024), (torch.bfloat16, 151, 1024), (torch.bfloat16, 152, 1024),
    (torch.bfloat16, 303, 2048), (torch.bfloat16, 304, 2048), (torch.bfloat16, 1216, 2056), (torch.bfloat16, 700, 8192),
    (torch.bfloat16, 700, 8200), (torch.bfloat16, 620, 14336), (torch.bfloat16, 620, 16384), (torch.float32, 608, 1016),
    (torch.float32, 608, 1024), (torch.float32, 620, 4104), (torch.float32, 620, 8192), (torch.float32, 620, 8200),
    (torch.float16, 1216, 255), (torch.float16, 1216, 257), (torch.float16, 1217, 4099), (torch.float32, 160, 16381)])
@pytest.mark.parametrize("gate", ["cols", "rows"])
def test_where_variants_take_over(g, dtype, T, H, gate):
    v, gen = block_inputs(T, H, dtype, gate, True, T + H)
    c = on_cpu(v)
    y, h = torch.empty_like(v["x"]), torch.empty_like(v["x"])
    r1, r2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    kw = dict(post_weight=v["post"], gate=v["gate"], alpha=0.75)
    g.block_norm(v["x"], v["residual"], v["weight"], y, h=h, post_rstd=r1, rstd=r2, **kw)
    wh, wy, _, w2, size = ref.block_norm(alpha=0.75, **c)
    close(h, wh, dtype, size, what="h")
    spread = (size.norm(dim=1) / wh.norm(dim=1))[:, None]
    close(y, wy, dtype, size * w2[:, None] * c["weight"].double().abs() + wy.abs() * (1 + spread), what="y")
    dy, dh = rows(T, H, dtype, gen), rows(T, H, dtype, gen)
    outs = {"dx": torch.empty_like(y), "dresidual": torch.empty_like(y), "dweight": torch.empty_like(v["weight"]),
            "dpost_weight": torch.empty_like(v["weight"]), "dgate": torch.empty_like(v["gate"])}
    g.block_norm_backward(dy, v["x"], h, v["weight"], r2, post_rstd=r1, dh=dh, **kw, **outs)
    want, sizes = ref.block_norm_backward(dy.cpu(), c["x"], h.cpu(), c["weight"], r2.cpu(), c["post"], r1.cpu(), c["gate"],
                                          0.75, dh.cpu())
    for k in want:
        close(outs[k], want[k], dtype, sizes[k], what=k)
    assert g.query_status() == gemm_ws.OK


@pytest.mark.parametrize("rows_,vocab,history", [(304, 8192, 10), (305, 8193, 4096), (40, 70001, 4096), (40, 70001, 4097),
                                                 (2, 600000, 9000), (1, 4096, 40000), (64, 40000, 3)])
def test_slices_lists_and_rounds(g, rows_, vocab, history):
    """One and several slices a block, histories in lists and read in rounds; every word as 64 bits have it."""
    gen = torch.Generator("cuda").manual_seed(vocab)
    z = 3.0 * torch.randn(rows_, vocab, device="cuda", generator=gen)
    t = torch.randint(0, vocab, (rows_, history), device="cuda", generator=gen)
    t[:, ::3] = torch.randint(0, 40, (rows_, (history + 2) // 3), device="cuda", generator=gen)
    prompts = torch.full((rows_,), history // 3, dtype=torch.int32, device="cuda")
    f = 0.25 + torch.rand(rows_, device="cuda", generator=gen)
    out = torch.empty_like(z)
    g.adjust_logits(z, out, tokens=t, prompt_lengths=prompts, repetition=f, frequency=f, presence=f)
    new = (torch.arange(history, device="cuda") >= history // 3).double().expand(rows_, -1)
    count = torch.zeros(rows_, vocab, device="cuda", dtype=torch.float64).scatter_add_(1, t, new)
    seen = torch.zeros(rows_, vocab, device="cuda", dtype=torch.float64).scatter_add_(1, t, torch.ones_like(new)) > 0
    r = f.double()[:, None]
    w = z.double()
    w = torch.where(seen, torch.where(w > 0, w / r, w * r), w)
    size = w.abs() + r * count + r
    w = w - torch.where(count > 0, r * count + r, 0.0)
    assert bool(((out.double() - w).abs() <= UNIT[torch.float32] * w.abs() + 2.0 ** -21 * size).all())
