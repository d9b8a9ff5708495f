"""Block norms of unaligned rows whose shared memory, with what the kernels declare themselves, comes close to the 48 KB that a kernel
has unasked: 12288 columns forward, 4096 for the gradients."""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import gemm_ws
from tests import lm_block_reference as ref
from tests.test_lm_block import block_inputs, close, on_cpu, output, rows, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture
def g():
    """A handle whose kernels have not been given more by another call."""
    handle = gemm_ws.GemmWS(0)
    yield handle
    assert handle.query_status() == gemm_ws.OK
    handle.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("H", [10241, 12153, 12161, 12200, 12287, 12289])
def test_forward(g, dtype, H):
    T = 5
    v, _ = block_inputs(T, H, dtype, "cols", True, H, 1, 1)
    c = on_cpu(v)
    y, ybuf = output(T, H, dtype, 1, 1)
    h, hbuf = output(T, H, dtype, 1, 1)
    g.block_norm(v["x"], v["residual"], v["weight"], y, post_weight=v["post"], gate=v["gate"], alpha=0.5, h=h)
    wh, wy, _, w2, size = ref.block_norm(alpha=0.5, **c)
    close(h, wh, dtype, size, what="h")
    spread = (size.norm(dim=1) / wh.norm(dim=1))[:, None]
    close(y, wy, dtype, size * w2[:, None] * c["weight"].double().abs() + wy.abs() * (1 + spread), what="y")
    assert untouched(ybuf, y, H) and untouched(hbuf, h, H)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T", [3, 1300])
@pytest.mark.parametrize("H", [3409, 4007, 4009, 4050, 4095, 4097])
def test_gradients(g, dtype, T, H):
    v, gen = block_inputs(T, H, dtype, "cols", True, H, 1, 1)
    c = on_cpu(v)
    h = rows(T, H, dtype, gen, 1, 1, 3.0)
    r1, r2 = 0.5 + torch.rand(T, generator=gen), 0.5 + torch.rand(T, generator=gen)
    dy, dh = rows(T, H, dtype, gen, 1, 1), rows(T, H, dtype, gen, 1, 1)
    outs = {"dx": output(T, H, dtype, 1, 1), "dresidual": output(T, H, dtype, 1, 1)}
    kw = {k: t for k, (t, _) in outs.items()}
    kw.update({k: torch.full((H,), 7.0, dtype=dtype, device="cuda") for k in ("dweight", "dpost_weight", "dgate")})
    g.block_norm_backward(dy, v["x"], h, v["weight"], r2.cuda(), post_weight=v["post"], post_rstd=r1.cuda(), gate=v["gate"], alpha=0.5,
                          dh=dh, **kw)
    want, sizes = ref.block_norm_backward(dy.cpu(), c["x"], h.cpu(), c["weight"], r2, c["post"], r1, c["gate"], 0.5, dh.cpu())
    for k in want:
        close(kw[k], want[k], dtype, sizes[k], what=k)
    for t, buf in outs.values():
        assert untouched(buf, t, H)
