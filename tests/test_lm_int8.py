"""The product of 8-bit integers with scales, against whole numbers and 64 bits.

Tolerances, fixed before the first run: the sums are exact, so d is off by the roundings of the sum to 32 bits, of its
product with a token's scale and of the last product and sum (2^-24 each of the magnitudes: within 2^-22), and by its own.
"""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import build, gemm_ws
from tests import lm_block_reference as ref
from tests.lm_reference import TINY, UNIT

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
gpu = pytest.mark.gpu


def test_null_handle_is_refused_without_a_gpu():
    build.ensure_built()
    lib = gemm_ws.load_library()
    assert lib.gemm_ws_int8_matmul(None, None, 16, None, None, 16, None, None, None, 16, 0, 1, 16, 16, None, 0, None) == \
        gemm_ws.ERR_INVALID_ARG
    assert lib.gemm_ws_int8_matmul_workspace(None, 1, 16, 16) == -gemm_ws.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    handle.close()


def integers(rows, cols, gen, pitch=None, shift=0):
    """rows x cols on the GPU, all 256 values among them; what lies between rows is not zero."""
    pitch = cols if pitch is None else pitch
    buf = torch.randint(-128, 128, (rows * pitch + shift,), generator=gen, dtype=torch.int8).cuda()
    return buf[shift:].view(rows, pitch)[:, :cols]


def scales(n, gen):
    return torch.exp(torch.randn(n, generator=gen)).cuda() * 1e-3


def close(got, want, dtype, size):
    tol = UNIT[dtype] * want.abs() + 2.0 ** -22 * size + TINY[dtype]
    off = (got.cpu().double() - want).abs()
    assert bool((off <= tol).all()), f"worst {float((off / tol).max()):.3g} of the tolerance"


def check(g, M, N, K, dtype, bias=False, a_pitch=None, a_shift=0, d_pad=0, seed=0):
    gen = torch.Generator().manual_seed(seed + M + 3 * N + 5 * K)
    a = integers(M, K, gen, a_pitch, a_shift)
    w = integers(N, K, gen, (K + 15) // 16 * 16)
    sa, sw = scales(M, gen), scales(N, gen)
    b = (0.1 * torch.randn(N, generator=gen)).cuda() if bias else None
    buf = torch.full((M, N + d_pad), 7.0, dtype=dtype, device="cuda")
    d = buf[:, :N]
    g.int8_matmul(a, w, sa, sw, d, bias=b)
    _, want, size = ref.int8_matmul(a.cpu(), w.cpu(), sa.cpu(), sw.cpu(), None if b is None else b.cpu())
    close(d, want, dtype, size)
    assert bool((buf[:, N:] == 7).all())
    assert g.query_status() == gemm_ws.OK


TOKENS = [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 100, 128, 129, 200, 257, 500]


@gpu
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("N,K", [(1, 1), (7, 15), (128, 64), (130, 200), (513, 1000), (96, 4100)])
def test_sizes(g, M, N, K):
    check(g, M, N, K, DTYPES[(M + N) % 3], bias=N % 2 == 0)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,K", [(1, 5000, 512), (1, 300, 16000), (70, 2500, 8192), (1000, 1000, 1024), (700, 1536, 3000),
                                   (3, 20000, 128)])
def test_larger_sizes(g, dtype, M, N, K):
    check(g, M, N, K, dtype, bias=True)


@gpu
@pytest.mark.parametrize("M", [1, 6, 40, 300])
@pytest.mark.parametrize("a_pitch,a_shift,d_pad", [(321, 0, 0), (336, 1, 1), (400, 3, 3), (352, 16, 8), (320, 5, 0)])
def test_rows_that_lie_anywhere(g, M, a_pitch, a_shift, d_pad):
    check(g, M, 200, 320, torch.bfloat16, a_pitch=a_pitch, a_shift=a_shift, d_pad=d_pad)
    check(g, M, 130, 320, torch.float32, a_pitch=a_pitch, a_shift=a_shift, d_pad=d_pad)


@gpu
@pytest.mark.parametrize("M", [1, 4, 8, 20, 150, 400])
@pytest.mark.parametrize("K", [1024, 1040, 8200, 131071])
def test_sums_of_the_largest_values_are_exact(g, M, K):
    """All -128, all 127, and signs in turn: sums up to 2^31, far past what fp32 holds."""
    N = 200
    a = torch.full((M, K), -128, dtype=torch.int8)
    a[M // 2] = 127
    padded = torch.full((N, (K + 15) // 16 * 16), -128, dtype=torch.int8)
    w = padded[:, :K]
    w[1::3] = 127
    w[2::3, ::2] = 127
    w[0, K - 1] = 1   # odd sums
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    d = torch.empty(M, N, device="cuda")
    g.int8_matmul(a.cuda(), padded.cuda()[:, :K], one(M), one(N), d)
    sums, _, _ = ref.int8_matmul(a, w, torch.ones(M), torch.ones(N))
    assert float(sums.abs().max()) > 127 * 127 * K * 0.9
    assert torch.equal(d.cpu(), sums.float())


@gpu
def test_a_row_of_scale_nan_stays_its_own(g):
    M, N, K = 70, 300, 640
    gen = torch.Generator().manual_seed(4)
    a, w, sa, sw = integers(M, K, gen), integers(N, K, gen), scales(M, gen), scales(N, gen)
    d0, d1 = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    g.int8_matmul(a, w, sa, sw, d0)
    sa[7] = float("nan")
    sw[11] = float("inf")
    g.int8_matmul(a, w, sa, sw, d1)
    rows, cols = torch.arange(M) != 7, torch.arange(N) != 11
    assert torch.equal(d0.cpu()[rows][:, cols], d1.cpu()[rows][:, cols])
    assert bool(torch.isnan(d1[7]).all()) and bool(torch.isinf(d1[rows.cuda(), 11]).any())


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 700, 900), (60, 700, 2000), (600, 700, 900)])
def test_streams_graphs_and_used_workspaces(g, M, N, K):
    gen = torch.Generator().manual_seed(8)
    a, w, sa, sw = integers(M, K, gen), integers(N, K, gen, (K + 15) // 16 * 16), scales(M, gen), scales(N, gen)
    d = [torch.empty(M, N, device="cuda") for _ in range(4)]
    g.int8_matmul(a, w, sa, sw, d[0])
    need = g.int8_matmul_workspace(M, N, K)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g.int8_matmul(a, w, sa, sw, d[1], workspace=ws, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        g.int8_matmul(a, w, sa, sw, d[2], workspace=ws)
        g.int8_matmul(a, w, sa, sw, d[3])
    for _ in range(3):
        ws.fill_(255)
        graph.replay()
    torch.cuda.synchronize()
    for k in range(1, 4):
        assert torch.equal(d[0], d[k])
    assert g.query_status() == gemm_ws.OK


@gpu
def test_refusals(g):
    gen = torch.Generator().manual_seed(1)
    M, N, K = 20, 48, 64
    a, w, sa, sw = integers(M, K, gen), integers(N, K, gen), scales(M, gen), scales(N, gen)
    d = torch.empty(M, N, device="cuda")

    def refused(error, *args, **k):
        with pytest.raises(error):
            g.int8_matmul(*args, **k)

    refused(ValueError, a.float(), w, sa, sw, d)
    refused(ValueError, a, w[:, :32], sa, sw, d)
    refused(ValueError, a, w, sa[:3], sw, d)
    refused(ValueError, a, w, sa, sw, d[:, :7])
    refused(ValueError, a, w, sa, sw, d, bias=sw.double())
    refused(ValueError, a.t(), w, sa, sw, d)
    refused(gemm_ws.GemmWSError, a, integers(N, K, gen, 72), sa, sw, d)            # w's rows off 16-byte boundaries
    refused(gemm_ws.GemmWSError, a, integers(N, K, gen, 64, 8), sa, sw, d)
    refused(gemm_ws.GemmWSError, a, w, sa, sw, d, bias=d.view(-1)[:N])             # d over the bias
    big = torch.empty(1, 1 << 17, dtype=torch.int8, device="cuda")
    refused(gemm_ws.GemmWSError, big, big, sa[:1], sw[:1], d[:1, :1])              # sums could pass 32 bits
    need = g.int8_matmul_workspace(M, N, K)
    if need > 0:
        refused(gemm_ws.GemmWSError, a, w, sa, sw, d, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    g.int8_matmul(a[:0], w, sa[:0], sw, d[:0])
    for bad in ((-1, 5, 5), (5, 0, 5), (5, 5, 0), (1 << 31, 5, 5), (5, 1 << 31, 5), (1 << 30, 16, 1 << 12)):
        with pytest.raises(gemm_ws.GemmWSError):
            g.int8_matmul_workspace(*bad)
    assert g.query_status() == gemm_ws.OK
