"""Penalties, biases and masks on logits, against a plain implementation in 64 bits.

Tolerances, fixed before the first run: five operations of 32 bits (2^-24 each of the magnitudes that they add: within 2^-21)
and one addition for each bias of the same token, then one rounding to the output's type.
"""
from __future__ import annotations

import math

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
    assert lib.gemm_ws_adjust_logits(None, 0, None, 8, 0, None, 8, None, 8, 0, 0, None, None, None, None, None, None, 8, 0,
                                     None, 0, 0, None, 0, 1, 8, None) == gemm_ws.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def g():
    handle = gemm_ws.GemmWS(0)
    yield handle
    handle.close()


def close(got, want, dtype, size, slack=2.0 ** -20):
    got = got.cpu().double()
    most = torch.finfo(dtype).max
    fine = want.abs() < most * 0.99
    assert torch.equal(got[~fine & (want == -math.inf)], want[~fine & (want == -math.inf)])
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    tol = UNIT[dtype] * want.abs() + slack * size + TINY[dtype]
    off = (got - want).abs()[fine]
    assert bool((off <= tol[fine]).all()), f"worst {float((off / tol[fine]).max()):.3g} of the tolerance"


def words(rows, vocab, gen, share):
    bits = torch.rand(rows, (vocab + 31) // 32, 32, generator=gen) < share
    value = (bits.long() << torch.arange(32)).sum(2)
    return (value - ((value >> 31) << 32)).int()


def inputs(rows, vocab, dtype, history, biases, share, seed, wide=True, pad=0):
    gen = torch.Generator().manual_seed(seed)
    kind = torch.int64 if wide else torch.int32
    v = {"logits": (3.0 * torch.randn(rows, vocab + pad, generator=gen)).to(dtype)[:, :vocab]}
    if history:
        t = (vocab ** torch.rand(rows, history, generator=gen) - 1).long().clamp(0, vocab - 1)
        t[torch.rand(rows, history, generator=gen) < 0.05] = -1         # padding
        t[torch.rand(rows, history, generator=gen) < 0.05] = vocab      # and past the end
        v["tokens"] = t.to(kind)
        v["lengths"] = torch.randint(0, history + 1, (rows,), generator=gen).int()
        v["prompt_lengths"] = torch.randint(0, history + 1, (rows,), generator=gen).int()
        v["repetition"] = 0.7 + torch.rand(rows, generator=gen)
        v["frequency"] = torch.randn(rows, generator=gen)
        v["presence"] = torch.randn(rows, generator=gen)
    if biases:
        b = torch.randint(0, vocab, (rows, biases), generator=gen)
        b[:, biases // 2:] = b[:, :biases - biases // 2]                # tokens given twice
        b[torch.rand(rows, biases, generator=gen) < 0.05] = -7
        v["bias_tokens"], v["bias_values"] = b.to(kind), torch.randn(rows, biases, generator=gen)
    if share is not None:
        v["allowed"] = words(rows, vocab, gen, share)
    return v


def check(g, v, out_type, pad=0):
    logits = v["logits"]
    rows, vocab = logits.shape
    dev = {k: t.cuda() for k, t in v.items()}
    dev["logits"] = torch.as_strided(logits, (rows, logits.stride(0)), (logits.stride(0), 1)).cuda()[:, :vocab] \
        if rows > 1 else logits.cuda()
    buf = torch.full((rows, vocab + pad), 7.0, dtype=out_type, device="cuda")
    out = buf[:, :vocab]
    g.adjust_logits(dev.pop("logits"), out, **dev)
    names = {"prompt_lengths": "prompts"}
    want, size = ref.adjust_logits(**{names.get(k, k): t for k, t in v.items()})
    close(out, want, out_type, size)
    assert bool((buf[:, vocab:] == 7).all())


SIZES = [(1, 1), (1, 8), (3, 31), (2, 33), (2, 100), (5, 2048), (3, 2049), (2, 5000), (1, 40007), (2, 33000), (400, 65)]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_everything_at_once(g, dtype, rows, vocab):
    for out_type in {dtype, torch.float32}:
        check(g, inputs(rows, vocab, dtype, 60, 12, 0.5, rows + vocab), out_type)


@gpu
@pytest.mark.parametrize("history,biases,share", [(0, 0, None), (1, 0, None), (500, 0, None), (0, 1, None), (0, 300, None),
                                                  (0, 1024, None), (0, 0, 0.02), (0, 0, 0.0), (40, 0, 0.9), (40, 300, None)])
@pytest.mark.parametrize("wide", [True, False])
def test_each_alone(g, history, biases, share, wide):
    check(g, inputs(3, 1000, torch.bfloat16, history, biases, share, history + biases, wide), torch.bfloat16)
    check(g, inputs(2, 20011, torch.float32, history, biases, share, history + biases, wide), torch.float32)


@gpu
@pytest.mark.parametrize("dtype,out_type", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
@pytest.mark.parametrize("pad,out_pad", [(1, 0), (8, 3), (0, 1), (24, 8)])
def test_rows_that_lie_anywhere(g, dtype, out_type, pad, out_pad):
    check(g, inputs(4, 2600, dtype, 100, 7, 0.8, pad, pad=pad), out_type, out_pad)
    check(g, inputs(3, 2603, dtype, 100, 7, 0.8, pad, pad=pad), out_type, out_pad)


@gpu
def test_parts_that_are_not_given(g):
    v = inputs(3, 500, torch.float32, 80, 0, None, 3)
    for keep in ((), ("repetition",), ("frequency",), ("presence",), ("lengths", "presence"),
                 ("prompt_lengths", "repetition", "frequency")):
        check(g, {k: t for k, t in v.items() if k in keep + ("logits", "tokens")}, torch.float32)


@gpu
def test_counts_of_long_histories(g):
    """One token 40000 times, in the prompt and after it; lengths outside the history."""
    n = 40000
    tokens = torch.full((4, n), 5, dtype=torch.int32)
    tokens[:, ::2] = torch.arange(n // 2, dtype=torch.int32) % 700
    v = {"logits": torch.randn(4, 700, generator=torch.Generator().manual_seed(1)), "tokens": tokens,
         "lengths": torch.tensor([n, n + 5, -3, 17], dtype=torch.int32),
         "prompt_lengths": torch.tensor([n // 2, 0, 5, 100], dtype=torch.int32),
         "repetition": torch.tensor([1.5, 1.0, 2.0, 1.3]), "frequency": torch.tensor([1e-3, 0.5, 1.0, 2.0]),
         "presence": torch.tensor([0.5, 0.25, 1.0, 2.0])}
    check(g, v, torch.float32)


@gpu
def test_infinities_and_nan(g):
    inf, nan = math.inf, math.nan
    row = torch.tensor([inf, -inf, nan, 0.0, -0.0, torch.finfo(torch.float32).min, 1.0, 2.0] * 5)
    logits = torch.stack([row, row, row])
    tokens = torch.arange(40)[None].repeat(3, 1)
    v = {"logits": logits, "tokens": tokens, "repetition": torch.tensor([1.5, 1.0, 0.5]),
         "presence": torch.tensor([0.0, 1.0, -1.0]), "bias_tokens": torch.tensor([[0, 1, 6], [0, 2, 7], [1, 1, 3]]),
         "bias_values": torch.tensor([[-inf, 5.0, inf], [1.0, 1.0, -inf], [1.0, 2.0, nan]])}
    out = torch.empty(3, 40, device="cuda")
    g.adjust_logits(logits.cuda(), out, **{k: t.cuda() for k, t in v.items() if k != "logits"})
    want, _ = ref.adjust_logits(**v)
    # what passes the type's range is an infinity in 32 bits
    want = want.float()
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    assert torch.equal(out.cpu().isposinf(), want.isposinf()) and torch.equal(out.cpu().isneginf(), want.isneginf())
    # a place that is not allowed is -inf whatever it held
    none = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    g.adjust_logits(logits.cuda(), out, allowed=none)
    assert bool((out == -inf).all())


@gpu
@pytest.mark.parametrize("vocab", [3000, 3001])
def test_in_place_graphs_and_streams(g, vocab):
    v = inputs(20, vocab, torch.bfloat16, 200, 20, 0.7, 5)
    dev = {k: t.cuda() for k, t in v.items()}
    logits = dev.pop("logits")
    first, second = torch.empty_like(logits), torch.empty_like(logits)
    g.adjust_logits(logits, first, **dev)
    place = logits.clone()
    g.adjust_logits(place, place, **dev)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        g.adjust_logits(logits, second, **dev)
    for _ in range(2):
        second.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(place, first) and torch.equal(second, first)
    # the history is read when the graph runs
    dev["lengths"].zero_()
    graph.replay()
    g.adjust_logits(logits, first, **dev)
    torch.cuda.synchronize()
    assert torch.equal(second, first)


@gpu
def test_refusals(g):
    z = torch.zeros(3, 100, device="cuda")
    out, t = torch.empty_like(z), torch.zeros(3, 10, dtype=torch.int64, device="cuda")
    f, n = torch.ones(3, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")

    def refused(error, *a, **k):
        with pytest.raises(error):
            g.adjust_logits(*a, **k)

    refused(ValueError, z, out.half())
    refused(ValueError, z, out[:, :50])
    refused(ValueError, z, out, tokens=t.short())
    refused(ValueError, z, out, tokens=t[:2])
    refused(ValueError, z, out, repetition=f)                       # no history
    refused(ValueError, z, out, tokens=t, lengths=n.long())
    refused(ValueError, z, out, tokens=t, presence=f.double())
    refused(ValueError, z, out, bias_tokens=t)
    refused(ValueError, z, out, bias_tokens=t, bias_values=out[:, :9])
    refused(ValueError, z, out, allowed=torch.zeros(3, 3, dtype=torch.int32, device="cuda"))
    refused(gemm_ws.GemmWSError, z, z[:, :], allowed=z.view(torch.int32)[:, :4])       # out over the mask
    wide = torch.zeros(3, 1025, device="cuda")
    refused(gemm_ws.GemmWSError, z, out, bias_tokens=wide.long(), bias_values=wide)
    shifted = torch.zeros(400, device="cuda")
    refused(gemm_ws.GemmWSError, shifted[:300].view(3, 100), shifted[50:350].view(3, 100))
    g.adjust_logits(z[:0], out[:0])
    assert g.query_status() == gemm_ws.OK
