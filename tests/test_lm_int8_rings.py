"""The barriers of the 8-bit product's kernel: no wait by parity may find its barrier more than one phase further than the
one that it waits for, nor one behind, however late any of the kernel's warps, copies or commits are.

On the CPU a model of the warps, their waits and their arrivals runs with the rings that the kernel is launched with, each
party in turn held back as long as anything else can go on, and all of them in random order. On the GPU the warps that free
the tokens' stages are held up, by the debug build, and the product is the same.
"""
from __future__ import annotations

import ctypes
import random

import pytest
import torch

from async_pipelines_gb300 import build, gemm_ws
from tests.debug_helpers import configure, debug_handle
from tests.test_lm_int8 import integers, scales

WIDTHS = [32, 64, 96, 128, 160]
UNITS = [11, 3, 8, 1, 17, 9]   # stages of K of a cluster's units of work


class Barrier:
    def __init__(self, name, arrivals):
        self.name, self.arrivals, self.here, self.done = name, arrivals, 0, 0

    def arrive(self, phase, n=1):
        assert self.done == phase, f"{self.name}: an arrival for phase {phase} falls into phase {self.done}"
        self.here += n
        assert self.here <= self.arrivals, f"{self.name}: too many arrivals"
        if self.here == self.arrivals:
            self.here, self.done = 0, self.done + 1


class Model:
    """Parties are generators that yield the barrier and the number of the phase that they wait for (-1: one that a new
    barrier counts as past); what is in flight is in queues, each in its own order."""

    def __init__(self, bufs, w_stages, a_stages, t_full, converters, cut):
        self.bufs, self.ws, self.as_, self.cut, self.half = bufs, w_stages, a_stages, cut, converters // 2
        self.tellers = t_full - converters
        two = range(2)
        ring = lambda name, n, arrivals: [Barrier(f"{name}{i}", arrivals) for i in range(n)]  # noqa: E731
        self.w_full = [ring(f"w_full{r}.", w_stages, 2) for r in two]          # armed, and the copy
        self.w_empty = [ring(f"w_empty{r}.", w_stages, self.half) for r in two]
        self.a_full = ring("a_full", a_stages, 3)                              # armed, and both CTAs' copies
        self.a_empty = [ring(f"a_empty{r}.", a_stages, 1) for r in two]
        self.t_full = ring("t_full", bufs, t_full)
        self.t_empty = [ring(f"t_empty{r}.", bufs, 1) for r in two]
        self.acc_full = [ring(f"acc_full{r}.", 2, 1) for r in two]
        self.acc_empty = ring("acc_empty", 2, 2)
        self.steps = sum(UNITS)
        self.queues = {f"commits{r}": [] for r in two}
        self.parties = {"issue": self.issue()}
        for r in two:
            self.parties[f"w{r}"], self.parties[f"a{r}"] = self.load_w(r), self.load_a(r)
            self.parties[f"tell{r}"], self.parties[f"epilogue{r}"] = self.tell(r), self.epilogue(r)
            for g in two:
                for k in range(self.half):
                    self.parties[f"convert{r}.{g}.{k}"] = self.convert(r, g)
        self.at = {k: next(p) for k, p in self.parties.items()}

    def load_w(self, r):
        for i in range(self.steps):
            s, n = i % self.ws, i // self.ws
            yield self.w_empty[r][s], n - 1
            self.w_full[r][s].arrive(n)
            self.queues[f"copy w{r} {i}"] = [(self.w_full[r][s], n)]

    def load_a(self, r):
        for i in range(self.steps):
            s, n = i % self.as_, i // self.as_
            yield self.a_empty[r][s], n - 1
            if r == 0:
                self.a_full[s].arrive(n)
            self.queues[f"copy a{r} {i}"] = [(self.a_full[s], n)]

    def convert(self, r, group):
        for i in range(group, self.steps, 2):
            yield self.w_full[r][i % self.ws], i // self.ws
            self.w_empty[r][i % self.ws].arrive(i // self.ws)
            yield self.t_empty[r][i % self.bufs], i // self.bufs - 1
            self.t_full[i % self.bufs].arrive(i // self.bufs)

    def tell(self, r):
        if self.tellers:
            for t in range(self.bufs):
                self.t_full[t].arrive(0)
        for i in range(self.steps):
            yield self.t_empty[r][i % self.bufs], i // self.bufs
            self.a_empty[r][i % self.as_].arrive(i // self.as_)
            if self.tellers:
                self.t_full[i % self.bufs].arrive(i // self.bufs + 1)

    def issue(self):
        i = handed = 0
        for unit in UNITS:
            for first in range(0, unit, self.cut):
                yield self.acc_empty[handed % 2], handed // 2 - 1
                for _ in range(first, min(first + self.cut, unit)):
                    yield self.a_full[i % self.as_], i // self.as_
                    yield self.t_full[i % self.bufs], i // self.bufs
                    for r in range(2):
                        self.queues[f"commits{r}"].append((self.t_empty[r][i % self.bufs], i // self.bufs))
                    i += 1
                for r in range(2):
                    self.queues[f"commits{r}"].append((self.acc_full[r][handed % 2], handed // 2))
                handed += 1

    def epilogue(self, r):
        handed = 0
        for unit in UNITS:
            for _ in range(0, unit, self.cut):
                yield self.acc_full[r][handed % 2], handed // 2
                self.acc_empty[handed % 2].arrive(handed // 2)
                handed += 1

    def check(self):
        for k, (bar, n) in self.at.items():
            assert bar.done <= n + 1, f"{k} waits for phase {n} of {bar.name}, which is at {bar.done}: overtaken"
            assert bar.done >= n, f"{k} waits for phase {n} of {bar.name}, which is at {bar.done}: seen too early"

    def ready(self):
        """Who can go on; a wait by parity sees one bit of the phase."""
        return [k for k, (bar, n) in self.at.items() if (bar.done - n) % 2] + [k for k, q in self.queues.items() if q]

    def go(self, who):
        if who in self.queues:
            bar, n = self.queues[who].pop(0)
            bar.arrive(n)
            if who.startswith("copy"):
                del self.queues[who]
        else:
            try:
                self.at[who] = next(self.parties[who])
            except StopIteration:
                del self.at[who]
        self.check()

    def run(self, choose):
        while True:
            can = self.ready()
            if not can:
                break
            self.go(choose(can))
        assert not self.at, f"{sorted(self.at)} wait for ever"


def rings(bn):
    build.ensure_built()
    out = (ctypes.c_int * 6)()
    assert gemm_ws.load_debug_library().gemm_ws_debug_int8_rings(bn, out) == gemm_ws.OK
    return list(out)


def late(who, rng):
    """What `who` names, or begins the name of, only goes on once nothing else can."""
    def choose(can):
        others = [k for k in can if not (k in who if isinstance(who, tuple) else k.startswith(who))]
        return rng.choice(others or can)
    return choose


# ------------------------------------------------------------------ on the CPU

@pytest.mark.parametrize("who", ["tell0", "tell1", "tell", "convert0.0", "convert1.1", "convert0", "convert1.0.2", "w0", "w", "a1",
                                 "issue", "epilogue0", "epilogue", "copy w1", "copy a0", "commits0", "commits1", "nobody"])
@pytest.mark.parametrize("bn", WIDTHS)
def test_no_wait_is_overtaken(bn, who):
    shape = rings(bn)
    for seed in range(4):
        Model(*shape).run(late(who, random.Random(seed)))


@pytest.mark.parametrize("bn", WIDTHS)
def test_no_wait_is_overtaken_by_a_late_copy(bn):
    shape = rings(bn)
    for i in range(sum(UNITS)):
        for copy in (f"copy w0 {i}", f"copy a1 {i}"):
            Model(*shape).run(late((copy,), random.Random(i)))


@pytest.mark.parametrize("bn", WIDTHS)
def test_the_model_finds_late_tellers(bn):
    """Without the tellers' arrivals on the buffers' barriers."""
    bufs, ws, as_, _, converters, cut = rings(bn)
    with pytest.raises(AssertionError, match="tell0 waits .* overtaken"):
        Model(bufs, ws, as_, converters, converters, cut).run(late("tell0", random.Random(0)))


@pytest.mark.parametrize("bn", WIDTHS)
def test_the_model_finds_a_short_ring(bn):
    """An odd number of w's stages below that of its buffers and two: what one warpgroup takes for its stage is what the other
    has not been given yet."""
    bufs, _, as_, t_full, converters, cut = rings(bn)
    with pytest.raises(AssertionError, match="convert0.* waits .* too early"):
        for i in range(sum(UNITS)):
            Model(bufs, bufs - 1 + bufs % 2, as_, t_full, converters, cut).run(
                late((f"copy w0 {i}",), random.Random(i)))


def test_arguments_of_the_rings():
    build.ensure_built()
    dbg, out = gemm_ws.load_debug_library(), (ctypes.c_int * 6)()
    for bn in (0, 16, 33, 192, -32):
        assert dbg.gemm_ws_debug_int8_rings(bn, out) == gemm_ws.ERR_INVALID_ARG
    assert dbg.gemm_ws_debug_int8_rings(32, None) == gemm_ws.ERR_INVALID_ARG


# ------------------------------------------------------------------ on the GPU

@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(20, 600, 4096), (60, 600, 8192), (90, 3000, 2048), (130, 20000, 1100), (160, 5000, 1500),
                                   (700, 3000, 640), (2000, 9000, 1500)])
def test_late_tellers(M, N, K):
    """20 us for each tokens' stage, some thirty times a stage's own time."""
    gen = torch.Generator().manual_seed(M)
    g = debug_handle(timeout_ms=1000)
    a, w, sa, sw = integers(M, K, gen), integers(N, K, gen, (K + 15) // 16 * 16), scales(M, gen), scales(N, gen)
    d, late_d = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    g.int8_matmul(a, w, sa, sw, d)
    assert g.query_status() == gemm_ws.OK
    configure(g, fault=4)
    g.int8_matmul(a, w, sa, sw, late_d)
    assert g.query_status() == gemm_ws.OK
    configure(g, fault=0)
    assert torch.equal(d, late_d)
    g.close()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(20, 600, 4096), (160, 5000, 1500), (700, 3000, 640), (2000, 9000, 1500)])
def test_another_warp_gives_up_while_copies_are_under_way(M, N, K):
    """Copies of both operands have been started when the warp that issues the matrix instructions gives up: they land before the
    kernel ends, the call reports the timeout, and the next one is untroubled."""
    gen = torch.Generator().manual_seed(M)
    g = debug_handle(timeout_ms=100)
    a, w, sa, sw = integers(M, K, gen), integers(N, K, gen, (K + 15) // 16 * 16), scales(M, gen), scales(N, gen)
    want, d = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    g.int8_matmul(a, w, sa, sw, want)
    assert g.query_status() == gemm_ws.OK
    for _ in range(3):
        configure(g, fault=5)
        g.int8_matmul(a, w, sa, sw, d)
        assert g.query_status() == gemm_ws.ERR_TIMEOUT
        configure(g, fault=0)
        d.fill_(float("nan"))
        g.int8_matmul(a, w, sa, sw, d)
        assert g.query_status() == gemm_ws.OK
        assert torch.equal(d, want)
    g.close()
