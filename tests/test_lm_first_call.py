"""What a program pays before its first call, and first calls inside a graph's capture.

Each case runs in a process of its own, where nothing is loaded yet.
"""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(script):
    out = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    return out.stdout.split()[-1]


def test_a_handle_loads_no_operator():
    """Loading the operators' kernels takes about 20 ms, the rest of a handle below 1."""
    took = run("""
import time, torch
from async_pipelines_gb300 import gemm_ws
torch.zeros(1, device="cuda"); torch.cuda.synchronize()
gemm_ws.load_library()
start = time.perf_counter()
gemm_ws.GemmWS(0)
print(1e3 * (time.perf_counter() - start))
""")
    assert float(took) < 8.0


@pytest.mark.parametrize("order", ["captured", "eager"])
def test_first_calls_inside_a_capture(order):
    """Kernels that take more shared memory than usual, first used while a graph is captured."""
    same = run(f"""
import torch
from async_pipelines_gb300 import gemm_ws
g = gemm_ws.GemmWS(0)
T, H, V = 1300, 1024, 9000
gen = torch.Generator("cuda").manual_seed(1)
x, res, dy = (torch.randn(T, H, device="cuda", generator=gen).bfloat16() for _ in range(3))
head = (torch.randn(V, H, device="cuda", generator=gen) / 32).bfloat16()
norm = torch.ones(H, device="cuda", dtype=torch.bfloat16)
t = torch.randint(V, (T,), device="cuda", generator=gen)
rng = torch.tensor([3, 4], device="cuda")
y, h, dx, dy2, du = (torch.empty_like(x) for _ in range(5))
rstd, loss, lse, mean = (torch.empty(n, device="cuda") for n in (T, T, T, 2))
dhead, dnorm = torch.empty_like(head), torch.empty_like(norm)
ws = torch.empty(max(g.linear_cross_entropy_workspace(T, H, V, b) for b in (False, True)),
                 dtype=torch.uint8, device="cuda")
def step():
    g.add_rms_norm(x, norm, y, residual=res, h=h, rstd=rstd, p=0.1, rng=rng)
    g.linear_cross_entropy(y, head, t, loss, lse, mean=mean, workspace=ws)
    g.linear_cross_entropy_backward(y, head, t, lse, mean[1:], dx=dy2, dweight=dhead, workspace=ws)
    g.add_rms_norm_backward(dy2, h, norm, rstd, du, dnorm, p=0.1, rng=rng)
outs = (y, h, rstd, loss, lse, mean, dy2, dhead, du, dnorm)
if "{order}" == "eager":
    step()
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    step()
for v in outs:
    v.fill_(float("nan"))
graph.replay()
torch.cuda.synchronize()
first = [v.clone() for v in outs]
for v in outs:
    v.fill_(float("nan"))
step()
assert g.query_status() == gemm_ws.OK
print(all(torch.equal(a, b) and torch.isfinite(a.float()).all() for a, b in zip(first, outs)))
""")
    assert same == "True"
