"""What the 8-bit product refuses, it refuses before anything is launched; and the build itself looks at the registers that the
product's warpgroups share out."""
from __future__ import annotations

import pytest
import torch

from async_pipelines_gb300 import build, gemm_ws
from tests.debug_helpers import configure, debug_handle
from tests.test_lm_int8 import integers, scales

REPORT = """ptxas info    : Compiling entry function '_ZN3gws2i810dot_kernelILi1EEEvNS0_9DotParamsE' for 'sm_103a'
ptxas info    : Function properties for _ZN3gws2i810dot_kernelILi1EEEvNS0_9DotParamsE
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 40 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN3gws2i814product_kernelENS0_6ParamsE' for 'sm_103a'
ptxas info    : Function properties for _ZN3gws2i814product_kernelENS0_6ParamsE
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers
"""


def test_registers_of_the_build():
    assert build.used_registers(REPORT % 96, "product_kernel") == 96
    assert build.used_registers(REPORT % 96, "dot_kernel") == 40
    build.check_registers(REPORT % 96)
    for other in (88, 104):
        with pytest.raises(RuntimeError, match=f"{other} registers"):
            build.check_registers(REPORT % other)
    with pytest.raises(RuntimeError, match="no product_kernel"):
        build.check_registers("")


def test_status_of_its_own():
    build.ensure_built()
    text = gemm_ws.status_string(gemm_ws.ERR_BUILD)
    assert "registers" in text and text != gemm_ws.status_string(gemm_ws.ERR_UNSUPPORTED)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(20, 600, 4096), (700, 3000, 640)])
def test_a_refused_product_launches_nothing(M, N, K):
    gen = torch.Generator().manual_seed(M)
    g = debug_handle()
    a, w, sa, sw = integers(M, K, gen), integers(N, K, gen), scales(M, gen), scales(N, gen)
    d = torch.full((M, N), 7.0, device="cuda")
    ws = torch.full((g.int8_matmul_workspace(M, N, K),), 255, dtype=torch.uint8, device="cuda")
    configure(g, fault=6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.add_(1.0)
        with pytest.raises(gemm_ws.GemmWSError) as e:
            g.int8_matmul(a, w, sa, sw, d, workspace=ws)
    assert e.value.status == gemm_ws.ERR_BUILD
    with pytest.raises(gemm_ws.GemmWSError):
        g.int8_matmul(a, w, sa, sw, d, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert bool((ws == 255).all()) and bool((d == 8.0).all())
    configure(g, fault=0)
    g.int8_matmul(a, w, sa, sw, d, workspace=ws)
    assert g.query_status() == gemm_ws.OK and not bool((ws == 255).all())
    g.close()
