"""The first call of a process, captured: a kernel is loaded while its stream
records, and the replays give the eager results."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import fp8_grouped_gemm_amd as moe
rows, n, k = {sizes}
u = lambda *s: torch.randint(0, 120, s, dtype=torch.uint8, device="cuda")
x = torch.randn(rows, k, device="cuda")
b, b_sf = u(n, k // 2), u(n, k // 32)
src = torch.arange(rows, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
def run():
    p = moe.moe_permute(x, src, src, None)
    a, a_sf = moe.moe_quantize_mxfp4(p)
    y = moe.moe_gemm_mxfp4(a, a_sf, b, b_sf, dtype=torch.float32)
    z = moe.moe_unpermute(y, src, rows)
    dyp, dw = moe.moe_unpermute_bwd(z, y, src, src, None)
    return y, z, dyp, dw, moe.moe_permute_bwd(p, src, rows), moe.moe_dequantize_mxfp4(a, a_sf)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
for _ in range(3):
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    got = [v.clone() for v in out]
    assert all(torch.equal(v, w) for v, w in zip(got, run()))
print("replays equal", moe.moe_gemm_mxfp4_info(rows, n, k))
"""


@pytest.mark.parametrize("sizes", [(5, 600, 512), (4096, 4096, 1024)])
def test_first_call_is_captured(sizes):
    run = subprocess.run([sys.executable, "-c", PROGRAM.format(sizes=sizes)], cwd=Path(__file__).parents[1],
                         capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and "replays equal" in run.stdout, run.stdout + run.stderr
