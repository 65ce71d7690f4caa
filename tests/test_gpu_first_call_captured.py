"""The operators' first call in a process inside a graph capture: kernel attributes and
occupancies are asked for then, and no call may need one outside first. In a process of its
own, since the calls of other tests would come before.
"""

import os
import subprocess
import sys

import pytest
import torch

from rank_bottleneck_online_gb300 import build as build_mod

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
from rank_bottleneck_online_gb300 import binding as B
bf = torch.bfloat16
x, w = torch.randn(300, 512, device="cuda").to(bf), torch.randn(512, 512, device="cuda").to(bf)
pos, f = torch.arange(300, dtype=torch.int32, device="cuda"), torch.ones(32, dtype=torch.float64, device="cuda")
ws = B.Workspace(B.fp8_matmul_workspace_bytes(300, 512, 512))

def step():
    (a, sa), _ = B.fp8_quantize(x, way="both")
    (b, sb), _ = B.fp8_quantize(w, block_rows=128, way="both")
    y = B.fp8_matmul(a, sa, b, sb, 512, ws)
    z = B.fp8_matmul(a[:5].contiguous(), sa[:512].contiguous(), b, sb, 512, ws)   # few rows
    y = B.dropout_add(y, 0.5, 1, residual=x)
    return y, z, B.rope(y.view(300, 8, 64), None, pos, f)[0]

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
B.check(ws)
for a, b in zip(got, step()):
    assert torch.equal(a, b)
print("same")
"""


def test_first_call_inside_a_capture():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
