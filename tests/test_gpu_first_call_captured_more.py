"""The first calls in a process of attention, its gradients, the norm with an 8-bit output and
gradient clipping inside a graph capture, in a process of its own."""

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
dims = (64, 128)
data = {d: [torch.randn(n, 4, d, device="cuda").to(bf) for n in (600, 900, 900, 600)] for d in dims}
few = {d: torch.randn(2, 4, d, device="cuda").to(bf) for d in dims}
ws = B.Workspace(1 << 26)
x, y = torch.randn(300, 512, device="cuda").to(bf), torch.randn(300, 512, device="cuda").to(bf)
grads = [torch.randn(n, device="cuda") for n in range(8, 8 * 200, 8)]
outs = [torch.empty_like(t) for t in grads]

def step():
    got = []
    for d in dims:
        q, k, v, do = data[d]
        o, l = B.attention(q, k, v, ws)
        got += [o, l, *B.attention_bwd(q, k, v, o, l, do, ws)]
        got += B.attention(few[d], k, v, ws)              # keys in parts, and their join
        got += B.attention_bwd(q[:70], k[:90], v[:90], o[:70], l[:, :70].contiguous(), do[:70], ws)
    h, rstd, (q8, sf) = B.norm_quantize(x, residual=y)
    got += [h, rstd, q8.view(torch.uint8), sf, B.norm_quantize(x)[1]]
    return got + [B.grad_clip(grads, 1.0, ws, outs=outs), B.grad_clip(grads[:5], None, ws)]

torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
B.check(ws)
again = [t.clone() for t in outs]
for a, b in zip(got, step()):
    assert torch.equal(a, b)
for a, b in zip(again, outs):
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
