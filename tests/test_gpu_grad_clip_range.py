"""Clipping by factors below fp32's normal numbers: gradients of which even the smallest factor leaves
values that count. A scaled value is off by the factor's rounding, the product's and the norm's (2^-20,
test_gpu_grad_clip), and by half a step of its type, which below the normal numbers is absolute."""

import numpy as np
import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF, f64

pytestmark = pytest.mark.gpu

NORM = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("big,most", [(3e38, 1.0), (3e38, 1e-3), (1e38, 1e-20), (3e38, 1e-38), (1.0, 1e-36),
                                      (1e30, 1e-30), (2e38, 1e-44), (1e-3, 1e-42), (1e20, 0.0)])
def test_small_factors(big, most, dtype, in_place):
    """Whole chunks and a ragged one, of values from 2^-20 to 1 times `big`."""
    g = torch.Generator().manual_seed(11)
    sizes = (8192 * 8, 8192 + 77, 5)
    grads = [(torch.randn(n, generator=g).clamp(-1, 1).double() * big
              * torch.exp2(-20 * torch.rand(n, generator=g).double())).to(dtype).cuda() for n in sizes]
    before = [t.clone() for t in grads]
    ws = B.Workspace(B.grad_clip_workspace_bytes())
    outs = None if in_place else [torch.empty_like(t) for t in grads]
    B.grad_clip(grads, most, ws, outs=outs)
    _, want = ops.grad_clip([f64(t) for t in before], most)
    half, tiny = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    for a, w in zip(grads if in_place else outs, want):
        # (a product below the normal numbers is rounded in fp32 and, for bf16, once more)
        slack = (half + 2 * NORM) * np.abs(w) + tiny / 2 + 2.0 ** -149
        assert (np.abs(f64(a) - w) <= slack).all()
