"""Gradients of zeros in clipping: as quick as any values, and told from values whose squares fp32
does not hold. Tolerances: test_gpu_grad_clip."""

import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF

pytestmark = pytest.mark.gpu

NORM = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


@pytest.fixture(scope="module")
def ws():
    return B.Workspace(B.grad_clip_workspace_bytes())


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_zeros_of_either_sign_and_values_too_small_to_square(dtype, ws):
    """Threads of zeros beside threads whose squares are 0 in fp32, in whole chunks and ragged ones."""
    tiny = 2.0 ** -100
    for n in (5, 8192, 3 * 8192 + 77):
        g = torch.zeros(n, dtype=dtype, device="cuda")
        assert B.grad_clip([g], None, ws).item() == 0
        g[::2] = -0.0
        assert B.grad_clip([g], None, ws).item() == 0
        g[n // 2] = tiny
        assert B.grad_clip([g], None, ws).item() == tiny
        g[-1] = -2.0 * tiny
        assert abs(B.grad_clip([g], None, ws).item() - 5 ** 0.5 * tiny) <= NORM * 3 * tiny


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_zeros_take_no_longer_than_values(dtype, ws):
    """The norm of 2^27 zeros and of as many values, in turn: the least of ten times each. (Threads
    that read their zeros again, one by one, took several times as long.)"""
    some = torch.randn(1 << 27, device="cuda").to(dtype)
    none = torch.zeros_like(some)
    norm = torch.empty(1, device="cuda")
    times = {}
    for _ in range(11):                  # (the first round warms up)
        for name, t in (("some", some), ("none", none)):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            B.grad_clip([t], None, ws, norm=norm)
            b.record()
            b.synchronize()
            times.setdefault(name, []).append(a.elapsed_time(b))
    least = {name: min(t[1:]) for name, t in times.items()}
    assert least["none"] <= 1.3 * least["some"], least
