"""Shared helpers of the GPU tests of the operators around the block."""

import math

import numpy as np
import torch

BF = torch.bfloat16
HALF_STEP = torch.finfo(BF).eps / 2
SENTINEL = 0x5A


def f64(t):
    return t.detach().cpu().double().numpy()


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def guarded(shape, dtype):
    """A tensor between two guards, and a function that says whether the guards are whole."""
    pad = 512
    n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((2 * pad + (n + 255) // 256 * 256,), SENTINEL, dtype=torch.uint8, device="cuda")

    def whole():
        return bool((raw[:pad] == SENTINEL).all() and (raw[pad + n:] == SENTINEL).all())

    return raw[pad:pad + n].view(dtype).view(shape), whole


def close(got, want, slack):
    """|got - want| <= half a bf16 step of the value before rounding + slack, what the fp32
    arithmetic before the rounding may lose."""
    g = f64(got)
    assert g.shape == want.shape and np.isfinite(g).all()
    off = np.abs(g - want) - (HALF_STEP * (np.abs(want) + slack) + slack)
    assert off.max(initial=-1.0) <= 0, f"off by {off.max():.3e} more than allowed"
