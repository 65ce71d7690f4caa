"""Rotary positions with frequencies of many turns a position, against their fp64 definition.

Tolerance: the angle is (1 + |w| 2^-64) 2^-64 |p| turns off at most, under 2^-63 |p| for the
frequencies that are allowed, beside what an angle of any size loses (2^-20 of |u| + |v|: the
rounding of the angle, the sine, the cosine and the three operations).
"""

import math

import numpy as np
import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import close, f64, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


FAST = [7.0, -1e3, 1e6, -1e9, 1e12, 3e15, -2.0 ** 63, math.nextafter(2.0 ** 64, 0)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [1, 8191, (1 << 31) - 1, 1 << 40])
def test_fast_frequencies(far, interleaved):
    T, w = 24, np.array(FAST)
    rng = np.random.default_rng(far)
    pos = rng.integers(-far, far + 1, (1, T))
    pos[0, :2] = far, -far
    q = normal(1, T, 2, 16)
    out, _ = B.rope(q, None, torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(),
                    interleaved=interleaved)
    a = np.abs(f64(q))
    u, v = (a[..., 0::2], a[..., 1::2]) if interleaved else (a[..., :8], a[..., 8:])
    s = np.stack([u + v, u + v], -1).reshape(a.shape) if interleaved else np.concatenate([u + v] * 2, -1)
    close(out, ops.rope(f64(q), pos, w, [0] * 8, interleaved),
          s * (2.0 ** -20 + 2 * math.pi * far * 2.0 ** -63))


def test_frequencies_without_an_angle():
    """Those of 2^64 and more, and those that are not finite, give NaN."""
    w = [2.0 ** 64, -2.0 ** 64, 1e300, math.inf, -math.inf, math.nan, 1.0, 0.0]
    q = normal(2, 3, 1, 16)
    out = f64(B.rope(q, None, torch.tensor([0, 1, 5], dtype=torch.int32, device="cuda"),
                     torch.tensor(w, dtype=torch.float64, device="cuda"))[0])
    bad = [0, 1, 2, 3, 4, 5, 8, 9, 10, 11, 12, 13]
    assert np.isnan(out[..., bad]).all() and np.isfinite(np.delete(out, bad, axis=2)).all()


@pytest.mark.parametrize("w", [2.0 ** -64, 2.0 ** -41 * 1.7, -2.0 ** -40, 1e-9])
def test_slow_frequencies(w):
    far = 1 << 40
    pos = np.array([[far, -far, 1, 0]])
    q = normal(3, 4, 1, 16)
    out, _ = B.rope(q, None, torch.from_numpy(pos).cuda(),
                    torch.full((8,), w, dtype=torch.float64, device="cuda"))
    a = np.abs(f64(q))
    s = np.concatenate([a[..., :8] + a[..., 8:]] * 2, -1)
    close(out, ops.rope(f64(q), pos, np.full(8, w), [0] * 8),
          s * (2.0 ** -20 + 2 * math.pi * far * 2.0 ** -63))
