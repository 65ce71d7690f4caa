"""Dropout with a residual on the GPU against its fp64 definition.

Tolerance: half a bf16 step, plus 2^-23 of |res| + |x| / (1 - p) for the fp32 product and
sum. The mask is exact.
"""

import numpy as np
import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF, close, f64, guarded, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.99])
@pytest.mark.parametrize("count", [1, 7, 8, 9, 4095, 4096, 4101])
@pytest.mark.parametrize("residual", [False, True])
def test_parity(count, p, residual):
    x, res = normal(1, count), normal(2, count)
    seed, offset = 0xFEDCBA9876543210, (1 << 40) + 5
    out, whole = guarded((count,), BF)
    B.dropout_add(x, p, seed, offset, residual=res if residual else None, out=out)
    assert whole()
    keep = ops.dropout_keep(range(count), p, seed, offset)
    scaled = f64(x) * 65536 / (65536 - ops.dropout_drop(p))
    base = f64(res) if residual else 0.0
    close(out, base + np.where(keep, scaled, 0.0), 2.0 ** -23 * (np.abs(base) + np.abs(scaled)))
    if not residual:
        assert (f64(out)[~keep] == 0).all()


def test_gradient_uses_the_forward_mask():
    """d out / d x by differences of the call itself: 0 where dropped, 1 / (1 - p) elsewhere."""
    p, args = 0.3, (0.3, 77, 123456789012)
    x = torch.zeros(50, 100, dtype=BF, device="cuda")
    up = B.dropout_add(x + 1, *args).double() - B.dropout_add(x, *args).double()
    dx = B.dropout_bwd(torch.ones_like(x), *args)
    assert torch.equal(dx.double(), up)
    scale = torch.tensor(65536 / (65536 - ops.dropout_drop(p))).to(BF).item()
    assert set(dx.unique().tolist()) == {0.0, scale}
    # 5000 draws: within five standard deviations of the share
    assert abs((dx != 0).double().mean().item() - 0.7) < 5 * (0.3 * 0.7 / 5000) ** 0.5
    dout = normal(3, 50, 100)
    keep = ops.dropout_keep(range(5000), *args).reshape(50, 100)
    exact = np.where(keep, f64(dout) * 65536 / (65536 - ops.dropout_drop(p)), 0.0)
    close(B.dropout_bwd(dout, *args), exact, 2.0 ** -23 * np.abs(exact))


def test_drops_what_is_not_finite_and_keeps_the_residual():
    x = torch.full((4096,), float("nan"), dtype=BF, device="cuda")
    x[::2] = float("inf")
    res = normal(4, 4096)
    out = B.dropout_add(x, 0.5, 9, residual=res)
    keep = torch.from_numpy(ops.dropout_keep(range(4096), 0.5, 9, 0)).cuda()
    assert torch.equal(out[~keep], res[~keep]) and not torch.isfinite(out[keep]).any()


@pytest.mark.parametrize("which", ["x", "residual"])
def test_in_place(which):
    x, res = normal(5, 1001), normal(6, 1001)
    want = B.dropout_add(x, 0.2, 1, 2, residual=res)
    out = x if which == "x" else res
    assert B.dropout_add(x, 0.2, 1, 2, residual=res, out=out) is out
    assert torch.equal(out, want)


def test_masks_differ_by_seed_and_offset_and_counter_adds_to_the_offset():
    x = torch.ones(4096, dtype=BF, device="cuda")
    a = B.dropout_add(x, 0.5, 1, 0)
    assert not torch.equal(a, B.dropout_add(x, 0.5, 2, 0))
    assert not torch.equal(a, B.dropout_add(x, 0.5, 1 << 32, 0))
    b = B.dropout_add(x, 0.5, 1, 7)
    assert not torch.equal(a, b)
    assert torch.equal(b, B.dropout_add(x, 0.5, 1, 4, counter=torch.tensor([3], device="cuda")))
    top = B.dropout_add(x, 0.5, 1, (1 << 64) - 1, counter=torch.tensor([8], device="cuda"))
    assert torch.equal(b, top)                          # the sum wraps


def test_beyond_2_31_elements():
    n = (1 << 31) + 1003
    x = torch.ones(n, dtype=BF, device="cuda")
    B.dropout_add(x, 0.5, 11, 12, out=x)
    for e0 in (0, (1 << 31) - 500, n - 777):
        at = range(e0, min(n, e0 + 777))
        np.testing.assert_array_equal(f64(x[at.start:at.stop]) != 0, ops.dropout_keep(at, 0.5, 11, 12))


def test_refuses_what_the_binding_sees():
    x = normal(7, 64)
    for kw in (dict(residual=normal(8, 32)), dict(out=torch.empty(32, dtype=BF, device="cuda")),
               dict(residual=x.cpu()), dict(counter=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            B.dropout_add(x, 0.1, 0, **kw)
    for seed, offset in ((-1, 0), (1 << 64, 0), (0, -1)):
        with pytest.raises(ValueError):
            B.dropout_add(x, 0.1, seed, offset)
    with pytest.raises(TypeError):
        B.dropout_add(x.float(), 0.1, 0)
    with pytest.raises(ValueError):
        B.dropout_add(normal(7, 8, 8).T, 0.1, 0)
    for p in (1.0, -0.5, 1e-6):
        with pytest.raises(B.BoostError):
            B.dropout_add(x, p, 0)
    assert B.dropout_add(x[:0], 0.5, 0).numel() == 0


def test_another_stream_and_a_replayed_graph_that_takes_new_masks():
    x, res = normal(9, 300, 520), normal(10, 300, 520)
    want = B.dropout_add(x, 0.25, 5, 3, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = B.dropout_add(x, 0.25, 5, 3, residual=res, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = B.dropout_add(x, 0.25, 5, residual=res, counter=counter)
        counter.add_(1)
    for at in range(3):
        graph.replay()
        assert torch.equal(out, B.dropout_add(x, 0.25, 5, at, residual=res))
