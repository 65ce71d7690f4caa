"""Gradient clipping on the GPU. Tolerances: a thread's squares are summed in fp32, 32 of them,
each step off by 2^-24 of the sum, so the norm by 2^-20 of itself at most; a scaled value by that
and half a step of its type."""

import numpy as np
import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF, f64, guarded

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


def make(sizes, dtypes, seed=0, std=0.1):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(d).cuda() for n, d in zip(sizes, dtypes)]


def compare(got, norm, grads, max_norm):
    want_norm, want = ops.grad_clip([f64(t) for t in grads], max_norm)
    assert abs(norm.item() - want_norm) <= (NORM + 2.0 ** -24) * want_norm
    for a, g, w in zip(got, grads, want):
        assert a.dtype == g.dtype
        half = torch.finfo(g.dtype).eps / 2
        assert (np.abs(f64(a) - w) <= (half + 2 * NORM) * np.abs(w)).all()


SIZES = [1, 7, 8, 9, 4095, 8191, 8192, 8193, 100001, 3 * 8192]


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 3.0, 1e6])
@pytest.mark.parametrize("types", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("in_place", [True, False])
def test_parity(in_place, types, max_norm, ws):
    dtypes = {"bf16": [BF], "fp32": [torch.float32], "mixed": [BF, torch.float32]}[types] * 10
    grads = make(SIZES, dtypes)
    before = [t.clone() for t in grads]
    outs = None if in_place else [guarded(t.shape, t.dtype) for t in grads]
    norm = B.grad_clip(grads, max_norm, ws, outs=None if in_place else [t for t, _ in outs])
    if in_place:
        compare(grads, norm, before, max_norm)
    else:
        assert all(whole() for _, whole in outs)
        for a, b in zip(grads, before):
            assert torch.equal(a, b)
        compare([t for t, _ in outs], norm, before, max_norm)
    if max_norm == 1e6:                                 # nothing to scale: the same bits
        for a, b in zip(grads if in_place else [t for t, _ in outs], before):
            assert torch.equal(a, b)


@pytest.mark.parametrize("count", [119, 120, 121, 241, 1000])
def test_more_tensors_than_a_launch_takes(count, ws):
    rng = np.random.default_rng(count)
    grads = make([int(n) for n in rng.integers(0, 20000, count)], [BF, torch.float32] * count, seed=1)
    before = [t.clone() for t in grads]
    norm = B.grad_clip(grads, 1.0, ws)
    compare(grads, norm, before, 1.0)
    assert torch.equal(norm, B.grad_clip(before, None, ws))       # the same bits, and no scaling
    compare(before, norm, before, float("inf"))


def test_the_norm_alone_writes_nothing_else(ws):
    grads = make(SIZES, [BF] * 10, seed=2)
    before = [t.clone() for t in grads]
    norm = B.grad_clip(grads, None, ws)
    for a, b in zip(grads, before):
        assert torch.equal(a, b)
    compare(before, norm, before, float("inf"))


def test_small_values_beside_a_large_one(ws):
    """2^26 values whose squares are 2^-24 of the first's: a running fp32 sum would lose them."""
    n = 1 << 26
    big, small = torch.ones(1, device="cuda"), torch.full((n,), 2.0 ** -12, device="cuda")
    norm = B.grad_clip([big, small], None, ws)
    assert abs(norm.item() - 5 ** 0.5) <= 5 ** 0.5 * NORM


def test_empty_and_no_tensors(ws):
    assert B.grad_clip([], 1.0, ws).item() == 0
    empty = torch.empty(0, dtype=BF, device="cuda")
    assert B.grad_clip([empty, empty], 1.0, ws).item() == 0
    g = make([100], [BF], seed=3)
    before = g[0].clone()
    norm = B.grad_clip([empty, g[0], empty], 0.1, ws)
    compare(g, norm, [before], 0.1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(bad, ws):
    """As the formula: all NaN from a NaN; from an infinity zeros, and NaN in its place."""
    g = make([9000, 50], [BF, torch.float32], seed=4)
    g[0][17] = bad
    norm = B.grad_clip(g, 1.0, ws)
    if np.isnan(bad):
        assert torch.isnan(norm).all() and all(torch.isnan(t).all() for t in g)
    else:
        assert norm.item() == float("inf") and torch.isnan(g[0][17])
        g[0][17] = 0
        assert all((t == 0).all() for t in g)


def test_replayed_graph_and_another_stream(ws):
    g = make(SIZES, [BF, torch.float32] * 5, seed=5)
    outs = [torch.empty_like(t) for t in g]
    graph = torch.cuda.CUDAGraph()
    own = B.Workspace(B.grad_clip_workspace_bytes())
    with torch.cuda.graph(graph):
        norm = B.grad_clip(g, 1.0, own, outs=outs)
    for seed in (6, 7):
        for t, new in zip(g, make(SIZES, [BF, torch.float32] * 5, seed=seed)):
            t.copy_(new)
        graph.replay()
        compare(outs, norm, g, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = [torch.empty_like(t) for t in g]
    n2 = B.grad_clip(g, 1.0, ws, outs=again, stream=side)
    side.synchronize()
    assert torch.equal(n2, norm) and all(torch.equal(a, b) for a, b in zip(again, outs))


def test_beyond_2_31_elements(ws):
    n = (1 << 31) + 12345
    g = torch.full((n,), 0.5, dtype=BF, device="cuda")
    g[-1] = 3.0
    norm = B.grad_clip([g], 1.0, ws)
    want = ((n - 1) * 0.25 + 9) ** 0.5
    assert abs(norm.item() - want) <= want * NORM
    assert abs(g[-1].item() - 3 / want) <= 2.0 ** -7 * 3 / want
    assert abs(g[n // 2].item() - 0.5 / want) <= 2.0 ** -7 * 0.5 / want


def test_refuses_what_the_binding_sees(ws):
    g = make([64, 64], [BF, BF])
    with pytest.raises(TypeError):
        B.grad_clip([g[0].half()], 1.0, ws)
    with pytest.raises(ValueError):
        B.grad_clip([g[0].view(8, 8).T], 1.0, ws)
    with pytest.raises(ValueError):
        B.grad_clip([g[0].cpu()], 1.0, ws)
    with pytest.raises(ValueError):
        B.grad_clip(g, 1.0, ws, outs=g[:1])
    with pytest.raises(ValueError):
        B.grad_clip(g, 1.0, ws, outs=[g[0], g[1][:32]])
    for max_norm in (-1.0, float("nan")):
        with pytest.raises(B.BoostError):
            B.grad_clip(g, max_norm, ws)
    with pytest.raises(B.BoostError):                   # the same tensor twice, in place
        B.grad_clip([g[0], g[0]], 1.0, ws)
    assert B.grad_clip([g[0], g[0]], None, ws).item() > 0
    with pytest.raises(B.BoostError):                   # an output over another's gradient
        B.grad_clip(g, 1.0, ws, outs=[g[1], torch.empty_like(g[1])])
    with pytest.raises(B.BoostError):
        B.grad_clip([g[0][1:]], 1.0, ws)                # not 16-byte aligned
    with pytest.raises(B.BoostError):
        B.grad_clip(g, 1.0, B.Workspace(256))


@pytest.mark.parametrize("big", [1e-44, 1e-30, 1e-20, 1e19, 1e25, 3e36])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_gradients_whose_squares_leave_fp32(dtype, big, ws):
    """Their squares in fp64, every rounding below NORM; beside zeros, and in ragged tensors. (The
    norm of 17269 values of 3e36 is 131 times that, 3.9e38, which rounds to fp32's infinity; what
    scales is the fp64 norm.)"""
    g = make([8192, 9000, 77], [dtype] * 3, seed=8, std=1.0)
    g = [(t.double() * big).to(dtype) for t in g] + [torch.zeros(20000, dtype=dtype, device="cuda")]
    before = [t.clone() for t in g]
    norm = B.grad_clip(g, None, ws)
    want, _ = ops.grad_clip([f64(t) for t in before], float("inf"))
    if want > torch.finfo(torch.float32).max:
        assert norm.item() == float("inf")
    else:
        assert abs(norm.item() - want) <= (NORM + 2.0 ** -24) * want + 2.0 ** -149
    if big >= 1e19:
        assert torch.equal(B.grad_clip(g, 0.5 * want, ws), norm)
        compare(g, torch.tensor(want, dtype=torch.float64), before, 0.5 * want)
