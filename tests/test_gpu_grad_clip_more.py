"""Gradient clipping with more tensors than a launch's table holds, and tensors that only count:
results and launches. Tolerances: test_gpu_grad_clip."""

import numpy as np
import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF, f64

pytestmark = pytest.mark.gpu

NORM = 2.0 ** -20
TABLE = 1100                            # tensors of one launch


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


@pytest.fixture(scope="module")
def ws():
    return B.Workspace(B.grad_clip_workspace_bytes())


def make(count, seed, most=3000):
    """`count` gradients of 1 to `most` values and, not counted, one empty one for each 100."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    sizes = [int(n) for n in rng.integers(1, most, count)]
    for at in range(0, count, 100):
        sizes.insert(at, 0)
    return [(torch.randn(n, generator=g) * 0.1).to((BF, torch.float32)[i % 2]).cuda()
            for i, n in enumerate(sizes)]


def compare(got, before, norm, want_norm, want):
    assert abs(norm.item() - want_norm) <= (NORM + 2.0 ** -24) * want_norm
    for a, g, w in zip(got, before, want):
        half = torch.finfo(g.dtype).eps / 2
        assert (np.abs(f64(a) - w) <= (half + 2 * NORM) * np.abs(w)).all()


@pytest.fixture
def kernels():
    """How many kernels clipping has launched since it was asked last."""
    def count():
        n = B.profile_kernels().get("grad_clip", 0)
        B.profile_enable(True)          # (counts from 0 again)
        return n

    B.profile_enable(True)
    yield count
    B.profile_enable(False)


@pytest.mark.parametrize("count", [TABLE, TABLE + 1, 2 * TABLE, 2 * TABLE + 1, 3 * TABLE + 7])
def test_several_launches(count, ws, kernels):
    grads = make(count, count)
    before = [t.clone() for t in grads]
    launches = -(-count // TABLE)
    norm = B.grad_clip(grads, 1.0, ws)
    assert kernels() == 2 * launches
    compare(grads, before, norm, *ops.grad_clip([f64(t) for t in before], 1.0))
    # the same bits, and no scaling: one launch more for the norm
    again = [t.clone() for t in before]
    assert torch.equal(norm, B.grad_clip(again, None, ws))
    assert kernels() == launches + 1
    for a, b in zip(again, before):
        assert torch.equal(a, b)


def test_launches_of_tensors_that_only_count(ws, kernels):
    """Of three launches the first, or the middle one, or the last, or two of them, scale nothing; of
    the others every third tensor."""
    count = 3 * TABLE
    grads = make(count, 1)
    full = [t for t in grads if t.numel()]
    want_norm, want = ops.grad_clip([f64(t) for t in grads], 1.0)
    norm = torch.empty(1, device="cuda")
    for idle in ((0,), (1,), (2,), (0, 1), (1, 2), (0, 2)):
        outs = [None if t.numel() and (full_at // TABLE in idle or full_at % 3 == 0)
                else torch.full_like(t, -7.25)
                for t, full_at in zip(grads, np.cumsum([t.numel() > 0 for t in grads]) - 1)]
        table = (B.Grad * len(grads))()
        for i, (t, o) in enumerate(zip(grads, outs)):
            table[i] = (t.data_ptr(), None if o is None else o.data_ptr(), t.numel(),
                        int(t.dtype == torch.float32))
        norm.fill_(-1.0)
        before = [t.clone() for t in grads]
        assert B.lib().boost_grad_clip(len(grads), table, 1.0, norm.data_ptr(), ws.ptr, ws.nbytes,
                                       torch.cuda.current_stream().cuda_stream) == 0
        # (the first launch of the tables has the norm, whether it scales or not)
        assert kernels() == 3 + len({0, 1, 2} - set(idle) | {0})
        for a, b in zip(grads, before):
            assert torch.equal(a, b)
        kept = [(o, t, w) for o, t, w in zip(outs, grads, want) if o is not None]
        compare(*(list(x) for x in zip(*((o, t) for o, t, _ in kept))), norm, want_norm,
                [w for _, _, w in kept])


def test_nothing_to_launch(ws, kernels):
    assert B.grad_clip([torch.empty(0, dtype=BF, device="cuda")], 1.0, ws).item() == 0
    assert kernels() == 0
