"""The layer's rotary positions called by themselves: what they return."""

import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod
from rank_bottleneck_online_gb300.block import Rotary

from ops_parity import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


@pytest.mark.parametrize("T", [0, 1, 37])
@pytest.mark.parametrize("with_k", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_returns_what_it_turned(T, with_k, inverse):
    """Without outputs it returns new tensors [T, heads * dim], given outputs themselves."""
    rotary = Rotary(32, rot=16, interleaved=True)
    q, k = normal(1, T, 128), normal(2, T, 64) if with_k else None
    pos = torch.arange(5, 5 + T, dtype=torch.int32, device="cuda")
    want_q, want_k = B.rope(q.view(T, 4, 32), k.view(T, 2, 32) if with_k else None, pos,
                            rotary.inv_freq, interleaved=True, inverse=inverse)
    before = q.clone()
    got_q, got_k = rotary(q, k, pos, inverse=inverse)
    assert got_q.shape == q.shape and torch.equal(got_q, want_q.flatten(1))
    assert torch.equal(q, before)
    if with_k:
        assert got_k.shape == k.shape and torch.equal(got_k, want_k.flatten(1))
    else:
        assert got_k is None
    out = torch.empty_like(q)
    again, other = rotary(q, k, pos, inverse=inverse, q_out=out)
    assert again is out and torch.equal(out, got_q)
    assert other is None if k is None else torch.equal(other, got_k)
    same, _ = rotary(q, k, pos, inverse=inverse, q_out=q, k_out=k)      # in place
    assert same is q and torch.equal(q, got_q) and (k is None or torch.equal(k, got_k))


def test_slices_of_a_packed_projection():
    rotary = Rotary(32)
    whole = normal(3, 20, 256)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    want = rotary(whole[:, :128].contiguous(), whole[:, 128:192].contiguous(), pos)
    got = rotary(whole[:, :128], whole[:, 128:192], pos)
    assert all(a.shape == b.shape and torch.equal(a, b) for a, b in zip(got, want))


def test_heads_given_apart():
    rotary = Rotary(32)
    q, k = normal(4, 20, 4, 32), normal(5, 20, 2, 32)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    got = rotary(q, k, pos)
    want = rotary(q.flatten(1), k.flatten(1), pos)
    assert got[0].shape == q.shape and got[1].shape == k.shape
    assert all(torch.equal(a.flatten(1), b) for a, b in zip(got, want))
    out = torch.empty(20, 128, dtype=q.dtype, device="cuda")
    assert rotary(q, None, pos, q_out=out)[0] is out and torch.equal(out, want[0])
