"""Which dropout masks a layer's branches use: those of layers with other seeds are others."""

import itertools

import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod
from rank_bottleneck_online_gb300 import inputs
from rank_bottleneck_online_gb300.block import Layer

from ops_parity import normal

pytestmark = pytest.mark.gpu

T, D, R = 16, 64, 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def make(seed):
    """A layer whose branches dwarf the residual they are added to, so that a kept element
    differs from the residual and a dropped one is it."""
    w = inputs.make_layer(T, D, R, D, seed=3)
    w["p"]["B_o"] = w["p"]["B_o"] * 2.0 ** 30
    w["p"]["B_dn"] = w["p"]["B_dn"] * 2.0 ** 60
    return w, Layer(T, D, R, D, weights=w["p"], dropout=0.5, seed=seed)


def masks(seed, mask=0):
    """The two branches' masks in the forward, after a check of the backward's."""
    w, layer = make(seed)
    x, dout, dq, dk = (w[k].cuda() for k in ("x", "dout", "dq", "dk"))
    layer.forward(x, mask=mask)
    attention, mlp = layer.x1 != x, layer.out != layer.x1
    layer.backward(x, dout, dq, dk, mask=mask)
    B.check(layer.qkv.ws)
    # the O block's upstream gradient is the last that went through a mask
    assert torch.equal(layer.dbranch != 0, attention)
    got = [t.clone() for t in (layer.mlp.gu.dx, layer.mlp.dn.dA, layer.mlp.dn.dB)]
    layer.mlp.backward(layer.x1, torch.where(mlp, 2 * dout, torch.zeros_like(dout)), dx_residual=dout)
    for a, b in zip(got, (layer.mlp.gu.dx, layer.mlp.dn.dA, layer.mlp.dn.dB)):
        assert torch.equal(a, b)
    return attention, mlp


def test_seeds_and_branches_share_no_mask():
    seeds = [0, 1, 2, 3, 76, 77, 78, (1 << 63) - 1, 1 << 63, (1 << 64) - 2, (1 << 64) - 1]
    found = [(s, which, m) for s in seeds for which, m in enumerate(masks(s))]
    for (s, i, a), (t, j, b) in itertools.combinations(found, 2):
        # 1024 draws of a half: five standard deviations are 0.08
        assert abs((a == b).double().mean().item() - 0.5) < 0.08, (s, i, t, j)


def test_same_words_same_masks_and_other_words_others():
    a, b = masks(4, 9), masks(4, 9)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    for other in (masks(4, 10), masks(4, (1 << 63) - 1)):
        assert not any(torch.equal(p, q) for p, q in zip(a, other))


def test_refuses_masks_beyond_63_bits():
    w, layer = make(1)
    for mask in (-1, 1 << 63):
        with pytest.raises(ValueError):
            layer.forward(w["x"].cuda(), mask=mask)
        with pytest.raises(ValueError):
            layer.backward(*(w[k].cuda() for k in ("x", "dout", "dq", "dk")), mask=mask)


def test_dropout_of_nothing_is_a_plain_add():
    a, b = normal(1, 300, 72), normal(2, 300, 72)
    assert torch.equal(B.dropout_add(a, 0.0, 5, residual=b), B.add(a, b))
    assert torch.equal(B.dropout_add(a, 0.0, 5), a)
