"""Layers with their attention cores: several of one model, and beside one without a core."""

import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod
from rank_bottleneck_online_gb300 import inputs
from rank_bottleneck_online_gb300.block import Attention, Layer, Rotary

pytestmark = pytest.mark.gpu

T, D, R, FFN, HEADS = 200, 128, 64, 136, 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def core(**kw):
    return Attention(T, HEADS, D // HEADS, **kw)


def grads(layer):
    return [layer.dx, layer.dqkv, *layer.weight_grads()]


def test_two_layers_given_one_core():
    """Forward through both, back through both: as with a core each."""
    ws = [inputs.make_layer(T, D, R, FFN, seed=s) for s in (1, 2)]
    x, dout = (ws[0][n].cuda() for n in ("x", "dout"))
    starts = torch.tensor([0, 77, T], dtype=torch.int32, device="cuda")

    def step(cores):
        layers = [Layer(T, D, R, FFN, S=2, weights=w["p"], attention=c) for w, c in zip(ws, cores)]
        h = layers[0].forward(x, starts=starts)
        out = layers[1].forward(h, starts=starts).clone()
        d = layers[1].backward(h, dout, starts=starts)
        layers[0].backward(x, d, starts=starts)
        for layer in layers:
            B.check(layer.qkv.ws)
        return [out, *grads(layers[0]), *grads(layers[1])], layers

    want, _ = step([core(sequences=2), core(sequences=2)])
    one = core(sequences=2)
    got, layers = step([one, one])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert layers[0].attention is one               # whose result its owner reads there
    assert layers[1].attention.out.data_ptr() != one.out.data_ptr()


def test_a_core_of_other_settings_is_made_alike():
    one = core(causal=False, scale=0.3, sequences=5)
    w = inputs.make_layer(T, D, R, FFN, seed=3)
    layers = [Layer(T, D, R, FFN, weights=w["p"], attention=one) for _ in range(2)]
    assert len({id(layer.attention) for layer in layers}) == 2
    other = layers[1].attention
    for name in ("T", "heads", "dim", "causal", "scale", "sequences", "workspace_bytes"):
        assert getattr(other, name) == getattr(one, name), name


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("rotary", [True, False])
def test_sequences_of_one_token_are_the_layer_without_a_core(rotary, p):
    """The softmax of a single key is 1: the core gives v, and 0 for the gradients of q and k. So a
    layer without a core, given those gradients, makes the same step, bit for bit."""
    w = inputs.make_layer(T, D, R, FFN, seed=4)
    x, dout = (w[n].cuda() for n in ("x", "dout"))
    kw = dict(S=2, weights=w["p"], dropout=p, seed=9, rotary=Rotary(D // HEADS) if rotary else None)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") if rotary else None
    with_core = Layer(T, D, R, FFN, attention=core(sequences=T), **kw)
    without = Layer(T, D, R, FFN, **kw)
    starts = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    with_core.forward(x, positions=pos, starts=starts, mask=3)
    without.forward(x, positions=pos, mask=3)
    assert torch.equal(with_core.attention.out, without.qkv.y[2])
    assert torch.equal(with_core.x1, without.x1) and torch.equal(with_core.out, without.out)
    with_core.backward(x, dout, positions=pos, starts=starts, mask=3)
    zeros = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    without.backward(x, dout, zeros, zeros.clone(), positions=pos, mask=3)
    for layer in (with_core, without):
        B.check(layer.qkv.ws)
    assert (with_core.dqkv[:2] == 0).all() and torch.equal(with_core.dqkv[2], with_core.dattention)
    for a, b in zip(grads(with_core), grads(without)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("p", [0.0, 0.2])
def test_the_cores_gradients_given_to_a_layer_without_one(p):
    """The gradients that a core makes of q and k, given to a layer without one: its QKV block sees
    them as they are, and its v's from O's backward, whatever the core's layer did with v."""
    w = inputs.make_layer(T, D, R, FFN, seed=5)
    x, dout = (w[n].cuda() for n in ("x", "dout"))
    kw = dict(S=2, weights=w["p"], dropout=p, seed=9)
    with_core, without = Layer(T, D, R, FFN, attention=core(), **kw), Layer(T, D, R, FFN, **kw)
    with_core.forward(x)
    with_core.backward(x, dout)
    dq, dk, dv = (t.clone() for t in with_core.dqkv)
    without.forward(x)
    without.backward(x, dout, dq, dk)
    for layer in (with_core, without):
        B.check(layer.qkv.ws)
    assert torch.equal(without.dqkv[0], dq) and torch.equal(without.dqkv[1], dk)
    assert not torch.equal(without.dqkv[2], dv)
    # the same gradients sent into the QKV block give the same, whichever layer it is of
    dx1 = with_core.dx1.clone()
    want = [t.clone() for t in (with_core.dx, *with_core.qkv.weight_grads())]
    without.qkv.backward(x, with_core.dqkv, dx_residual=dx1)
    for a, b in zip((without.dx, *without.qkv.weight_grads()), want):
        assert torch.equal(a, b)
