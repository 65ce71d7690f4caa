"""A layer with its attention core, as a training step runs it: QKV, rotary positions, attention
over packed sequences, O, dropout, MLP, all backward, and the gradients clipped; against the
oracle's composition, and captured into a replayed graph. An 8-bit layer with the fused norm.

The composition is checked stage by stage on the GPU's own intermediates: what a rounding of a
probability makes of a gradient is bounded by the magnitudes that the gradient's sum adds up
(attention_parity), many times its own where they cancel, and not by the gradient.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod
from rank_bottleneck_online_gb300 import inputs
from rank_bottleneck_online_gb300.block import (MLP, Attention, Block, Layer, Rotary, SVDPair,
                                                clip_gradients)

from attention_parity import SLACK
from ops_parity import HALF_STEP, close, f64, normal
from parity import assert_close

pytestmark = pytest.mark.gpu

R = oracle.to_bf16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def masks(shape, p, seed, offset):
    keep = ops.dropout_keep(range(int(np.prod(shape))), p, seed, offset).reshape(shape)
    return keep * 65536 / (65536 - ops.dropout_drop(p))


def check_step(layer, w, pos, p, seed, mask, lengths, causal, S=2):
    """Every stage of the step that `layer` has just made."""
    P = {k: inputs.as_f64(v) for k, v in w["p"].items()}
    x, dout = (inputs.as_f64(w[k]) for k in ("x", "dout"))
    T, d = x.shape
    rotary, heads = layer.rotary, layer.attention.heads
    freq, axis = f64(rotary.inv_freq), np.zeros(rotary.inv_freq.numel(), dtype=int)
    pairs = [(n, n) for n in lengths]

    def split(t):
        return t.reshape(T, heads, d // heads)

    def turn(t, inverse):
        return ops.rope(split(t), pos, freq, axis, rotary.interleaved, inverse)

    w0, w1 = (masks((T, d), p, seed + i, mask) if p else 1.0 for i in (0, 1))
    # into the core
    qkv = R(oracle.block_fwd(x, P["gamma1"], P["A_qkv"], P["B_qkv"], S=S, flow="bf16")[0])
    q, k, v = (split(f64(t)) for t in layer.qkv.y)
    assert_close("q", q, R(turn(qkv[0], False)))
    assert_close("k", k, R(turn(qkv[1], False)))
    assert_close("v", v, split(qkv[2]))
    # the core, from its own q, k, v and upstream gradient
    core = ops.attention(q, k, v, pairs, causal, dout=split(f64(layer.dattention)))
    close(split_t(layer.attention.out, heads), core["out"], SLACK * core["out_size"])
    # behind it, from its own out; the MLP from its own input, O's backward from its own upstream
    # gradient
    o = f64(layer.attention.out)
    yo = oracle.block_fwd(o, None, P["A_o"], P["B_o"], has_norm=False, flow="bf16")[0][0]
    want_x1 = x + R(yo) * w0 if p else x + yo
    x1 = f64(layer.x1)
    mlp = (P["gamma2"], P["A_gu"], P["B_gu"], P["A_dn"], P["B_dn"])
    m, _ = oracle.mlp_fwd(x1, *mlp, S=S)
    gm = oracle.mlp_bwd(x1, *mlp, R(dout * w1), S=S)
    dx1 = f64(layer.dx1)
    go = oracle.block_bwd(o, None, P["A_o"], P["B_o"], R(dx1 * w0)[None], has_norm=False, flow="bf16")
    want = {"x1": want_x1, "out": x1 + R(m) * w1 if p else x1 + m, "dattention": go["dx"],
            "dx1": dout + (R(gm["dx"]) if p else gm["dx"]),
            "dA_o": go["dA"], "dB_o": go["dB"], "dA_gu": gm["dA1"], "dB_gu": gm["dB1"],
            "dA_dn": gm["dA2"], "dB_dn": gm["dB2"]}
    # its gradients; those of q and k are rounded and then turned back: both values of a pair
    # bring what they are off by
    for i, name in enumerate(("dq", "dk", "dv")):
        slack = SLACK * core[f"{name}_size"]
        exact = core[name]
        if name != "dv":
            slack = slack + HALF_STEP * (np.abs(exact) + slack)
            half = slack.shape[-1] // 2
            slack = np.tile(slack[..., :half] + slack[..., half:], 2)
            exact = turn(exact, True)
        close(split_t(layer.dqkv[i], heads), exact, slack)
    # and out of it, from its own gradients
    gq = oracle.block_bwd(x, P["gamma1"], P["A_qkv"], P["B_qkv"], f64(layer.dqkv), S=S, flow="bf16")
    want |= {"dx": dx1 + R(gq["dx"]), "dA_qkv": gq["dA"], "dB_qkv": gq["dB"], "dgamma1": gq["dgamma"]}
    got = results(layer)
    for key in want:
        assert_close(key, got[key], want[key])


def split_t(t, heads):
    return t.view(t.shape[0], heads, -1)


def make(T=200, d=128, r=64, ffn=136, heads=2, *, p=0.0, causal=True, sequences=3, seed=5, **kw):
    w = inputs.make_layer(T, d, r, ffn, seed=seed)
    rotary = Rotary(d // heads)
    attention = Attention(T, heads, d // heads, causal=causal, sequences=sequences)
    layer = Layer(T, d, r, ffn, S=2, weights=w["p"], rotary=rotary, attention=attention, dropout=p,
                  seed=77, **kw)
    pos = np.arange(T)[None] % 77
    return w, layer, rotary, pos, torch.from_numpy(pos[0]).int().cuda()


def bounds(lengths):
    return torch.tensor([0, *np.cumsum(lengths)], dtype=torch.int32, device="cuda")


def results(layer):
    return {"attention": layer.attention.out, "x1": layer.x1, "out": layer.out, "dqkv": layer.dqkv,
            "dx": layer.dx, "dA_qkv": layer.qkv.dA, "dB_qkv": layer.qkv.dB,
            "dgamma1": layer.qkv.dgamma, "dA_o": layer.o.dA, "dB_o": layer.o.dB,
            "dA_gu": layer.mlp.gu.dA, "dB_gu": layer.mlp.gu.dB, "dA_dn": layer.mlp.dn.dA,
            "dB_dn": layer.mlp.dn.dB, "dattention": layer.dattention, "dx1": layer.dx1}


def step(layer, w, pos, starts=None, **kw):
    x, dout = (w[k].cuda() for k in ("x", "dout"))
    layer.forward(x, positions=pos, starts=starts, **kw)
    layer.backward(x, dout, positions=pos, starts=starts, **kw)
    for blk in (layer.qkv, layer.o, layer.mlp.gu, layer.mlp.dn):
        B.check(blk.ws)


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", [None, [77, 123], [1, 130, 69]])
def test_layer_step(lengths, causal, p):
    w, layer, rotary, pos, gpos = make(p=p, causal=causal)
    step(layer, w, gpos, None if lengths is None else bounds(lengths), mask=3)
    check_step(layer, w, pos, p, 77, 3, lengths or [200], causal)


def test_step_of_several_tiles_and_clipped_gradients():
    w, layer, rotary, pos, gpos = make(T=700, d=256, r=64, ffn=264, heads=2)
    starts = bounds([600, 100])
    step(layer, w, gpos, starts)
    check_step(layer, w, pos, 0.0, 77, 0, [600, 100], True)
    got = {k: v.clone() for k, v in results(layer).items()}
    before = [t.clone() for t in layer.weight_grads()]
    assert len(before) == 10                            # A and B of four blocks, two gammas
    ws = B.Workspace(B.grad_clip_workspace_bytes())
    norm = clip_gradients([layer], 0.5, ws)
    want_norm, scaled = ops.grad_clip([f64(t) for t in before], 0.5)
    assert abs(norm.item() - want_norm) <= 2.0 ** -19 * want_norm
    for t, s in zip(layer.weight_grads(), scaled):
        assert (np.abs(f64(t) - s) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(s)).all()
    assert torch.equal(layer.dx, got["dx"])             # not a weight's


def test_captured_step_with_clipping_takes_new_sequences():
    w, layer, _, _, gpos = make(p=0.1)
    x, dout = (w[k].cuda() for k in ("x", "dout"))
    starts = bounds([77, 123, 0])
    ws = B.Workspace(B.grad_clip_workspace_bytes())
    norm = torch.empty(1, device="cuda")

    def whole():
        layer.forward(x, positions=gpos, starts=starts, mask=2)
        layer.backward(x, dout, positions=gpos, starts=starts, mask=2)
        clip_gradients([layer], 1.0, ws, norm=norm)

    whole()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole()
    for lengths in ([77, 123, 0], [10, 20, 170], [200, 0, 0]):
        starts.copy_(bounds(lengths))
        graph.replay()
        got = [t.clone() for t in (*results(layer).values(), norm)]
        whole()
        for a, b in zip(got, (*results(layer).values(), norm)):
            assert torch.equal(a, b)
    for ws in (layer.qkv.ws, layer.mlp.dn.ws):
        B.check(ws)


def test_layer_without_the_core_is_unchanged():
    """The attention core's gradients from outside: what the layer with a core sends into its QKV
    block, given to one without, gives the same, bit for bit, where O works on the same."""
    w, layer, rotary, pos, gpos = make()
    x, dout = (w[k].cuda() for k in ("x", "dout"))
    plain = Layer(200, 128, 64, 136, S=2, weights=w["p"])
    plain.forward(x)
    plain.backward(x, dout, w["dq"].cuda(), w["dk"].cuda())
    again = Layer(200, 128, 64, 136, S=2, weights=w["p"])
    again.forward(x)
    again.backward(x, dout, w["dq"].cuda(), w["dk"].cuda())
    assert torch.equal(plain.dx, again.dx) and torch.equal(plain.out, again.out)
    for bad in (dict(dq=w["dq"].cuda(), dk=w["dk"].cuda()),):
        layer.forward(x, positions=gpos)
        with pytest.raises(ValueError):
            layer.backward(x, dout, positions=gpos, **bad)
    with pytest.raises(ValueError):
        plain.backward(x, dout)
    with pytest.raises(ValueError):
        plain.forward(x, starts=bounds([200]))
    with pytest.raises(ValueError):
        Layer(200, 128, 64, 136, weights=w["p"], attention=Attention(100, 2, 64))
    with pytest.raises(ValueError):
        Layer(200, 128, 64, 136, weights=w["p"], fused_norm=True)
    with pytest.raises(ValueError):
        MLP(200, 128, 64, 136, weights=inputs.make_mlp(200, 128, 64, 136)).forward(x, add=x)


@pytest.mark.parametrize("p", [0.0, 0.2])
def test_8_bit_layer_with_the_fused_norm(p):
    """One reading of each norm's input in the place of three: the sum and the operands are the
    same bits, the row scales the same up to the order of their sums."""
    kw = dict(p=p, fp8=True)
    w, plain, _, _, gpos = make(**kw)
    _, fused, *_ = make(fused_norm=True, **kw)
    step(plain, w, gpos)
    step(fused, w, gpos)
    assert torch.equal(plain.qkv.x8[0].view(torch.uint8), fused.qkv.x8[0].view(torch.uint8))
    assert torch.equal(plain.qkv.x8[1], fused.qkv.x8[1])
    np.testing.assert_allclose(f64(plain.qkv.rstd), f64(fused.qkv.rstd), rtol=1e-6)
    a, b = results(plain), results(fused)
    for key in a:
        # a row scale off by 2^-22 turns a rounding here and there, an 8-bit one by 2^-3 of its value
        g, e = f64(b[key]), f64(a[key])
        assert np.linalg.norm(g - e) <= 0.02 * np.linalg.norm(e), key
    x1 = f64(fused.x1)
    np.testing.assert_allclose(f64(fused.mlp.gu.rstd), ops.row_scale(x1, 1e-5), rtol=1e-5)


def test_clipping_over_several_kinds_of_workload():
    blk = Block(64, 64, 64, 2, 64, weights=inputs.make_block(64, 64, 64, 2, 64, seed=1))
    pw = inputs.make_svd_pair(64, 64, 64, 72, seed=2)
    pair = SVDPair(64, 64, 64, 72, weights=pw["p"])
    x = normal(3, 64, 64)
    blk.forward(x)
    blk.backward(x, normal(4, 2, 64, 64))
    pair.forward(x)
    pair.backward(x, normal(5, 3, 64, 64), normal(6, 2, 64, 72))
    grads = [f64(t) for w in (blk, pair) for t in w.weight_grads()]
    assert len(grads) == 9
    blk.ws.ensure(B.grad_clip_workspace_bytes())
    norm = clip_gradients([blk, pair], None, blk.ws)
    assert abs(norm.item() - ops.grad_clip(grads, 1.0)[0]) <= 2.0 ** -19 * norm.item()
    for t, g in zip([t for w in (blk, pair) for t in w.weight_grads()], grads):
        assert np.array_equal(f64(t), g)
