"""The operators around the block together, as a training step of the layer uses them: rotary
positions on q and k, dropout on both residual branches, 8-bit products; against the
oracle's composition, and captured into a replayed graph.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod
from rank_bottleneck_online_gb300 import inputs
from rank_bottleneck_online_gb300.block import MLP, Fp8Block, Layer, Rotary

from ops_parity import close, f64, normal
from parity import assert_close, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def masks(shape, p, seed, offset):
    keep = ops.dropout_keep(range(int(np.prod(shape))), p, seed, offset).reshape(shape)
    return keep * 65536 / (65536 - ops.dropout_drop(p))


def layer_oracle(w, heads, rotary, pos, p, seed, mask, S):
    """Forward and gradients of the layer with rotary positions and dropout, in the oracle's
    bf16 flow."""
    R = oracle.to_bf16
    P = {k: inputs.as_f64(v) for k, v in w["p"].items()}
    x, dout, dq, dk = (inputs.as_f64(w[k]) for k in ("x", "dout", "dq", "dk"))
    T, d = x.shape
    pairs = rotary.inv_freq.numel()
    axis = np.repeat(np.arange(len(rotary.sections)), rotary.sections)
    freq = f64(rotary.inv_freq)

    def turn(t, inverse):
        t = t.reshape(T, heads, d // heads)
        return R(ops.rope(t, pos, freq, axis, rotary.interleaved, inverse)).reshape(T, d)

    assert pairs == len(axis)
    w0, w1 = (masks((T, d), p, seed + i, mask) for i in (0, 1))
    yq, _ = oracle.block_fwd(x, P["gamma1"], P["A_qkv"], P["B_qkv"], S=S, flow="bf16")
    qkv = R(yq)
    yo, _ = oracle.block_fwd(qkv[2], None, P["A_o"], P["B_o"], has_norm=False, flow="bf16")
    x1 = R(x + R(yo[0]) * w0)
    mlp = (P["gamma2"], P["A_gu"], P["B_gu"], P["A_dn"], P["B_dn"])
    m, _ = oracle.mlp_fwd(x1, *mlp, S=S)
    out = x1 + R(m) * w1
    gm = oracle.mlp_bwd(x1, *mlp, R(dout * w1), S=S)
    dx1 = R(dout + R(gm["dx"]))
    go = oracle.block_bwd(qkv[2], None, P["A_o"], P["B_o"], R(dx1 * w0)[None], has_norm=False,
                          flow="bf16")
    dqkv = np.stack([turn(dq, True), turn(dk, True), R(go["dx"])])
    gq = oracle.block_bwd(x, P["gamma1"], P["A_qkv"], P["B_qkv"], dqkv, S=S, flow="bf16")
    return ({"q": turn(qkv[0], False), "k": turn(qkv[1], False), "v": qkv[2], "x1": x1, "out": out},
            {"dx": dx1 + R(gq["dx"]), "dA_qkv": gq["dA"], "dB_qkv": gq["dB"],
             "dgamma1": gq["dgamma"], "dA_o": go["dA"], "dB_o": go["dB"], "dA_gu": gm["dA1"],
             "dB_gu": gm["dB1"], "dA_dn": gm["dA2"], "dB_dn": gm["dB2"]})


def make_layer(T=200, d=128, r=64, ffn=136, *, fp8=False, interleaved=False, p=0.2, seed=5):
    w = inputs.make_layer(T, d, r, ffn, seed=seed)
    rotary = Rotary(32, sections=[4, 12], interleaved=interleaved)
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, 5000, (2, T))
    layer = Layer(T, d, r, ffn, S=2, weights=w["p"], rotary=rotary, dropout=p, seed=77, fp8=fp8)
    return w, layer, rotary, pos, torch.from_numpy(pos).int().cuda()


def step(layer, w, pos, **kw):
    x, dout, dq, dk = (w[k].cuda() for k in ("x", "dout", "dq", "dk"))
    layer.forward(x, positions=pos, **kw)
    layer.backward(x, dout, dq, dk, positions=pos, **kw)
    for blk in (layer.qkv, layer.o, layer.mlp.gu, layer.mlp.dn):
        B.check(blk.ws)


def results(layer):
    return {"q": layer.qkv.y[0], "k": layer.qkv.y[1], "v": layer.qkv.y[2], "x1": layer.x1,
            "out": layer.out, "dx": layer.dx, "dA_qkv": layer.qkv.dA, "dB_qkv": layer.qkv.dB,
            "dgamma1": layer.qkv.dgamma, "dA_o": layer.o.dA, "dB_o": layer.o.dB,
            "dA_gu": layer.mlp.gu.dA, "dB_gu": layer.mlp.gu.dB, "dA_dn": layer.mlp.dn.dA,
            "dB_dn": layer.mlp.dn.dB}


@pytest.mark.parametrize("interleaved", [False, True])
def test_layer_step_with_rotary_and_dropout(interleaved):
    w, layer, rotary, pos, gpos = make_layer(interleaved=interleaved)
    step(layer, w, gpos, mask=3)
    fwd, grads = layer_oracle(w, 4, rotary, pos, 0.2, 77, 3, 2)
    got = results(layer)
    for k, v in {**fwd, **grads}.items():
        assert_close(k, got[k], v)


def test_layer_without_them_is_unchanged():
    """No rotation and no dropout: the layer of before, bit for bit; a rotation by nothing and
    dropout of nothing give it too, up to the roundings of separate adds."""
    w, layer, rotary, pos, gpos = make_layer(p=0.0)
    plain = Layer(200, 128, 64, 136, S=2, weights=w["p"])
    x, dout, dq, dk = (w[k].cuda() for k in ("x", "dout", "dq", "dk"))
    plain.forward(x)
    plain.backward(x, dout, dq, dk)
    layer.rotary = None
    step(layer, w, None)
    a, b = results(plain), results(layer)
    assert all(torch.equal(a[k], b[k]) for k in a)
    layer.rotary = rotary
    step(layer, w, torch.zeros_like(gpos))
    c = results(layer)
    assert all(torch.equal(a[k], c[k]) for k in a)


def test_captured_layer_step_takes_a_new_mask_each_time():
    w, layer, rotary, pos, gpos = make_layer()
    x, dout, dq, dk = (w[k].cuda() for k in ("x", "dout", "dq", "dk"))
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    step(layer, w, gpos)                                # first use outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, positions=gpos, counter=counter)
        layer.backward(x, dout, dq, dk, positions=gpos, counter=counter)
        counter.add_(1)
    seen = []
    for at in range(3):
        graph.replay()
        got = {k: v.clone() for k, v in results(layer).items()}
        step(layer, w, gpos, mask=at)
        want = results(layer)
        assert all(torch.equal(got[k], want[k]) for k in got)
        seen.append(got["out"])
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


@pytest.mark.parametrize("T,d,r,k,n,norm,act", [(200, 264, 136, 3, 264, True, "silu"),
                                               (1, 512, 256, 2, 520, True, "silu"),
                                               (130, 128, 64, 1, 136, False, "identity")])
def test_fp8_block_forward(T, d, r, k, n, norm, act):
    """Stage by stage on the GPU's own intermediates, whose 8-bit roundings the oracle then
    repeats exactly: a = act(s x8 A8), y = a8 B8."""
    w = inputs.make_block(T, d, r, k, n, has_norm=norm, seed=8)
    blk = Fp8Block(T, d, r, k, n, S=2 if norm else 1, has_norm=norm, act=act, weights=w)
    y = blk.forward(w["x"].cuda())
    B.check(blk.ws8)

    def values(t, rows):
        return ops.fp8_dequantize(*ops.fp8_quantize(t, "e4m3", rows))

    A = inputs.as_f64(w["A"])
    if norm:
        A = oracle.to_bf16(inputs.as_f64(w["gamma"])[:, None] * A)
        _, rstd = oracle.rmsnorm_stats(inputs.as_f64(w["x"]), 2, 1e-5)
        np.testing.assert_allclose(to_np(blk.rstd), rstd, rtol=1e-5)
    rs = to_np(blk.rstd) if norm else None
    a, size = ops.fp8_matmul(values(inputs.as_f64(w["x"]), 1), values(A.T, 128), rs, act)
    # the product's bound: (K / 32 + 32) additions of 2^-23 of the summed magnitudes each, and
    # 2^-20 of the value for the fast logistic
    close(blk.a, a, (d / 32 + 32) * 2.0 ** -23 * 1.1 * size + 2.0 ** -20 * np.abs(a))
    ga = f64(blk.a)
    for g in range(k):
        want, size = ops.fp8_matmul(values(ga[:, g * r:(g + 1) * r], 1),
                                    values(inputs.as_f64(w["B"])[g].T, 128))
        close(y[g], want, (r / 32 + 32) * 2.0 ** -23 * size)


def test_fp8_block_takes_updated_weights():
    w = inputs.make_block(64, 128, 128, 1, 128, seed=9)
    blk = Fp8Block(64, 128, 128, 1, 128, weights=w)
    x = w["x"].cuda()
    before = blk.forward(x).clone()
    blk.B.mul_(2.0)                                     # exact in both formats
    assert torch.equal(blk.forward(x), before)          # until they are taken again
    blk.quantize_weights()
    assert torch.equal(blk.forward(x), 2 * before)


def test_fp8_layer_step():
    """The layer's step with every forward product in 8 bits, rotary positions and dropout:
    near the bf16 layer's. An 8-bit operand is off by at most half a step of 2^-3, so by a
    uniform error of rms 2^-4 / sqrt(3) of its value at most; a block multiplies four operands
    like that, and three such blocks follow one another on the way to out:
    sqrt(3 * 4) 2^-4 / sqrt(3) < 0.13 of the branches, which dropout scales but leaves in
    proportion."""
    w, layer, rotary, pos, gpos = make_layer(fp8=True)
    w2, plain, *_ = make_layer()
    step(layer, w, gpos, mask=1)
    step(plain, w2, gpos, mask=1)
    got, want = results(layer), results(plain)
    for key in ("q", "k", "v", "x1", "out"):
        g, e = f64(got[key]), f64(want[key])
        assert np.linalg.norm(g - e) <= 0.13 * np.linalg.norm(e), key
    assert all(torch.isfinite(v).all() for v in got.values())
    for blk in (layer.qkv, layer.o, layer.mlp.gu, layer.mlp.dn):
        B.check(blk.ws8)


def test_refusals():
    with pytest.raises(ValueError):
        MLP(16, 64, 64, 64, weights=inputs.make_mlp(16, 64, 64, 64), fp8=True, checkpoint="bottleneck")
    w = inputs.make_block(16, 64, 64, 2, 64, seed=1)
    blk = Fp8Block(16, 64, 64, 2, 64, weights=w)
    with pytest.raises(ValueError):
        blk.forward(w["x"].cuda(), residual=normal(1, 16, 64))
    _, layer, *_ = make_layer()
    with pytest.raises(ValueError):
        layer.forward(normal(2, 200, 128))              # no positions
