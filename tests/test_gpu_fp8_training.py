"""Blocks whose forward multiplies in 8 bits, in training: their gradients, and where their
products report an error."""

import numpy as np
import pytest
import torch

import oracle
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod
from rank_bottleneck_online_gb300 import inputs
from rank_bottleneck_online_gb300.block import MLP, Block, Fp8Block, Layer, Rotary

from ops_parity import f64
from parity import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def test_the_products_report_to_the_blocks_workspace():
    """One check of a block's workspace sees its 8-bit products too, shared or not."""
    w = inputs.make_layer(64, 128, 64, 128, seed=1)
    layer = Layer(64, 128, 64, 128, S=2, weights=w["p"], rotary=Rotary(32), fp8=True)
    blocks = (layer.qkv, layer.o, layer.mlp.gu, layer.mlp.dn)
    assert len({id(blk.ws) for blk in blocks}) == 1
    own = inputs.make_block(64, 128, 64, 2, 128, seed=2)
    alone = Fp8Block(64, 128, 64, 2, 128, weights=own)
    for blk in (*blocks, alone):
        assert blk.ws8 is blk.ws
        assert blk.ws.nbytes >= B.fp8_matmul_workspace_bytes(64, 128, 128)
    want = alone.forward(own["x"].cuda()).clone()
    alone.backward(own["x"].cuda(), own["dy"].cuda())
    assert torch.equal(alone.forward(own["x"].cuda()), want)
    B.check(alone.ws)


@pytest.mark.parametrize("T,d,r,k,n,norm,act", [(200, 264, 136, 3, 264, True, "silu"),
                                               (130, 128, 64, 1, 136, False, "identity")])
def test_block_gradients_are_the_bf16_blocks(T, d, r, k, n, norm, act):
    """The backward goes straight through the 8-bit roundings: the bf16 block's gradients."""
    w = inputs.make_block(T, d, r, k, n, has_norm=norm, seed=4)
    S = 2 if norm else 1
    x, dy = w["x"].cuda(), w["dy"].cuda()
    blk = Fp8Block(T, d, r, k, n, S=S, has_norm=norm, act=act, weights=w)
    blk.forward(x)
    blk.backward(x, dy)
    B.check(blk.ws)
    a = inputs
    want = oracle.block_bwd(a.as_f64(w["x"]), a.as_f64(w["gamma"]) if norm else None, a.as_f64(w["A"]),
                            a.as_f64(w["B"]), a.as_f64(w["dy"]), act=act, has_norm=norm, S=S,
                            flow="bf16")
    for key in ("dx", "dA", "dB") + (("dgamma",) if norm else ()):
        assert_close(key, getattr(blk, key), want[key])
    plain = Block(T, d, r, k, n, S=S, has_norm=norm, act=act, weights=w)
    plain.forward(x)
    plain.backward(x, dy)
    for key in ("dx", "dA", "dB"):
        assert_close(key, getattr(blk, key), f64(getattr(plain, key)))


@pytest.mark.parametrize("fused", [True, False])
def test_mlp_gradients_stage_by_stage(fused):
    """The MLP's backward from the gate, up and h of its own 8-bit forward."""
    T, d, r, ffn, S = 200, 128, 64, 136, 2
    w = inputs.make_mlp(T, d, r, ffn, seed=6)
    mlp = MLP(T, d, r, ffn, S=S, weights=w, fused_glu=fused, fp8=True)
    x, dout = w["x"].cuda(), w["dout"].cuda()
    mlp.forward(x)
    mlp.backward(x, dout)
    B.check(mlp.gu.ws)
    R, F = oracle.to_bf16, {key: inputs.as_f64(v) for key, v in w.items()}
    gate, up, h = f64(mlp.gu.y[0]), f64(mlp.gu.y[1]), f64(mlp.h)
    # (the fast logistic, the product and the rounding)
    np.testing.assert_allclose(h, oracle.swiglu_fwd(gate, up), rtol=2.0 ** -8 * 1.01, atol=1e-6)
    dn = oracle.block_bwd(h, None, F["A2"], F["B2"], F["dout"][None], has_norm=False, flow="bf16")
    dgate, dup = oracle.swiglu_bwd(gate, up, R(dn["dx"]))
    gu = oracle.block_bwd(F["x"], F["gamma"], F["A1"], F["B1"], np.stack([R(dgate), R(dup)]), S=S,
                          flow="bf16")
    for key, want in {"dx": gu["dx"], "dgamma": gu["dgamma"], "dA1": gu["dA"], "dB1": gu["dB"],
                      "dA2": dn["dA"], "dB2": dn["dB"]}.items():
        assert_close(key, mlp.grads()[key], want)
