"""The norm behind a residual with an 8-bit output, on the GPU: the sum, the operand and its
scales are exact, the row scale within what fp32 sums lose."""

import numpy as np
import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF, f64, guarded, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def call(x, residual, gamma, fmt, **kw):
    T, d = x.shape
    h, whole_h = guarded((T, d), BF)
    rstd, whole_r = guarded((T,), torch.float32)
    q, whole_q = guarded((T, -(-d // 16) * 16), B.FP8_FORMATS[fmt][1])
    sf, whole_s = guarded((B.fp8_scale_bytes(T, d),), torch.uint8)
    got = B.norm_quantize(x, residual=residual, gamma=gamma, fmt=fmt, h=h, rstd=rstd,
                          rows_out=(q, sf), **kw)
    assert got[0] is h and whole_h() and whole_r() and whole_q() and whole_s()
    return h, rstd, q, sf


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("residual,weighted", [(True, False), (False, False), (True, True), (False, True)])
@pytest.mark.parametrize("T,d", [(1, 8), (1, 2048), (3, 504), (33, 520), (127, 1032), (129, 4096),
                                 (5, 4104), (66, 11008), (200, 264)])
def test_parity(T, d, residual, weighted, fmt):
    x, res = normal(1, T, d) * 4, normal(2, T, d)
    gamma = normal(3, d) if weighted else None
    h, rstd, q, sf = call(x, res if residual else None, gamma, fmt)
    want = torch.from_numpy(f64(x) + f64(res)).to(BF) if residual else x.cpu()
    assert torch.equal(h.cpu(), want)
    # d squares in fp32, each step off by 2^-24 of the sum at most, then a root: far below 1e-5
    np.testing.assert_allclose(f64(rstd), ops.row_scale(f64(h), 1e-5), rtol=1e-5)
    y = f64(h)
    if weighted:
        y = torch.from_numpy(y * f64(gamma)).to(BF).double().numpy()
    values, e = ops.fp8_quantize(y, fmt)
    np.testing.assert_array_equal(f64(q)[:, :d], values)
    assert (q[:, d:].view(torch.uint8) == 0).all()
    np.testing.assert_array_equal(sf.cpu().numpy(), ops.fp8_scales(e))


def test_the_operand_is_the_quantisers():
    x = normal(4, 300, 1000)
    x[5] = 0
    x[7, 3], x[8, 200], x[9, 900] = float("nan"), float("inf"), -float("inf")
    x[10] *= 2.0 ** -120
    x[11] *= 2.0 ** 100
    for fmt in ("e4m3", "e5m2"):
        h, rstd, (q, sf) = B.norm_quantize(x, fmt=fmt)
        (want, want_sf), _ = B.fp8_quantize(x, fmt=fmt)
        assert h is x
        assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)) and torch.equal(sf, want_sf)
        assert torch.isnan(rstd[7]) and rstd[8] == 0 and rstd[9] == 0
        assert abs(rstd[5].item() - 1e-5 ** -0.5) < 1e-3


@pytest.mark.parametrize("which", ["x", "residual"])
def test_in_place(which):
    x, res = normal(5, 50, 320), normal(6, 50, 320)
    want = B.norm_quantize(x, residual=res)
    to = x if which == "x" else res
    got = B.norm_quantize(x, residual=res, h=to)
    assert got[0] is to and torch.equal(to, want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[2][0].view(torch.uint8), want[2][0].view(torch.uint8))


def test_feeds_the_product():
    """The operand with its row scale gives the normed projection."""
    T, d, n = 70, 384, 64
    x, res, w = normal(7, T, d), normal(8, T, d), normal(9, n, d)
    h, rstd, (q, sf) = B.norm_quantize(x, residual=res)
    (w8, wsf), _ = B.fp8_quantize(w, block_rows=128)
    ws = B.Workspace(B.fp8_matmul_workspace_bytes(T, n, d))
    y = B.fp8_matmul(q, sf, w8, wsf, d, ws, row_scale=rstd)
    B.check(ws)
    hv, e = ops.fp8_quantize(f64(h), "e4m3")
    wv, we = ops.fp8_quantize(f64(w), "e4m3", 128)
    want, size = ops.fp8_matmul(ops.fp8_dequantize(hv, e), ops.fp8_dequantize(wv, we), f64(rstd))
    assert (np.abs(f64(y) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * size).all()


def test_captured_on_another_stream():
    x, res = normal(10, 260, 2048), normal(11, 260, 2048)
    want = B.norm_quantize(x, residual=res)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, rstd, (q, sf) = B.norm_quantize(x, residual=res)
    graph.replay()
    for a, b in ((h, want[0]), (rstd, want[1]), (q.view(torch.uint8), want[2][0].view(torch.uint8)),
                 (sf, want[2][1])):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h2 = B.norm_quantize(x, residual=res, stream=side)[0]
    side.synchronize()
    assert torch.equal(h2, want[0])


def test_refuses_what_the_binding_sees():
    x = normal(12, 16, 64)
    with pytest.raises(TypeError):
        B.norm_quantize(x.float())
    with pytest.raises(ValueError):
        B.norm_quantize(x, fmt="e3m4")
    for kw in (dict(residual=normal(1, 8, 64)), dict(gamma=normal(1, 16)), dict(h=x[:8]),
               dict(rstd=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            B.norm_quantize(x, **kw)
    with pytest.raises(ValueError):
        B.norm_quantize(normal(1, 64))
    with pytest.raises(B.BoostError):
        B.norm_quantize(normal(1, 4, 60))
    with pytest.raises(B.BoostError):
        B.norm_quantize(x, eps=-1.0)
    assert B.norm_quantize(x[:0])[1].numel() == 0
