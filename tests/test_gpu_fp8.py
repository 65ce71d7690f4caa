"""The 8-bit quantiser and matrix product on the GPU against their fp64 definitions.

The quantiser's values and scales are exact. Tolerance of the product: half a bf16 step, plus
what the fp32 sums lose: every addition at most 2^-23 of the running magnitude (the tensor
core may truncate), and K / 32 + 32 of them follow one another (32 within one instruction):
(K / 32 + 32) 2^-23 of the summed magnitudes. The fast logistic is within 2^-20, and silu's
slope is below 1.1.
"""

import math

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


# ---------------------------------------------------------------------- quantiser
QUANT = [(1, 8), (1, 512), (7, 24), (31, 520), (127, 128), (128, 136), (129, 120), (300, 1000),
         (16, 4096), (513, 256)]


def quant_check(x, fmt, block_rows, got, transposed):
    v = f64(x).T if transposed else f64(x)
    rows, K = v.shape
    want, e = ops.fp8_quantize(v, fmt, block_rows)
    q, sf = got
    g = f64(q)
    assert g.shape == (rows, -(-K // 16) * 16)
    np.testing.assert_array_equal(sf.cpu().numpy(), ops.fp8_scales(e))
    np.testing.assert_array_equal(g[:, :K], want)
    assert (g[:, K:] == 0).all()


def wide_normal(seed, *shape):
    """Rows of magnitudes far apart, one of zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp2(
        torch.randint(-20, 21, shape[:-1] + (1,), generator=g).float())
    x[..., shape[-2] // 2, :] = 0
    return x.to(BF).cuda()


@pytest.mark.parametrize("way", ["rows", "columns", "both"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("shape", QUANT, ids=lambda s: f"{s[0]}x{s[1]}")
def test_quantise(shape, fmt, block_rows, way):
    rows, cols = shape
    x = wide_normal(rows, rows, cols)
    outs, checks = {}, []
    for name, r, K in (("rows", rows, cols), ("cols", cols, rows)):
        if way != {"rows": "columns", "cols": "rows"}[name]:
            q, whole_q = guarded((r, -(-K // 16) * 16), B.FP8_FORMATS[fmt][1])
            sf, whole_s = guarded((B.fp8_scale_bytes(r, K),), torch.uint8)
            outs[name + "_out"] = (q, sf)
            checks += [whole_q, whole_s]
    by_rows, by_cols = B.fp8_quantize(x, fmt=fmt, block_rows=block_rows, way=way, **outs)
    assert all(c() for c in checks)
    if by_rows is not None:
        quant_check(x, fmt, block_rows, by_rows, False)
    if by_cols is not None:
        quant_check(x, fmt, block_rows, by_cols, True)


@pytest.mark.parametrize("way", ["rows", "both"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantise_extreme_values(fmt, block_rows, way):
    x = normal(3, 260, 264)
    top = torch.finfo(BF).max
    x[0] = 0
    x[1, :] = 1e-39                                    # subnormal: the scale stops at 2^-127
    x[2, 5], x[2, 130] = top, -top
    x[3, 7], x[3, 200] = float("inf"), float("-inf")
    x[4, 9] = float("nan")
    x[5, :] = float("inf")
    x[6, :] = float("nan")
    x[7, 0:128] = 1.75                                 # exactly fmax times a power of two
    x[8, 0:128] = 1.7578125                            # one step above it
    x[200, 3] = 2.0 ** -133
    by_rows, by_cols = B.fp8_quantize(x, fmt=fmt, block_rows=block_rows, way=way)
    quant_check(x, fmt, block_rows, by_rows, False)
    if by_cols is not None:
        quant_check(x, fmt, block_rows, by_cols, True)


def test_quantise_strided_matrices():
    # the groups of a [T, k r] bottleneck activation as k matrices [T, r]
    T, k, r = 70, 3, 136
    a = wide_normal(5, T, k * r)
    x = a.view(T, k, r).transpose(0, 1)
    by_rows, by_cols = B.fp8_quantize(x, way="both")
    only, _ = B.fp8_quantize(x)
    for g in range(k):
        quant_check(x[g], "e4m3", 1, (by_rows[0][g], by_rows[1][g]), False)
        quant_check(x[g], "e4m3", 1, (by_cols[0][g], by_cols[1][g]), True)
        quant_check(x[g], "e4m3", 1, (only[0][g], only[1][g]), False)


@pytest.mark.parametrize("block_rows,way", [(1, "columns"), (1, "both"), (128, "rows"), (128, "both")])
def test_quantise_folds_gamma(block_rows, way):
    x, gamma = normal(6, 200, 136), normal(7, 200)
    got = B.fp8_quantize(x, way=way, block_rows=block_rows, gamma=gamma)
    folded = (x.float() * gamma.float()[:, None]).to(BF)
    want = B.fp8_quantize(folded, way=way, block_rows=block_rows)
    for a, b in zip(got, want):
        if a is not None:
            assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))
            assert torch.equal(a[1], b[1])


def test_quantise_refuses_what_the_binding_sees():
    x = normal(8, 16, 64)
    for kw in (dict(fmt="e3m4"), dict(way="all"), dict(gamma=normal(1, 64), way="columns"),
               dict(cols_out=(x, x))):
        with pytest.raises(ValueError):
            B.fp8_quantize(x, **kw)
    for bad in (x.T, x.cpu(), x[None, None]):
        with pytest.raises(ValueError):
            B.fp8_quantize(bad)
    with pytest.raises(TypeError):
        B.fp8_quantize(x.float())
    with pytest.raises(TypeError):
        B.fp8_quantize(x, rows_out=(torch.empty(16, 64, dtype=BF, device="cuda"), x))
    for bad in (x[:, :60], normal(9, 16, 68)[:, :64]):
        with pytest.raises(B.BoostError):
            B.fp8_quantize(bad)
    with pytest.raises(B.BoostError):
        B.fp8_quantize(x, gamma=normal(1, 16))          # a fold of rows alone
    with pytest.raises(B.BoostError):
        B.fp8_quantize(x, block_rows=2)


# ------------------------------------------------------------------------- product
def operand(seed, fmt, *shape):
    """Random codes (finite) of [.., rows, K] with scales far apart, and their fp64 values."""
    lead, (rows, K) = shape[:-2], shape[-2:]
    rng = np.random.default_rng(seed)
    G, pitch, blocks = math.prod(lead), -(-K // 16) * 16, -(-K // 128)
    codes = rng.integers(0, 256, (G, rows, pitch)).astype(np.uint8)
    # magnitudes of ordinary data: the exponent's upper half would drown the rest
    codes &= np.uint8(0xBF)
    codes[:, :, K:] = 0x7F                              # what lies behind K is not read
    exps = rng.integers(-6, 7, (G, rows, blocks))
    sf = np.stack([ops.fp8_scales(e) for e in exps])
    table = ops.fp8_values(fmt)
    values = np.stack([ops.fp8_dequantize(table[c[:, :K]], e) for c, e in zip(codes, exps)])
    q = torch.from_numpy(codes).cuda().view(B.FP8_FORMATS[fmt][1]).view(lead + (rows, pitch))
    return q, torch.from_numpy(sf).cuda().view(lead + (-1,)), values


def workspace(M, N, K, G=1):
    return B.Workspace(B.fp8_matmul_workspace_bytes(M, N, K, G))


def lost(K, size):
    return (K / 32 + 32) * 2.0 ** -23 * size


def product_check(lead, M, N, K, fa="e4m3", fb="e4m3", scaled=False, act="identity", seed=0):
    a, asf, va = operand(seed, fa, *lead, M, K)
    b, bsf, vb = operand(seed + 1, fb, *lead, N, K)
    rs = None
    if scaled:
        rs = torch.from_numpy(np.random.default_rng(seed).uniform(0.1, 2, M).astype(np.float32)).cuda()
    out, whole = guarded(tuple(lead) + (M, N), BF)
    ws = workspace(M, N, K, math.prod(lead))
    B.fp8_matmul(a, asf, b, bsf, K, ws, row_scale=rs, act=act, out=out)
    B.check(ws)
    assert whole()
    got = out.view(-1, M, N)
    for g in range(len(va)):
        want, size = ops.fp8_matmul(va[g], vb[g], None if rs is None else f64(rs), act)
        close(got[g], want, 1.1 * lost(K, size) + 2.0 ** -20 * np.abs(want))


PRODUCT = [(1, 8, 8), (1, 64, 128), (1, 1024, 1000), (2, 264, 129), (3, 136, 2056), (8, 512, 512),
           (15, 72, 4096), (17, 256, 256), (33, 128, 640), (64, 512, 1024), (65, 520, 384),
           (127, 8, 1), (128, 256, 127), (129, 264, 128), (200, 1000, 520), (256, 256, 1024),
           (257, 512, 2048), (300, 136, 16), (513, 776, 1160), (1030, 528, 4100)]


@pytest.mark.parametrize("shape", PRODUCT, ids=lambda s: "x".join(map(str, s)))
def test_product(shape):
    product_check((), *shape)


@pytest.mark.parametrize("shape", [(4700, 5128, 300), (2500, 6152, 1000), (100, 25608, 256)],
                         ids=lambda s: "x".join(map(str, s)))
def test_product_with_more_tiles_than_fit_at_once(shape):
    """Several tiles a CTA: both accumulators in turn (the wide tile's share columns), the ring
    and the scale buffers going on from tile to tile, for CTA pairs and single CTAs."""
    product_check((), *shape, scaled=True)


def test_product_batch_with_more_tiles_than_fit_at_once():
    product_check((3,), 1300, 2056, 140)


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M", [5, 300])
def test_product_formats(fa, fb, M):
    product_check((), M, 264, 700, fa, fb)


@pytest.mark.parametrize("M", [1, 30, 300])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("act", ["identity", "silu"])
def test_product_epilogue(M, scaled, act):
    product_check((), M, 264, 520, scaled=scaled, act=act)


@pytest.mark.parametrize("M", [1, 40, 130, 520])
@pytest.mark.parametrize("lead", [(1,), (3,)])
def test_product_batches(M, lead):
    product_check(lead, M, 520, 300)


@pytest.mark.parametrize("M", [1, 20, 300])
def test_product_extreme_scales(M):
    """A scale byte of 0 is 2^-127 and one of 255 NaN; the bytes of rows and blocks outside
    the operands are not read."""
    N, K = 136, 300
    a, asf, va = operand(1, "e4m3", M, K)
    b, bsf, vb = operand(2, "e4m3", N, K)

    def at(r, blk):
        return r // 128 * 512 + r % 32 * 16 + r // 32 % 4 * 4 + blk

    for sf, rows in ((asf, M), (bsf, N)):
        unused = np.ones(sf.numel(), dtype=bool)
        unused[[at(r, blk) for r in range(rows) for blk in range(3)]] = False
        sf[torch.from_numpy(unused).cuda()] = 255
    asf[at(0, 1)] = 0
    bsf[at(9, 2)] = 255
    out = B.fp8_matmul(a, asf, b, bsf, K, workspace(M, N, K))
    va[0, 0, 128:256] = f64(a)[0, 128:256] * 2.0 ** -127
    want, size = ops.fp8_matmul(va[0], vb[0])
    assert np.isnan(f64(out)[:, 9]).all()
    keep = [i for i in range(N) if i != 9]
    close(out[:, keep], want[:, keep], lost(K, size[:, keep]))


@pytest.mark.parametrize("M", [1, 20, 300])
def test_product_values_that_are_not_finite_stay_in_their_row_and_column(M):
    N, K = 264, 200
    a, asf, _ = operand(3, "e4m3", M, K)
    b, bsf, _ = operand(4, "e5m2", N, K)
    a.view(torch.uint8)[M - 1, 3] = 0x7F                # NaN
    a.view(torch.uint8)[:, 150] = 0x38                  # 1, against:
    b.view(torch.uint8)[17, 150] = 0x7C                 # infinity
    out = f64(B.fp8_matmul(a, asf, b, bsf, K, workspace(M, N, K)))
    assert np.isnan(out[M - 1]).all()
    assert (out[:M - 1, 17] == np.inf).all()
    assert np.isfinite(np.delete(out[:M - 1], 17, axis=1)).all()


def test_product_without_a_contraction_or_rows():
    ws = workspace(4, 8, 0)
    s = torch.empty(0, dtype=torch.uint8, device="cuda")
    out = torch.ones(4, 8, dtype=BF, device="cuda")
    B.fp8_matmul(torch.empty(4, 0, dtype=torch.float8_e4m3fn, device="cuda"), s,
                 torch.empty(8, 0, dtype=torch.float8_e4m3fn, device="cuda"), s, 0, ws, out=out)
    assert (out == 0).all()
    b, bsf, _ = operand(1, "e4m3", 8, 64)
    assert B.fp8_matmul(torch.empty(0, 64, dtype=torch.float8_e4m3fn, device="cuda"), s, b, bsf, 64,
                        workspace(0, 8, 64)).shape == (0, 8)


def test_product_is_the_same_every_time():
    for M, N, K in ((1, 1024, 4096), (40, 512, 8192), (300, 520, 4096)):
        a, asf, _ = operand(5, "e4m3", M, K)
        b, bsf, _ = operand(6, "e4m3", N, K)
        ws = workspace(M, N, K)
        first = B.fp8_matmul(a, asf, b, bsf, K, ws)
        for _ in range(5):
            assert torch.equal(first, B.fp8_matmul(a, asf, b, bsf, K, ws))


def test_product_refuses_what_the_binding_sees():
    a, asf, _ = operand(7, "e4m3", 16, 128)
    b, bsf, _ = operand(8, "e4m3", 64, 128)
    ws = workspace(16, 64, 128)
    for args, kw in (((a, asf[:-1], b, bsf, 128, ws), {}), ((a[None], asf[None], b, bsf, 128, ws), {}),
                     ((a, asf, b, bsf.cpu(), 128, ws), {}), ((a[:, ::2], asf, b, bsf, 64, ws), {}),
                     ((a, asf, b, bsf, 128, ws), dict(out=torch.empty(16, 72, dtype=BF, device="cuda"))),
                     ((a, asf, b, bsf, 128, ws), dict(row_scale=torch.ones(64, device="cuda")))):
        with pytest.raises(ValueError):
            B.fp8_matmul(*args, **kw)
    with pytest.raises(TypeError):
        B.fp8_matmul(a.view(torch.uint8), asf, b, bsf, 128, ws)
    with pytest.raises(B.BoostError):
        B.fp8_matmul(a, asf, b[:60], bsf, 128, ws)      # N % 8
    with pytest.raises(B.BoostError):                  # K beyond the operands' pitch
        B.fp8_matmul(a, asf, b, bsf, 144, ws)


def test_product_gradients_of_quantised_operands():
    """y = x W^T, dx = dy W and dW = dy^T x by operands quantised the other way, against the
    fp64 gradients of the same quantised values."""
    T, N, K = 200, 136, 264
    x, wgt, dy = normal(30, T, K), normal(31, N, K), normal(32, T, N)
    (xq, xt), (wq, wt) = B.fp8_quantize(x, way="both"), B.fp8_quantize(wgt, way="both", block_rows=128)
    gq, gt = B.fp8_quantize(dy, way="both", fmt="e5m2")
    y = B.fp8_matmul(*xq, *wq, K, workspace(T, N, K))
    dx = B.fp8_matmul(*gq, *wt, N, workspace(T, K, N))
    dw = B.fp8_matmul(*gt, *xt, T, workspace(N, K, T))

    def values(t, fmt, rows):
        return ops.fp8_dequantize(*ops.fp8_quantize(t, fmt, rows))

    X, W, G = f64(x), f64(wgt), f64(dy)
    for got, a, b, k in ((y, values(X, "e4m3", 1), values(W, "e4m3", 128), K),
                         (dx, values(G, "e5m2", 1), values(W, "e4m3", 128).T, N),
                         (dw, values(G.T, "e5m2", 1), values(X.T, "e4m3", 1), T)):
        want, size = ops.fp8_matmul(a, b)
        close(got, want, lost(k, size))


def test_another_stream_and_a_replayed_graph():
    M, N, K = 160, 256, 512
    x, wgt = normal(12, M, K), normal(13, N, K)
    wq, wsf = B.fp8_quantize(wgt, block_rows=128)[0]
    ws = workspace(M, N, K)

    def step(stream=None):
        xq, xsf = B.fp8_quantize(x, stream=stream)[0]
        return B.fp8_matmul(xq, xsf, wq, wsf, K, ws, act="silu", stream=stream)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = step()
    for trial in range(3):
        x.copy_(normal(20 + trial, M, K))
        graph.replay()
        B.check(ws)
        assert torch.equal(z, step())


def test_offsets_beyond_32_bits():
    """An operand of 4.3e9 values: its last rows, quantised both ways and multiplied, are what
    those rows alone give."""
    rows, K, N = 8281 * 128 + 37, 4096, 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 20 GB")
    x = torch.empty(rows, K, dtype=BF, device="cuda").normal_()
    w, wsf = B.fp8_quantize(normal(40, N, K), block_rows=128)[0]
    (q, sf), (qt, _) = B.fp8_quantize(x, way="both")
    only, only_sf = B.fp8_quantize(x)[0]
    assert torch.equal(sf, only_sf) and torch.equal(q[-1].view(torch.uint8), only[-1].view(torch.uint8))
    del only
    first = 8275 * 128
    (tq, tsf), (tqt, _) = B.fp8_quantize(x[first:], way="both")
    assert torch.equal(q[first:].view(torch.uint8), tq.view(torch.uint8))
    assert torch.equal(sf[-tsf.numel():], tsf)
    n = rows - first
    assert torch.equal(qt[:, first:rows].view(torch.uint8), tqt[:, :n].view(torch.uint8))
    out = B.fp8_matmul(q, sf, w, wsf, K, workspace(rows, N, K))
    tail = B.fp8_matmul(tq, tsf, w, wsf, K, workspace(n, N, K))
    # another order of the sums: a bf16 step where a value lies between two, and the fp32 sums'
    # loss near zero (K = 4096 values of about 1: 160 additions of 2^-23 of 4096)
    torch.testing.assert_close(out[first:], tail, rtol=torch.finfo(BF).eps, atol=160 * 2.0 ** -23 * 4096)
