"""Rotary positions on the GPU against their fp64 definition.

Tolerance: half a bf16 step, plus what fp32 loses before it: the angle is cut to 2^-31 half
turns and rounded to fp32 (2^-25 half turns), in radians pi (2^-31 + 2^-25) < 1e-7; the sine
and cosine add 2 ulp (2^-22 at most) and the three operations 2^-24 of their terms each:
under 2^-20 of |u| + |v| together.
"""

import math

import numpy as np
import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF, HALF_STEP, close, f64, guarded, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


CASES = [
    # T, hq, hk, dim, rot, axes, interleaved
    (1, 16, 16, 128, 128, 1, False),
    (1, 1, 0, 8, 8, 1, True),
    (3, 4, 2, 64, 64, 1, True),
    (130, 32, 8, 128, 128, 3, False),
    (257, 5, 1, 72, 72, 2, False),            # halves of 36: vectors of 4
    (64, 3, 3, 80, 40, 3, False),             # halves of 20, and values that do not turn
    (33, 2, 1, 96, 8, 1, False),
    (700, 2, 1, 256, 128, 2, True),
    (5, 2, 2, 512, 512, 8, False),
    (2000, 1, 1, 64, 64, 1, False),           # several tokens a block
    (4097, 2, 1, 16, 16, 2, True),
]


def make(T, hq, hk, dim, rot, axes, far, seed=0):
    rng = np.random.default_rng(seed)
    pos = rng.integers(-far, far, (axes, T))
    pos[:, :1] = far
    w = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    axis = rng.integers(0, axes, rot // 2)
    return normal(seed, T, hq, dim), (normal(seed + 1, T, hk, dim) if hk else None), pos, w, axis


def to_gpu(pos, w):
    return torch.from_numpy(pos).int().cuda(), torch.from_numpy(w).cuda()


def slack(x, w, interleaved=False):
    """2^-20 (|u| + |v|) of each value's pair."""
    a, n = np.abs(f64(x)), len(w)
    out = np.zeros_like(a)
    if interleaved:
        s = a[..., 0:2 * n:2] + a[..., 1:2 * n:2]
        out[..., 0:2 * n:2] = out[..., 1:2 * n:2] = s
    else:
        s = a[..., :n] + a[..., n:2 * n]
        out[..., :n] = out[..., n:2 * n] = s
    return out * 2.0 ** -20


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_parity(case, inverse):
    T, hq, hk, dim, rot, axes, inter = case
    q, k, pos, w, axis = make(T, hq, hk, dim, rot, axes, 1 << 20)
    qo, whole_q = guarded((T, hq, dim), BF)
    ko, whole_k = guarded((T, hk, dim), BF) if hk else (None, lambda: True)
    B.rope(q, k, *to_gpu(pos, w), pair_axis=axis.tolist(), interleaved=inter, inverse=inverse,
           q_out=qo, k_out=ko)
    assert whole_q() and whole_k()
    for x, o in ((q, qo), (k, ko)):
        if x is not None:
            close(o, ops.rope(f64(x), pos, w, axis, inter, inverse), slack(x, w, inter))
            assert torch.equal(o[..., rot:], x[..., rot:])


@pytest.mark.parametrize("far", [1 << 31, 1 << 45])
def test_far_and_negative_64_bit_positions(far):
    q, _, pos, w, axis = make(50, 2, 0, 64, 64, 2, far, seed=4)
    out, _ = B.rope(q, None, torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(),
                    pair_axis=axis.tolist())
    # A frequency (at most 1 here) is held to 2^-64 of a turn and its constant 2^64 / (2 pi) to
    # 2^-63 of itself: under 2^-63 |p| turns. That is nothing at 2^31 (2^-32 turns, below the
    # 2^-26 of the fp32 angle), and 2^-18 turns at 2^45.
    turns = far * 2.0 ** -63
    close(out, ops.rope(f64(q), pos, w, axis),
          slack(q, w) * (1 + 2 * math.pi * turns * 2.0 ** 20))


def test_sections_give_pairs_in_order():
    q, k, pos, w, _ = make(20, 2, 1, 64, 64, 3, 500, seed=5)
    p, f = to_gpu(pos, w)
    got = B.rope(q, k, p, f, sections=[8, 0, 24])
    want = B.rope(q, k, p, f, pair_axis=[0] * 8 + [2] * 24)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_frequencies_zero_large_and_not_finite():
    T, pairs = 4, 8
    q = normal(6, T, 1, 16)
    w = np.array([0.0, 5e-324, 1e-30, 1.0, -1.0, 6.5, 1e6, np.nan])
    pos = np.array([[0, 1, 77, 100003]])
    out, _ = B.rope(q, None, *to_gpu(pos, w))
    want = ops.rope(f64(q), pos, np.where(np.isfinite(w), w, 0.0), [0] * pairs)
    got = f64(out)
    assert np.isnan(got[..., [7, 15]]).all()
    keep = [i for i in range(16) if i not in (7, 15)]
    # (a frequency of 1e6 is 2^17.3 turns of which the constant loses 2^-63: 2^-29 turns at
    # these positions; values are below 4)
    np.testing.assert_allclose(got[..., keep], want[..., keep], rtol=HALF_STEP * 1.01,
                               atol=2.0 ** -17)


@pytest.mark.parametrize("layout", ["packed", "heads_first", "in_place", "packed_in_place"])
def test_layouts(layout):
    T, hq, hk, dim = 37, 4, 2, 64
    q, k, pos, w, axis = make(T, hq, hk, dim, dim, 2, 3000, seed=7)
    (p, f), a = to_gpu(pos, w), axis.tolist()
    want = B.rope(q, k, p, f, pair_axis=a)
    if layout == "heads_first":
        q1, k1 = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k))
        got = B.rope(q1, k1, p, f, pair_axis=a,
                     q_out=torch.empty(hq, T, dim, dtype=BF, device="cuda").transpose(0, 1))
    elif layout == "in_place":
        q1, k1 = q.clone(), k.clone()
        got = B.rope(q1, k1, p, f, pair_axis=a, q_out=q1, k_out=k1)
        assert got[0].data_ptr() == q1.data_ptr()
    else:
        rest = normal(8, T, 3, dim)
        whole = torch.cat([q, k, rest], 1)
        q1, k1 = whole[:, :hq], whole[:, hq:hq + hk]
        inside = layout == "packed_in_place"
        got = B.rope(q1, k1, p, f, pair_axis=a, q_out=q1 if inside else None,
                     k_out=k1 if inside else None)
        assert torch.equal(whole[:, hq + hk:], rest)
        if not inside:
            assert torch.equal(whole[:, :hq], q)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_inverse_is_the_gradient():
    """d <rope(q), g> / dq by central differences of the fp64 definition equals the call's."""
    q, _, pos, w, axis = make(6, 1, 0, 16, 16, 2, 100, seed=9)
    g = normal(10, 6, 1, 16)
    dq, _ = B.rope(g, None, *to_gpu(pos, w), pair_axis=axis.tolist(), inverse=True)
    x, gg, h = f64(q), f64(g), 1e-3
    want = np.zeros_like(x)
    for at in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[at] = h
        want[at] = ((ops.rope(x + e, pos, w, axis) - ops.rope(x - e, pos, w, axis)) * gg).sum() / (2 * h)
    # the definition is linear in q: the differences lose only their own rounding
    close(dq, want, slack(g, w) + 1e-9)


def test_offsets_beyond_32_bits():
    """Token rows 2^22 values apart over 1100 tokens: offsets pass 2^32 values."""
    T, step = 1100, 1 << 22
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 10 GB for the strided tensor")
    whole = torch.empty(T, step, dtype=BF, device="cuda")
    q = normal(11, T, 1, 64)
    whole[:, :64] = q[:, 0]
    pos, w = np.arange(T)[None], 10000.0 ** (-np.arange(32) / 32)
    p, f = to_gpu(pos, w)
    view = whole[:, :64].unsqueeze(1)
    got, _ = B.rope(view, None, p, f, q_out=view)
    assert torch.equal(got, B.rope(q, None, p, f)[0])


def test_refuses_what_the_binding_sees():
    q, k, pos, w, _ = make(4, 2, 1, 64, 64, 2, 10)
    p, f = to_gpu(pos, w)
    for kw in (dict(sections=[32]), dict(sections=[40, -8]), dict(pair_axis=[2] * 32),
               dict(sections=[16, 16], pair_axis=[0] * 32), dict(q_out=q[:3]),
               dict(k_out=torch.empty(4, 2, 64, dtype=BF, device="cuda"))):
        with pytest.raises(ValueError):
            B.rope(q, k, p, f, **kw)
    for args in ((q.float(), k, p, f), (q, k, p.float(), f), (q, k, p, f.float())):
        with pytest.raises(TypeError):
            B.rope(*args)
    for args in ((q.cpu(), k, p, f), (q, k, p.cpu(), f), (q[0], k, p, f), (q, k[:3], p, f),
                 (q, k, p[:, :3].contiguous(), f), (q.transpose(1, 2), k, p, f)):
        with pytest.raises(ValueError):
            B.rope(*args)
    with pytest.raises(B.BoostError):                  # 32 pairs do not fit 56 values
        B.rope(q[..., :56], None, p, f)


def test_no_tokens():
    e = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    out, _ = B.rope(e, None, torch.empty(0, dtype=torch.int32, device="cuda"),
                    torch.ones(32, dtype=torch.float64, device="cuda"))
    assert out.shape == e.shape


def test_another_stream_and_a_replayed_graph():
    q, k, pos, w, axis = make(200, 4, 4, 64, 64, 1, 900)
    p, f = to_gpu(pos, w)
    want = B.rope(q, k, p, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = B.rope(q, k, p, f, stream=side)
    with torch.cuda.stream(side):
        again = B.rope(q, k, p, f)
    side.synchronize()
    for g in (got, again):
        assert all(torch.equal(x, y) for x, y in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = B.rope(q, k, p, f)
    p.add_(5)
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(out, B.rope(q, k, p, f)))
