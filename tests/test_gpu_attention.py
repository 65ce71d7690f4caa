"""Attention and its gradients on the GPU against their fp64 definition (tolerances:
attention_parity)."""

import numpy as np
import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from attention_parity import FINE, SENTINEL, SLACK, Case
from ops_parity import BF, close, f64, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("n", [1, 2, 63, 127, 128, 129, 255, 256, 257, 400])
def test_one_sequence(n, dim, causal):
    Case([(n, n)], 2, 2, dim, causal=causal, seed=n + dim).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [(1, 1000), (1, 128), (5, 129), (130, 700), (300, 40), (129, 1),
                                   (513, 385), (200, 0), (257, 256)])
def test_other_numbers_of_queries_and_keys(nq, nk, causal):
    """New tokens behind a context, and queries that see nothing."""
    out, lse, (dq, _, _) = Case([(nq, nk)], 4, 2, 64, causal=causal, seed=nq).check()
    none = nq - nk if causal else (nq if nk == 0 else 0)
    if none > 0:
        assert (out[:none] == 0).all() and (dq[:none] == 0).all()
        assert (lse[:, :none] == -float("inf")).all()


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (8, 8), (10, 2), (24, 8), (7, 1), (40, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_shared_key_heads(hq, hk, dim):
    Case([(150, 150), (1, 300), (33, 5)], hq, hk, dim, seed=hq).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", ["planes", "packed", "heads"])
@pytest.mark.parametrize("tail", [0, 1, 200])
def test_packed_sequences(tail, layout, causal):
    lengths = [(1, 1), (0, 5), (130, 130), (7, 300), (5, 0), (0, 0), (256, 256), (64, 65), (3, 2)]
    Case(lengths, 4, 2, 96, causal=causal, tail=tail, layout=layout, seed=tail).check()


def test_many_sequences():
    rng = np.random.default_rng(3)
    lengths = [tuple(int(v) for v in rng.integers(0, 12, 2)) for _ in range(300)]
    Case(lengths, 2, 1, 64, tail=9).check()


@pytest.mark.parametrize("spread,scale", [(8.0, None), (0.01, None), (1.0, 0.03), (1.0, 1.0)])
def test_sharp_and_flat_rows(spread, scale):
    """Scores of up to +-50 (a row's maximum rises many times) and hardly any."""
    Case([(300, 700)], 2, 2, 64, spread=spread * 0.7, scale=scale, seed=5).check()


def test_rising_and_falling_scores():
    """Every key's score above, or below, all before it: the running maximum moves with each."""
    for sign in (1, -1):
        c = Case([(140, 900)], 1, 1, 64, causal=False, seed=6)
        c.q.zero_()
        c.q[:, :, 0] = 8.0
        c.k[:, :, 0] = (sign * torch.arange(900) / 16.0).to(BF).cuda()[:, None]
        c.check()


def test_long_sequences():
    Case([(2048, 2048), (1, 5000), (77, 4100)], 2, 1, 128, seed=8).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [72, 96, 104, 128])
@pytest.mark.parametrize("lengths", [[(512, 512)], [(640, 640)], [(1025, 1153)], [(900, 1300), (700, 515)],
                                     [(1300, 600)], [(1000, 1090), (130, 0), (511, 513)]])
def test_sequences_of_several_tiles(lengths, dim, causal):
    Case(lengths, 2, 2, dim, causal=causal, seed=dim, tail=70).check()


@pytest.mark.parametrize("hq,hk", [(6, 2), (5, 1)])
@pytest.mark.parametrize("layout", ["packed", "heads"])
def test_sequences_of_several_tiles_with_shared_key_heads(hq, hk, layout):
    Case([(700, 700), (1, 900), (850, 610)], hq, hk, 128, layout=layout, tail=3, seed=hq).check()


def behind(lengths, heads=2):
    """Rows behind the last sequence that make a sequence's share of all rows 2100, and that of scores
    2^24: the sizes that the gradients' kernels are chosen by, where the sequences are smaller."""
    n = len(lengths)
    return max(2100 * n, int((2.0 ** 24 * n / heads) ** 0.5) + 1) - min(map(sum, zip(*lengths))) + 70


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [72, 96, 104, 128])
@pytest.mark.parametrize("lengths", [[(1, 1)], [(129, 257)], [(512, 512)], [(1025, 1153)],
                                     [(900, 1300), (700, 515)], [(1300, 600)], [(2305, 2177)],
                                     [(1000, 1090), (130, 0), (0, 7), (511, 513)]])
def test_sequences_of_pairs_of_tiles(lengths, dim, causal):
    Case(lengths, 2, 2, dim, causal=causal, seed=dim, tail=behind(lengths)).check()


@pytest.mark.parametrize("hq,hk", [(6, 2), (5, 1)])
@pytest.mark.parametrize("layout", ["packed", "heads"])
def test_sequences_of_pairs_of_tiles_with_shared_key_heads(hq, hk, layout):
    lengths = [(700, 700), (1, 900), (850, 610)]
    Case(lengths, hq, hk, 128, layout=layout, tail=behind(lengths), seed=hq).check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_pairs_of_tiles_do_not_leak(bad):
    lengths = [(600, 790), (530, 570), (660, 660), (629, 840)]
    _leak(lengths, 128, bad, behind(lengths))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 128])
@pytest.mark.parametrize("n", [(1, 1), (2, 3), (7, 128), (63, 1), (127, 129), (256, 255), (400, 400)])
def test_one_sequence_of_many_rows(n, dim, causal):
    """Most rows lie behind the sequence."""
    Case([n], 3, 1, dim, causal=causal, tail=600, seed=n[0] + dim).check()


@pytest.mark.parametrize("n", [(1, 1), (7, 128), (127, 129), (400, 380)])
@pytest.mark.parametrize("dim", [64, 72, 128])
def test_two_sequences_of_many_rows(dim, n):
    """As many rows as hide how few scores there are."""
    Case([n, n[::-1]], 12, 6, dim, tail=1900, seed=n[0] + dim).check()


@pytest.mark.parametrize("layout", ["planes", "packed", "heads"])
@pytest.mark.parametrize("dim", [56, 96])
def test_packed_sequences_of_many_rows(dim, layout):
    lengths = [(1, 1), (0, 5), (130, 130), (7, 300), (5, 0), (0, 0), (256, 256), (64, 65), (3, 2)]
    Case(lengths, 4, 2, dim, tail=2000, layout=layout, seed=dim).check()
    Case(lengths, 4, 2, dim, tail=6000, layout=layout, seed=dim).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [16, 64, 80, 128])
@pytest.mark.parametrize("lengths,hq,hk", [([(1, 2)], 1, 1), ([(4, 4), (4, 4)], 2, 1), ([(6, 6)], 1, 1),
                                           ([(33, 65), (5, 1), (0, 3)], 4, 2), ([(130, 257)], 6, 2),
                                           ([(200, 140), (3, 200)], 6, 6),
                                           ([(867, 3), (3, 1350)], 2, 1)])
def test_few_scores(lengths, hq, hk, dim, causal):
    """Gradients that are off by little more than their own rounding."""
    for seed in range(4):
        Case(lengths, hq, hk, dim, causal=causal, seed=seed).check(FINE)


@pytest.mark.parametrize("tail", [0, 700, 4500])
@pytest.mark.parametrize("dim", [64, 128])
def test_a_single_key_has_no_gradient(dim, tail):
    """Its probability is 1 whatever its score: dq of a row that sees one key and dk of a sequence
    of one key are 0, to the bit."""
    c = Case([(150, 1), (70, 70)], 4, 2, dim, tail=tail, seed=dim, causal=False)
    _, _, (dq, dk, _) = c.check()
    assert (dq[:150] == 0).all() and (dk[:1] == 0).all()
    c = Case([(150, 1), (70, 70), (1, 1)], 4, 2, dim, tail=tail, seed=dim)
    _, _, (dq, dk, _) = c.check()
    assert (dq[:151] == 0).all() and (dk[:1] == 0).all() and (dq[220] == 0).all()
    assert (dk[71] == 0).all()


@pytest.mark.parametrize("nq", [1, 3])
def test_one_token_over_a_long_context(nq):
    Case([(nq, 30000), (nq, 1), (nq, 129), (nq, 9999)], 5, 1, 128, seed=9).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hk,dim", [(4, 4, 64), (6, 2, 128), (32, 1, 72), (40, 1, 128)])
@pytest.mark.parametrize("lengths", [[(1, 1100)], [(2, 1500), (0, 700), (1, 0), (3, 2049), (1, 640)],
                                     [(4, 900)] * 5 + [(1, 1)], [(12, 3000), (1, 5)]])
def test_parts_of_the_keys(lengths, hq, hk, dim, causal):
    """Few queries over many keys: the keys go in parts, joined at the end."""
    Case(lengths, hq, hk, dim, causal=causal, tail=2, seed=dim).check()


def test_equal_parts_of_the_keys():
    """More queries than a tile's, but too few tiles for the SMs."""
    Case([(300, 6000), (200, 3000)], 2, 2, 128, seed=20).check()
    Case([(400, 5000)], 1, 1, 64, causal=False, seed=21).check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim", [64, 128])
def test_other_sequences_do_not_leak(bad, dim):
    """NaN and infinities in one sequence and behind the last reach no other."""
    lengths = [(100, 190), (130, 70), (60, 60), (129, 140)]
    _leak(lengths, dim, bad)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_long_sequences_do_not_leak(bad):
    _leak([(600, 790), (530, 570), (660, 660), (629, 840)], 128, bad)


def _leak(lengths, dim, bad, tail=150):
    c = Case(lengths, 4, 2, dim, tail=tail, seed=10)
    want = c.want()
    (q0, k0), (nq, nk) = lengths[0], lengths[1]
    for t, at, n in ((c.q, q0, nq), (c.dout, q0, nq), (c.k, k0, nk), (c.v, k0, nk)):
        t[at:at + n] = bad
    for t, which in ((c.q, 0), (c.dout, 0), (c.k, 1), (c.v, 1)):
        t[c.rows(which)[1]] = bad
    out, lse = c.forward()
    grads = c.backward(out, lse)
    keep_q = torch.ones(c.Tq, dtype=torch.bool)
    keep_k = torch.ones(c.Tk, dtype=torch.bool)
    keep_q[q0:q0 + nq] = keep_k[k0:k0 + nk] = False
    # (the poisoned sequence's own rows stand for themselves)
    for t, name, keep in ((out, "out", keep_q), (grads[0], "dq", keep_q), (grads[1], "dk", keep_k),
                          (grads[2], "dv", keep_k)):
        t[~keep] = 0
        for key in (name, f"{name}_size"):
            want[key][~keep.numpy()] = 0
    lse[:, q0:q0 + nq] = 0
    want["lse"][:, q0:q0 + nq] = 0
    c.check_forward(out, lse, want)
    c.check_backward(grads, want)


def test_without_starts_and_without_gradients_of_rows_that_see_nothing():
    c = Case([(200, 200)], 2, 2, 64, seed=11)
    out, lse = c.forward()
    o, l = B.attention(c.q, c.k, c.v, c.ws)
    assert torch.equal(o, out) and torch.equal(l, lse)
    got = B.attention_bwd(c.q, c.k, c.v, o, l, c.dout, c.ws)
    for a, b in zip(got, c.backward(out, lse)):
        assert torch.equal(a, b)
    B.check(c.ws)


def test_the_same_bits_twice_and_on_another_stream():
    c = Case([(700, 900), (130, 2000), (1, 4000)], 6, 2, 128, tail=3, seed=12)
    out, lse = c.forward()
    first = c.backward(out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2, lse2 = c.forward(stream=side)
    side.synchronize()
    again = c.backward(out2, lse2, stream=side)
    side.synchronize()
    for a, b in zip((out, lse, *first), (out2, lse2, *again)):
        assert torch.equal(a, b)


def test_captured_and_replayed_with_other_lengths():
    """The lengths are read on the device: a replayed graph takes those it finds."""
    a = Case([(130, 130), (70, 300), (0, 40)], 4, 2, 64, seed=13)
    b = Case([(50, 210), (1, 10), (149, 250)], 4, 2, 64, seed=14)
    out, lse = a.forward()
    a.backward(out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = B.attention(a.q, a.k, a.v, a.ws, **a.args)
        grads = B.attention_bwd(a.q, a.k, a.v, o, l, a.dout, a.ws, **a.args)
    for c in (a, b, a):
        want = c.forward()
        want = (*want, *c.backward(*want))
        saved = [t.clone() for t in (a.q, a.k, a.v, a.dout, a.q_starts, a.k_starts)]
        for to, t in zip((a.q, a.k, a.v, a.dout, a.q_starts, a.k_starts),
                         (c.q, c.k, c.v, c.dout, c.q_starts, c.k_starts)):
            to.copy_(t)
        graph.replay()
        for x, y in zip((o, l, *grads), want):
            assert torch.equal(x, y)
        for to, t in zip((a.q, a.k, a.v, a.dout, a.q_starts, a.k_starts), saved):
            to.copy_(t)
    B.check(a.ws)


def test_outputs_between_the_heads_of_a_packed_buffer():
    """dq, dk, dv written into one [T, 3, heads, dim] buffer."""
    c = Case([(150, 150), (60, 60)], 2, 2, 64, seed=15)
    out, lse = c.forward()
    want = c.backward(out, lse)
    packed = torch.zeros(c.Tq, 3, 2, 64, dtype=BF, device="cuda")
    got = B.attention_bwd(c.q, c.k, c.v, out, lse, c.dout, c.ws, dq=packed[:, 0], dk=packed[:, 1],
                          dv=packed[:, 2], **c.args)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dim", [40, 64, 128])
def test_what_the_keys_have_in_common_adds_nothing_to_dq(dim):
    """A row's dS sum to 0, so rounding them may cost dq 2^-8 of the sum of |dS| |k - k'| alone, k' the
    row's mean key, and of |k| only what fp32 loses (2^-11: SLACK's fp32 part twice)."""
    n, heads = 700, 2
    common = 4 * normal(31, 1, heads, dim).float()
    q, k, v, do = (normal(32 + i, n, heads, dim) for i in range(4))
    k = (k.float() + common).to(BF)
    scale = dim ** -0.5
    ws = B.Workspace(B.attention_workspace_bytes(n, n, heads, heads, dim))
    out, lse = B.attention(q, k, v, ws, causal=False)
    dq, _, _ = B.attention_bwd(q, k, v, out, lse, do, ws, causal=False)
    B.check(ws)
    for h in range(heads):
        x, y, z, g = (f64(t[:, h]) for t in (q, k, v, do))
        s = x @ y.T * scale
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        ds = p * (g @ z.T - (g * (p @ z)).sum(1, keepdims=True)) * scale
        mean = p @ y
        apart = np.stack([np.abs(ds[i]) @ np.abs(y - mean[i]) for i in range(n)])
        close(dq[:, h], ds @ y, 2.0 ** -8 * apart + 2.0 ** -11 * (np.abs(ds) @ np.abs(y)))


def test_gradients_by_differences():
    """(f(x + e d) - f(x - e d)) / 2e of f = sum dout out in direction d, on the fp64 definition
    with the kernel's gradients: they point where the definition's values go."""
    c = Case([(40, 60)], 2, 1, 32, seed=16, scale=0.2)
    _, _, grads = c.check()
    rng = np.random.default_rng(0)
    x = [f64(t) for t in (c.q, c.k, c.v)]
    do = f64(c.dout)

    def f(*x):
        return float((ops.attention(*x, c.lengths, True, 0.2)["out"] * do).sum())

    for i, g in enumerate(grads):
        d = rng.standard_normal(x[i].shape)
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + 1e-4 * d, x[i] - 1e-4 * d
        slope = (f(*up) - f(*down)) / 2e-4
        size = float(np.abs(f64(g) * d).sum())
        # each gradient is off by a few 2^-8 of its magnitudes, of random signs
        assert abs(float((f64(g) * d).sum()) - slope) <= 2.0 ** -8 * size


def test_offsets_beyond_32_bits():
    """Keys behind 2^32 elements: the last tokens of a long cache."""
    T, heads, dim = (1 << 20) + 300, 32, 128
    k = torch.zeros(T, heads, dim, dtype=BF, device="cuda")
    v = torch.zeros(T, heads, dim, dtype=BF, device="cuda")
    k[-200:], v[-200:] = normal(17, 200, heads, dim), normal(18, 200, heads, dim)
    q = normal(19, 3, heads, dim)
    q_starts = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    k_starts = torch.tensor([T - 200, T], dtype=torch.int32, device="cuda")
    ws = B.Workspace(B.attention_workspace_bytes(3, T, heads, heads, dim))
    out, lse = B.attention(q, k, v, ws, q_starts=q_starts, k_starts=k_starts)
    B.check(ws)
    near = B.attention(q, k[-200:].contiguous(), v[-200:].contiguous(), ws)
    torch.testing.assert_close(out.float(), near[0].float(), atol=2.0 ** -7, rtol=2.0 ** -7)
    torch.testing.assert_close(lse, near[1], atol=2.0 ** -10, rtol=0)
    want = ops.attention(f64(q), f64(k[-200:]), f64(v[-200:]), [(3, 200)])
    assert np.abs(f64(out) - want["out"]).max() < 0.02


def test_gradients_beyond_32_bits():
    """The last tokens of long tensors, whose other rows lie in no sequence and stay as they are."""
    T, heads, dim, n = (1 << 20) + 300, 32, 128, 200
    big = [torch.full((T, heads, dim), SENTINEL, dtype=BF, device="cuda") for _ in range(4)]
    near = [normal(seed, n, heads, dim) for seed in (21, 22, 23, 24)]     # q, dout, k, v
    k, v, dk, dv = big
    k[-n:], v[-n:] = near[2], near[3]
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    far = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    ws = B.Workspace(B.attention_workspace_bytes(n, T, heads, heads, dim))
    out, lse = B.attention(near[0], k, v, ws, q_starts=starts, k_starts=far)
    dq, _, _ = B.attention_bwd(near[0], k, v, out, lse, near[1], ws, q_starts=starts, k_starts=far,
                               dk=dk, dv=dv)
    B.check(ws)
    want = ops.attention(*map(f64, (near[0], near[2], near[3])), [(n, n)], True, None, f64(near[1]))
    for got, name in ((dq, "dq"), (dk[-n:], "dk"), (dv[-n:], "dv")):
        close(got, want[name], SLACK * want[f"{name}_size"])
    for t in (dk, dv):
        assert (t[:-n] == SENTINEL).all()


@pytest.mark.parametrize("n", [2, 40])
def test_starts_beyond_the_rows_count_as_their_bounds(n):
    c = Case([(60, 90)] * n, 4, 2, 64, seed=25)
    want = c.forward()
    grads = c.backward(*want)
    for s in (c.q_starts, c.k_starts):
        s[0], s[-1] = -7, 1 << 30
    got = c.forward()
    for a, b in zip((*want, *grads), (*got, *c.backward(*got))):
        assert torch.equal(a, b)


def test_refuses_what_the_binding_sees():
    c = Case([(10, 20)], 4, 2, 64)
    with pytest.raises(TypeError):
        B.attention(c.q.float(), c.k, c.v, c.ws)
    for kw in (dict(out=torch.empty(9, 4, 64, dtype=BF, device="cuda")),
               dict(lse=torch.empty(4, 11, device="cuda")),
               dict(q_starts=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(q_starts=c.q_starts, k_starts=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            B.attention(c.q, c.k, c.v, c.ws, **kw)
    with pytest.raises(ValueError):
        B.attention(c.q, c.k, c.v[:, :1], c.ws)
    with pytest.raises(ValueError):
        B.attention(c.q.cpu(), c.k, c.v, c.ws)
    with pytest.raises(ValueError):
        B.attention(c.q.transpose(1, 2), c.k.transpose(1, 2), c.v.transpose(1, 2), c.ws)
    with pytest.raises(TypeError):
        B.attention(c.q, c.k, c.v, c.ws, q_starts=c.q_starts.long())
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0)):
        with pytest.raises(B.BoostError):
            B.attention(c.q, c.k, c.v, c.ws, **kw)
    with pytest.raises(B.BoostError):                   # in place
        B.attention(c.q, c.k, c.v, c.ws, out=c.q)
    with pytest.raises(B.BoostError):                   # 3 query heads of 2
        B.attention(c.q[:, :3], c.k, c.v, c.ws)
    with pytest.raises(B.BoostError):                   # one key for all tokens
        B.attention(c.q, c.k[:1].expand(20, 2, 64), c.v, c.ws)
    with pytest.raises(B.BoostError):
        B.attention(c.q, c.k, c.v, B.Workspace(256))
    empty = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    assert B.attention(empty, c.k, c.v, c.ws)[0].numel() == 0
    B.check(c.ws)
