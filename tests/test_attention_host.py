"""Host-side tests of attention, the norm with an 8-bit output and gradient clipping (no GPU
needed): their definitions against differences and closed forms, and the refusals, which come
before any CUDA call."""

import ctypes

import numpy as np
import pytest

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


def ptr(v):
    return ctypes.c_void_p(v) if v else None


# ---------------------------------------------------------------------- the definitions
@pytest.mark.parametrize("causal", [True, False])
def test_attention_definition_against_loops_and_differences(causal):
    rng = np.random.default_rng(0)
    lengths, hq, hk, dim = [(3, 5), (4, 2), (2, 0), (0, 3)], 4, 2, 6
    q, do = (rng.standard_normal((9, hq, dim)) for _ in range(2))
    k, v = (rng.standard_normal((10, hk, dim)) for _ in range(2))
    r = ops.attention(q, k, v, lengths, causal, dout=do)
    q0 = k0 = 0
    for nq, nk in lengths:                              # row by row over the keys it sees
        for i in range(nq):
            keys = range(nk if not causal else max(0, nk - nq + 1 + i))
            for h in range(hq):
                if not keys:
                    assert (r["out"][q0 + i, h] == 0).all() and r["lse"][h, q0 + i] == -np.inf
                    assert (r["dq"][q0 + i, h] == 0).all()
                    continue
                w = np.exp([q[q0 + i, h] @ k[k0 + j, h // 2] / dim ** 0.5 for j in keys])
                o = sum(x * v[k0 + j, h // 2] for x, j in zip(w, keys)) / w.sum()
                np.testing.assert_allclose(r["out"][q0 + i, h], o, rtol=1e-12, atol=1e-13)
                np.testing.assert_allclose(r["lse"][h, q0 + i], np.log(w.sum()), rtol=1e-12)
        q0, k0 = q0 + nq, k0 + nk

    def f(q, k, v):
        return np.nansum(ops.attention(q, k, v, lengths, causal)["out"] * do)

    x = [q, k, v]
    for n, name in enumerate(("dq", "dk", "dv")):
        got = np.zeros_like(x[n])
        for at in np.ndindex(x[n].shape):
            up, down = ([t.copy() for t in x] for _ in range(2))
            up[n][at] += 1e-5
            down[n][at] -= 1e-5
            got[at] = (f(*up) - f(*down)) / 2e-5
        np.testing.assert_allclose(got, r[name], atol=1e-8)


def test_clip_definition():
    norm, g = ops.grad_clip([np.array([3.0]), np.array([0.0, 4.0])], 1.0)
    assert norm == 5 and abs(g[0][0] - 0.6) < 1e-6 and abs(g[1][1] - 0.8) < 1e-6
    assert ops.grad_clip([np.array([3.0, 4.0])], 6.0)[1][0].tolist() == [3.0, 4.0]


# ------------------------------------------------------------------ attention refusals
def desc(**kw):
    d = dict(Tq=4, Tk=6, hq=4, hk=2, dim=64, sequences=1, causal=1, scale=0.125)
    d.update({k: v for k, v in kw.items() if k in d})
    s = {}
    for x in ("q", "o", "do", "dq"):
        s |= {f"{x}_ts": 256, f"{x}_hs": 64}
    for x in ("k", "v", "dk", "dv"):
        s |= {f"{x}_ts": 128, f"{x}_hs": 64}
    s.update({k: v for k, v in kw.items() if k in s})
    return B.AttentionDesc(**d, **s)


AT = dict(q=0x10000, k=0x20000, v=0x30000, out=0x40000, lse=0x50000, dout=0x60000, dq=0x70000,
          dk=0x80000, dv=0x90000, qs=0, ks=0, ws=0x1000000)


def forward(L, D, ws_bytes=None, **kw):
    a = AT | kw
    need = L.boost_attention_workspace_bytes(ctypes.byref(D))
    return L.boost_attention(ctypes.byref(D), ptr(a["q"]), ptr(a["k"]), ptr(a["v"]), ptr(a["qs"]),
                             ptr(a["ks"]), ptr(a["out"]), ptr(a["lse"]), ptr(a["ws"]),
                             need if ws_bytes is None else ws_bytes, None)


def backward(L, D, ws_bytes=None, **kw):
    a = AT | kw
    need = L.boost_attention_workspace_bytes(ctypes.byref(D))
    return L.boost_attention_bwd(
        ctypes.byref(D), ptr(a["q"]), ptr(a["k"]), ptr(a["v"]), ptr(a["out"]), ptr(a["lse"]),
        ptr(a["dout"]), ptr(a["qs"]), ptr(a["ks"]), ptr(a["dq"]), ptr(a["dk"]), ptr(a["dv"]),
        ptr(a["ws"]), need if ws_bytes is None else ws_bytes, None)


DESCS = [
    (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID), (dict(hq=0), INVALID), (dict(hk=0), INVALID),
    (dict(hq=3), INVALID), (dict(dim=0), INVALID), (dict(sequences=0), INVALID),
    (dict(causal=2), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=2.0 ** 127 * 1.5), INVALID),
    (dict(dim=60), SHAPE), (dict(dim=136), SHAPE), (dict(Tq=1 << 31), SHAPE),
    (dict(Tk=1 << 31), SHAPE), (dict(hq=1 << 17, hk=1), SHAPE), (dict(sequences=1 << 21), SHAPE),
    (dict(Tq=1 << 30, hq=256), SHAPE),                 # too many tiles
    (dict(q_ts=-8), INVALID), (dict(k_hs=0), INVALID), (dict(v_ts=0), INVALID),
    (dict(q_hs=68), SHAPE), (dict(k_ts=1 << 40), SHAPE),
    (dict(o_hs=56), INVALID), (dict(o_ts=64), INVALID),    # heads, tokens of out coincide
    (dict(sequences=2), INVALID),                          # without starts
]


@pytest.mark.parametrize("kw,want", DESCS)
def test_attention_desc_refusals(L, kw, want):
    assert forward(L, desc(**kw)) == want


@pytest.mark.parametrize("kw,want", [d for d in DESCS if "o_hs" not in d[0] and "o_ts" not in d[0]] + [
    (dict(dq_hs=56), INVALID), (dict(dk_ts=64), INVALID), (dict(dv_ts=-8), INVALID),
    (dict(do_ts=0), INVALID), (dict(dk_hs=68), SHAPE)])
def test_attention_bwd_desc_refusals(L, kw, want):
    assert backward(L, desc(**kw)) == want


@pytest.mark.parametrize("call,names,lse", [
    (forward, ("q", "k", "v", "out"), True),
    (backward, ("q", "k", "v", "out", "dout", "dq", "dk", "dv"), False)])
def test_attention_pointer_refusals(L, call, names, lse):
    D = desc()
    for name in names:
        assert call(L, D, **{name: 0}) == INVALID, name
        assert call(L, D, **{name: AT[name] + 8}) == ALIGN, name
    assert call(L, D, lse=AT["lse"] + 2) == ALIGN
    assert call(L, D, qs=0xA0002, ks=0xB0000) == ALIGN
    assert call(L, desc(sequences=3), qs=0xA0000) == INVALID
    assert call(L, D, ws=0) == WORKSPACE
    assert call(L, D, ws=AT["ws"] + 16) == WORKSPACE
    assert call(L, D, ws_bytes=255) == WORKSPACE
    outs = ("out",) if call is forward else ("dq", "dk", "dv")
    for o in outs:
        for other in set(names + ("lse",)) - {o}:
            assert call(L, D, **{o: AT[other]}) == INVALID, (o, other)
        assert call(L, D, **{o: 0xA0000}, qs=0xA0000) == INVALID
        assert call(L, D, **{o: AT["ws"]}) == INVALID
    for i in ("q", "k", "v"):
        assert call(L, D, **{i: AT["ws"]}) == INVALID
    if lse:
        assert call(L, D, lse=AT["q"]) == INVALID
        assert call(L, D, lse=0xA0000, ks=0xA0000) == INVALID
    else:
        assert call(L, D, lse=0) == INVALID
    assert call(L, D, lse=AT["ws"] + 256) == INVALID
    zero = desc(Tq=0, Tk=0)
    assert call(L, zero, **{n: 0 for n in names}) == 0


def test_attention_workspace_bytes(L):
    assert L.boost_attention_workspace_bytes(ctypes.byref(desc(dim=60))) == 0
    assert L.boost_attention_workspace_bytes(None) == 0
    assert B.attention_workspace_bytes(100, 100, 4, 2, 64) >= 256


# ----------------------------------------------------------------- the norm's refusals
def norm(L, T=16, d=64, fmt=0, eps=1e-5, x=0x10000, res=0x20000, gamma=0x30000, h=0x40000,
         rstd=0x50000, q=0x60000, sf=0x70000):
    return L.boost_norm_quantize(T, d, fmt, eps, ptr(x), ptr(res), ptr(gamma), ptr(h), ptr(rstd),
                                 ptr(q), ptr(sf), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(fmt=2), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(d=60), SHAPE), (dict(T=1 << 32), SHAPE),
    (dict(d=1 << 26), SHAPE), (dict(x=0), INVALID), (dict(rstd=0), INVALID), (dict(q=0), INVALID),
    (dict(sf=0), INVALID), (dict(x=0x10008), ALIGN), (dict(gamma=0x30002), ALIGN),
    (dict(rstd=0x50004), ALIGN), (dict(q=0x10000), INVALID), (dict(h=0x10010), INVALID),
    (dict(h=0x30000), INVALID), (dict(rstd=0x20000), INVALID), (dict(sf=0x60000), INVALID),
    (dict(h=0x60000), INVALID), (dict(T=0, x=0, rstd=0, q=0, sf=0), 0),
])
def test_norm_refusals(L, kw, want):
    assert norm(L, **kw) == want


# ------------------------------------------------------------------ clipping's refusals
def clip(L, grads, max_norm=1.0, norm=0x900000, ws=0x1000000, ws_bytes=None, count=None):
    table = (B.Grad * max(1, len(grads)))()
    for i, g in enumerate(grads):
        table[i] = g
    return L.boost_grad_clip(len(grads) if count is None else count, table, max_norm, ptr(norm),
                             ptr(ws), L.boost_grad_clip_workspace_bytes() if ws_bytes is None
                             else ws_bytes, None)


@pytest.mark.parametrize("grads,kw,want", [
    ([(0x10000, 0x10000, -1, 0)], {}, INVALID), ([(0, 0, 4, 0)], {}, INVALID),
    ([(0x10000, 0x10000, 4, 2)], {}, INVALID), ([(0x10008, 0x10008, 4, 0)], {}, ALIGN),
    ([(0x10000, 0x20004, 4, 0)], {}, ALIGN), ([(0x10000, 0, 1 << 41, 0)], {}, SHAPE),
    ([(0x10000, 0x10000, 4, 0)], dict(max_norm=-1.0), INVALID),
    ([(0x10000, 0x10000, 4, 0)], dict(max_norm=float("nan")), INVALID),
    ([(0x10000, 0x10000, 4, 0)], dict(norm=0), INVALID),
    ([(0x10000, 0x10000, 4, 0)], dict(norm=0x900002), ALIGN),
    ([(0x10000, 0x10000, 4, 0)], dict(ws=0), WORKSPACE),
    ([(0x10000, 0x10000, 4, 0)], dict(ws=0x1000010), WORKSPACE),
    ([(0x10000, 0x10000, 4, 0)], dict(ws_bytes=256), WORKSPACE),
    ([(0x10000, 0x10000, 4, 0)], dict(norm=0x1000100), INVALID),
    ([(0x10000, 0x10000, 4, 0)], dict(norm=0x10004), INVALID),
    ([(0x10000, 0x1000100, 4, 0)], {}, INVALID),        # an output in the workspace
    ([(0x10000, 0x10010, 100, 0)], {}, INVALID),        # shifted over its own gradient
    ([(0x10000, 0x10000, 100, 0), (0x10000, 0x20000, 100, 0)], {}, INVALID),
    ([(0x10000, 0x30000, 100, 0), (0x20000, 0x30040, 100, 0)], {}, INVALID),
    ([(0x10000, 0x20000, 100, 0), (0x20000, 0x30000, 100, 0)], {}, INVALID),
    ([(0x10000, 0x10000, 4, 0)], dict(count=-1), INVALID),
])
def test_clip_refusals(L, grads, kw, want):
    assert clip(L, grads, **kw) == want
