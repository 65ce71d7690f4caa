"""Host-side tests of the operators around the block (no GPU needed): the oracle against
published and closed forms, and the refusals, which come before any CUDA call.
"""

import ctypes

import numpy as np
import pytest
import torch

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


# ---------------------------------------------------------------------- the oracle
@pytest.mark.parametrize("counter,key,want", [
    # the generator's published known answers
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(ops.philox4x32_10(counter, key)) == want


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_fp8_codes_and_rounding_match_the_formats(fmt, dtype):
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(dtype).double().numpy()
    np.testing.assert_array_equal(ops.fp8_values(fmt), codes)
    v = np.random.default_rng(0).standard_normal(5000) * np.exp2(
        np.random.default_rng(1).uniform(-20, 7, 5000))
    # halfway points, which decide the ties
    t = codes[np.isfinite(codes) & (codes >= 0)]
    v = np.concatenate([v, (t[1:] + t[:-1]) / 2, -t])
    v = v.astype(np.float32).astype(np.float64)
    v = v[np.abs(v) <= ops.FMAX[fmt]]
    np.testing.assert_array_equal(ops.fp8_round(v, fmt),
                                  torch.from_numpy(v).float().to(dtype).double().numpy())


def test_rope_oracle_far_positions():
    # a position a whole number of turns away from a near one
    w = 2 * np.pi / 4096
    near = ops.rope_angles(np.array([[5]]), [w], [0])
    far = ops.rope_angles(np.array([[5 + 4096 * 1000003]]), [w], [0])
    # w itself is rounded to 2^-53 of itself: 4.1e9 positions make that 7e-10 radians
    assert abs(np.exp(1j * near) - np.exp(1j * far)).max() < 1e-8


# ------------------------------------------------------------------- rotary refusals
def rope_desc(**kw):
    d = dict(T=4, hq=2, hk=1, dim=64, rot=64, axes=1, interleaved=0, inverse=0, pos64=0)
    d.update({k: v for k, v in kw.items() if k in d})
    hq, hk, dim = d["hq"], d["hk"], d["dim"]
    s = dict(q_ts=hq * dim, q_hs=dim, k_ts=hk * dim, k_hs=dim, qo_ts=hq * dim, qo_hs=dim,
             ko_ts=hk * dim, ko_hs=dim)
    s.update({k: v for k, v in kw.items() if k in s})
    D = B.RopeDesc(**d, **s)
    for i, a in enumerate(kw.get("axis", [])):
        D.axis[i] = a
    return D


def rope_call(L, D, q=0x10000, k=0x20000, pos=0x30000, w=0x40000, qo=0x50000, ko=0x60000):
    return L.boost_rope(ctypes.byref(D), ptr(q), ptr(k), ptr(pos), ptr(w), ptr(qo), ptr(ko), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(hq=0), INVALID), (dict(hk=-1), INVALID), (dict(rot=0), INVALID),
    (dict(rot=72), INVALID), (dict(axes=0), INVALID), (dict(axes=9), INVALID),
    (dict(interleaved=2), INVALID), (dict(inverse=-1), INVALID), (dict(pos64=2), INVALID),
    (dict(axis=[0, 1]), INVALID),                      # an axis that is not there
    (dict(q_ts=-64), INVALID),
    (dict(dim=60, rot=56), SHAPE), (dict(rot=60), SHAPE), (dict(dim=520, rot=64), SHAPE),
    (dict(q_hs=68), SHAPE), (dict(ko_ts=68), SHAPE), (dict(T=1 << 31), SHAPE),
    (dict(T=1 << 30, q_ts=1 << 40), SHAPE),            # offsets that do not fit
    (dict(qo_hs=56), INVALID),                         # heads of an output overlap
    (dict(qo_ts=64), INVALID),                         # tokens of an output overlap
    (dict(ko_ts=0), INVALID),
])
def test_rope_desc_refusals(L, kw, want):
    assert rope_call(L, rope_desc(**kw)) == want


def test_rope_pointer_refusals(L):
    D = rope_desc()
    for name in ("q", "k", "pos", "w", "qo", "ko"):
        assert rope_call(L, D, **{name: 0}) == INVALID, name
    for name in ("q", "k", "pos", "w", "qo", "ko"):
        assert rope_call(L, D, **{name: 0x70008}) == ALIGN, name
    assert L.boost_rope(None, *([None] * 7)) == INVALID
    assert rope_call(L, rope_desc(hk=0)) == INVALID     # k without heads
    assert rope_call(L, rope_desc(T=0), q=0, k=0, pos=0, w=0, qo=0, ko=0) == 0


def test_rope_overlap_refusals(L):
    D = rope_desc()                                     # q: 4 x 128 values, k: 4 x 64
    assert rope_call(L, D, qo=0x10010) == INVALID       # shifted over its input
    assert rope_call(L, D, ko=0x10000) == INVALID       # k_out over q
    assert rope_call(L, D, ko=0x50000) == INVALID       # both outputs in one place
    assert rope_call(L, D, qo=0x20000) == INVALID       # q_out over k
    assert rope_call(L, D, qo=0x30000) == INVALID       # over the positions
    assert rope_call(L, D, ko=0x40000) == INVALID       # over the frequencies
    # in place but with other strides
    assert rope_call(L, rope_desc(qo_ts=256), qo=0x10000) == INVALID
    # packed [T, 3, 64]: k_out reaching into q's heads
    packed = dict(q_ts=192, k_ts=192, qo_ts=192, ko_ts=192)
    assert rope_call(L, rope_desc(**packed), q=0x10000, k=0x10100, qo=0x50000, ko=0x50080) == INVALID
    # k_out in the rows of the input's q heads
    assert rope_call(L, rope_desc(**packed), q=0x10000, k=0x10100, qo=0x50000, ko=0x10080) == INVALID


# ------------------------------------------------------------------ dropout refusals
def drop_call(L, count=64, x=0x10000, res=0x20000, out=0x30000, p=0.1, counter=0):
    return L.boost_dropout(count, ptr(x), ptr(res), ptr(out), p, 1, 2, ptr(counter), None)


@pytest.mark.parametrize("kw,want", [
    (dict(count=-1), INVALID), (dict(p=1.0), INVALID), (dict(p=-0.1), INVALID),
    (dict(p=float("nan")), INVALID), (dict(p=1e-6), INVALID), (dict(p=1 - 1e-6), INVALID),
    (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(x=0x10008), ALIGN),
    (dict(res=0x20002), ALIGN), (dict(out=0x30004), ALIGN), (dict(counter=0x40004), ALIGN),
    (dict(out=0x10010), INVALID), (dict(out=0x20010), INVALID),   # shifted over an input
    (dict(counter=0x30008), INVALID), (dict(count=1 << 42), SHAPE),
    (dict(count=0, x=0, res=0, out=0), 0),
])
def test_dropout_refusals(L, kw, want):
    assert drop_call(L, **kw) == want


# ------------------------------------------------------------------- 8-bit refusals
def quant_call(L, G=1, rows=16, cols=64, ldx=64, gstride=0, fmt=0, block_rows=1, x=0x10000, gamma=0,
               q=0x20000, sf=0x30000, qt=0x40000, sft=0x50000):
    D = B.Fp8QuantDesc(G, rows, cols, ldx, gstride, fmt, block_rows)
    return L.boost_fp8_quantize(ctypes.byref(D), ptr(x), ptr(gamma), ptr(q), ptr(sf), ptr(qt),
                                ptr(sft), None)


@pytest.mark.parametrize("kw,want", [
    (dict(G=0), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(fmt=2), INVALID),
    (dict(block_rows=64), INVALID), (dict(ldx=-8), INVALID), (dict(cols=60), SHAPE),
    (dict(ldx=68), SHAPE), (dict(gstride=4), SHAPE), (dict(G=70000), SHAPE),
    (dict(rows=1 << 32), SHAPE), (dict(sf=0), INVALID), (dict(qt=0), INVALID),
    (dict(q=0, sf=0, qt=0, sft=0), INVALID), (dict(x=0), INVALID), (dict(x=0x10008), ALIGN),
    (dict(q=0x20008), ALIGN), (dict(sft=0x50004), ALIGN), (dict(q=0x10000), INVALID),
    (dict(sf=0x20010), INVALID), (dict(qt=0x30000), INVALID),
    (dict(gamma=0x60000, qt=0, sft=0), INVALID),       # a fold needs the tiled layouts
    (dict(rows=0), 0),
])
def test_fp8_quantize_refusals(L, kw, want):
    assert quant_call(L, **kw) == want


def test_fp8_scale_bytes(L):
    for rows, K in ((1, 1), (128, 512), (129, 513), (0, 4), (4, 0), (300, 11008)):
        assert B.fp8_scale_bytes(rows, K) == L.boost_fp8_scale_bytes(rows, K)
    assert B.fp8_scale_bytes(1, 1) == 512
    assert B.fp8_scale_bytes(128, 512) == 512
    assert B.fp8_scale_bytes(129, 513) == 2048
    assert B.fp8_scale_bytes(0, 4) == B.fp8_scale_bytes(4, 0) == 0


def matmul_call(L, G=1, M=16, N=64, K=64, a_pitch=64, b_pitch=64, fa=0, fb=0, act=0, a=0x10000,
                asf=0x20000, b=0x30000, bsf=0x40000, rs=0, out=0x50000, ws=0x1000000, ws_bytes=None):
    D = B.Fp8MatmulDesc(G, M, N, K, a_pitch, b_pitch, fa, fb, act)
    need = L.boost_fp8_matmul_workspace_bytes(ctypes.byref(D))
    return L.boost_fp8_matmul(ctypes.byref(D), ptr(a), ptr(asf), ptr(b), ptr(bsf), ptr(rs), ptr(out),
                              ptr(ws), need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(G=0), INVALID), (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=-1), INVALID),
    (dict(fa=2), INVALID), (dict(fb=-1), INVALID), (dict(act=3), INVALID),
    (dict(a_pitch=48), INVALID), (dict(b_pitch=72), SHAPE), (dict(N=60), SHAPE),
    (dict(G=70000), SHAPE), (dict(M=1 << 31), SHAPE), (dict(N=1 << 21), SHAPE),
    (dict(M=1 << 30, K=2048, a_pitch=2048, b_pitch=2048), SHAPE),      # a matrix of 2^41 bytes
    (dict(M=1 << 29, N=2048), SHAPE),                                  # an output of 2^41 bytes
    (dict(G=60000, M=1 << 20, N=128), SHAPE),                          # too many tiles
    (dict(a=0), INVALID), (dict(bsf=0), INVALID), (dict(out=0), INVALID),
    (dict(a=0x10008), ALIGN), (dict(rs=0x60004), ALIGN), (dict(out=0x50002), ALIGN),
    (dict(ws=0), WORKSPACE), (dict(ws=0x1000010), WORKSPACE), (dict(ws_bytes=128), WORKSPACE),
    (dict(out=0x10000), INVALID), (dict(ws=0x50000), INVALID), (dict(M=0), 0),
])
def test_fp8_matmul_refusals(L, kw, want):
    assert matmul_call(L, **kw) == want
