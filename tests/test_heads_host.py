"""Where [T, heads, dim] operands lie in memory (csrc/heads.h, host code): operands of unequal
numbers of tokens and heads that share an element are found, and those that lie between each
other's are told apart, in either order of the two. Against sets of elements."""

import ctypes
import itertools
import os
import subprocess

import pytest

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

INVALID = 1
WRAP = """
#include "heads.h"
using boost_gb300::Slice;
extern "C" int share_no_element(const int64_t* a, const int64_t* b) {
  const Slice x{static_cast<uintptr_t>(a[0]), a[1], a[2], a[3], a[4], a[5]};
  const Slice y{static_cast<uintptr_t>(b[0]), b[1], b[2], b[3], b[4], b[5]};
  return boost_gb300::disjoint(x, y);
}
"""


@pytest.fixture(scope="module")
def disjoint(tmp_path_factory):
    at = tmp_path_factory.mktemp("heads")
    (at / "wrap.cpp").write_text(WRAP)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    build_mod.CSRC, str(at / "wrap.cpp"), "-o", str(at / "wrap.so")], check=True)
    f = ctypes.CDLL(str(at / "wrap.so")).share_no_element

    def call(a, b):
        x, y = (((ctypes.c_int64 * 6)(1 << 20, *s[1:])) for s in (a, b))
        x[0] += 2 * a[0]
        y[0] += 2 * b[0]
        return bool(f(x, y))

    return call


def elements(at, T, heads, dim, ts, hs):
    return {at + t * ts + h * hs + d for t in range(T) for h in range(heads) for d in range(dim)}


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


@pytest.mark.parametrize("Ta,Tb", [(1, 1), (1, 5), (2, 5), (3, 3), (4, 1)])
@pytest.mark.parametrize("ha,hb", [(1, 1), (1, 3), (2, 3), (3, 3), (4, 2)])
@pytest.mark.parametrize("rows", [True, False])
def test_as_the_sets_of_elements_say(disjoint, Ta, Tb, ha, hb, rows):
    """Operands of one packed buffer, one at every offset around the other: by rows of the heads
    and 3 more ([T, heads + 3, dim]), or head by head, of 2 rows more than the larger."""
    dim = 8
    ts, hs = ((max(ha, hb) + 3) * dim, dim) if rows else (dim, (max(Ta, Tb) + 2) * dim)
    span = (Ta + Tb) * ts + (ha + hb) * hs
    fixed = elements(0, Ta, ha, dim, ts, hs)
    met = apart = 0
    for at in range(-span, span + 1, 8):
        share = bool(fixed & elements(at, Tb, hb, dim, ts, hs))
        a, b = (0, Ta, ha, dim, ts, hs), (at, Tb, hb, dim, ts, hs)
        assert disjoint(a, b) is not share, at
        assert disjoint(b, a) is not share, at
        met, apart = met + share, apart + (not share)
    assert met and apart


def test_other_strides_never_hide_a_shared_element(disjoint):
    """Strides that differ may be refused though nothing is shared, never the other way round."""
    dim = 8
    of = [(T, h, dim, ts, hs) for T, h in itertools.product((1, 2, 4), (1, 3))
          for ts, hs in ((24, 8), (32, 8), (8, 32), (8, 40), (40, 16))]
    for x, y in itertools.product(of, of):
        mine = elements(0, *x)
        for at in range(-136, 137, 8):
            if mine & elements(at, *y):
                assert not disjoint((0, *x), (at, *y)) and not disjoint((at, *y), (0, *x)), (x, y, at)


AT = dict(q=1 << 24, out=2 << 24, dout=3 << 24, dq=4 << 24, k=5 << 24, v=6 << 24, dk=7 << 24,
          dv=8 << 24, lse=9 << 24, ws=1 << 30)


def calls(L, Tq, Tk, at, heads, dim):
    """The statuses of the forward and the backward with operands [T, heads, dim] at `at`."""
    D = B.AttentionDesc(Tq, Tk, heads, heads, dim, 1, 1, 1.0, *(heads * dim, dim) * 8)
    need = L.boost_attention_workspace_bytes(ctypes.byref(D))
    p = {n: ctypes.c_void_p(v) for n, v in (AT | at).items()}
    fwd = L.boost_attention(ctypes.byref(D), p["q"], p["k"], p["v"], None, None, p["out"], p["lse"],
                            p["ws"], need, None) if "out" in at else None
    bwd = L.boost_attention_bwd(ctypes.byref(D), p["q"], p["k"], p["v"], p["out"], p["lse"], p["dout"],
                                None, None, p["dq"], p["dk"], p["dv"], p["ws"], need,
                                None) if "out" not in at else None
    return fwd, bwd


@pytest.mark.parametrize("Tq", [1, 10, 400])
@pytest.mark.parametrize("row", [0, 1, 500, 599, 999])
def test_outputs_in_later_rows_of_longer_operands_are_refused(L, Tq, row):
    """Calls that are refused launch nothing."""
    heads, dim, Tk = 2, 64, 1000
    for other in ("k", "v"):
        at = AT[other] + 2 * row * heads * dim
        assert calls(L, Tq, Tk, dict(out=at), heads, dim)[0] == INVALID
        assert calls(L, Tq, Tk, dict(dq=at), heads, dim)[1] == INVALID
    for other in ("dk", "dv"):
        assert calls(L, Tq, Tk, dict(dq=AT[other] + 2 * row * heads * dim), heads, dim)[1] == INVALID
    # and of shorter ones: q and dout behind the first rows of dk
    for other in ("q", "dout"):
        at = AT[other] - 2 * row * heads * dim
        assert calls(L, Tq, Tk, dict(dk=at), heads, dim)[1] == INVALID
