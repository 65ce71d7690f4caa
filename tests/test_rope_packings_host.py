"""Host checks of rotary positions of q and k in one buffer (no GPU needed): operands that
share an element are refused in every packing. Calls that are refused launch nothing."""

import ctypes
import itertools

import pytest

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

INVALID = 1
BASE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


def elements(at, T, heads, dim, ts, hs):
    return {at + t * ts + h * hs + d for t in range(T) for h in range(heads) for d in range(dim)}


def call(L, T, hq, hk, dim, places, strides):
    """Offsets of q, k, q_out and k_out in elements from one base."""
    D = B.RopeDesc(T=T, hq=hq, hk=hk, dim=dim, rot=dim, axes=1)
    for (ts, hs), a, b in zip(strides, ("q_ts", "k_ts", "qo_ts", "ko_ts"),
                              ("q_hs", "k_hs", "qo_hs", "ko_hs")):
        setattr(D, a, ts)
        setattr(D, b, hs)
    p = [ctypes.c_void_p(BASE + 2 * at) for at in places]
    return L.boost_rope(ctypes.byref(D), p[0], p[1], ctypes.c_void_p(1 << 12),
                        ctypes.c_void_p(1 << 13), p[2], p[3], None)


@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 3, 3), (3, 1, 1), (3, 3, 3), (3, 3, 1), (2, 2, 3)])
@pytest.mark.parametrize("token_first", [True, False])
def test_shared_elements_are_refused(L, T, hq, hk, token_first):
    """q_out at every offset around k in a packed buffer, k in place: where they meet."""
    dim, heads = 16, max(hq, hk)
    st = (heads * 3 * dim, 3 * dim) if token_first else (3 * dim, T * 3 * dim)
    strides = [(heads * 64 * dim * T, 64 * dim), st, st, st]
    k_at, span, refused = 1024, 3 * dim * heads * T, 0
    taken = elements(k_at, T, hk, dim, *st)
    for at in range(max(k_at - span, 0), k_at + span, 8):
        if taken & elements(at, T, hq, dim, *st):
            refused += 1
            assert call(L, T, hq, hk, dim, (1 << 16, k_at, at, k_at), strides) == INVALID, at
    assert refused
