"""Sizes that the 8-bit quantiser refuses, one beyond those that it takes (no GPU needed: a
refused call launches nothing)."""

import ctypes

import pytest

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

SHAPE = 2


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


@pytest.mark.parametrize("outputs", [(1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_one_row_too_many(L, block_rows, outputs):
    D = B.Fp8QuantDesc(1, 2097121, 8, 8, 0, 0, block_rows)
    p = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(5)]
    q, sf = p[1:3] if outputs[0] else (None, None)
    qt, sft = p[3:5] if outputs[1] else (None, None)
    assert L.boost_fp8_quantize(ctypes.byref(D), p[0], None, q, sf, qt, sft, None) == SHAPE
