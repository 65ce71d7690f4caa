"""Where rotary positions begin in a table: the descriptor's layout, and what it refuses (no
GPU needed: a refused call launches nothing)."""

import ctypes
import os
import shutil
import subprocess

import pytest

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

INVALID, SHAPE, ALIGN = 1, 2, 3
POS, OUT = 0x30000, 0x50000


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


def call(L, pos=POS, **kw):
    """q [4, 2, 64] at 0x10000, its output (1 KB) at OUT."""
    D = B.RopeDesc(T=4, hq=2, dim=64, rot=64, q_ts=128, q_hs=64, qo_ts=128, qo_hs=64,
                   **{"axes": 1, **kw})
    return L.boost_rope(ctypes.byref(D), 0x10000, None, pos, 0x40000, OUT, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(pos_at=-1), INVALID), (dict(axes=2, pos_as=-4), INVALID), (dict(axes=2, pos_as=3), INVALID),
    (dict(pos_at=1 << 51), SHAPE), (dict(axes=2, pos_as=1 << 51), SHAPE), (dict(pos=POS + 4), ALIGN),
    # positions that lie in the output, although the table begins elsewhere
    (dict(pos=OUT - 64, pos_at=16), INVALID), (dict(pos=OUT - 64, pos_at=13), INVALID),
    (dict(pos=OUT - 64, pos_at=7, pos64=1), INVALID),
    (dict(pos=OUT - 4096, axes=3, pos_as=512), INVALID),
])
def test_refusals(L, kw, want):
    assert call(L, **kw) == want


def test_the_descriptor_is_the_headers(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no host compiler")
    names = [f for f, _ in B.RopeDesc._fields_]
    code = '#include <stdio.h>\n#include <stddef.h>\n#include "boost_ops.h"\nint main(void) {\n'
    code += "".join(f'printf("%zu ", offsetof(boost_rope_desc, {n}));' for n in names)
    code += 'printf("%zu", sizeof(boost_rope_desc)); return 0; }\n'
    out = str(tmp_path / "layout")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-std=c11", "-x", "c", "-", "-I", include, "-o", out], input=code, text=True,
                   check=True)
    got = [int(v) for v in subprocess.run([out], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(B.RopeDesc, n).offset for n in names] + [ctypes.sizeof(B.RopeDesc)]
