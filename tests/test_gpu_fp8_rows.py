"""The 8-bit quantiser at its largest number of rows."""

import pytest
import torch

from oracle import ops
from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF, f64, guarded

pytestmark = pytest.mark.gpu

MOST = 2097120                                          # 65535 lines of 32 rows


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows", [MOST - 96, MOST - 95, MOST - 32, MOST - 31, MOST])
def test_rows_alone_to_the_limit(rows, fmt):
    """What the tile kernel gives, which holds 128 rows a block: values, scales and the bytes of
    the last tile's missing rows; and the definition over the last rows."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, 8, generator=g, device="cuda").to(BF)
    q, whole_q = guarded((rows, 16), B.FP8_FORMATS[fmt][1])
    sf, whole_s = guarded((B.fp8_scale_bytes(rows, 8),), torch.uint8)
    B.fp8_quantize(x, fmt=fmt, rows_out=(q, sf))
    assert whole_q() and whole_s()
    (want_q, want_sf), _ = B.fp8_quantize(x, fmt=fmt, way="both")
    assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(sf, want_sf)
    first = MOST - 96                                   # the last tile's first row
    tail = x[first - 128:]
    values, e = ops.fp8_quantize(f64(tail), fmt)
    assert (f64(q[first - 128:])[:, :8] == values).all()
    assert (sf[-1024:].cpu().numpy() == ops.fp8_scales(e)).all() if rows > first else True


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 95, 96, 97, 129, 225])
@pytest.mark.parametrize("cols", [8, 520])
def test_missing_rows_of_the_last_tile(rows, cols):
    """Lines of 32 rows that the last tile lacks have scale bytes of 127 in every block."""
    x = torch.randn(2, rows, cols, device="cuda").to(BF)
    sf = torch.zeros(2, B.fp8_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    q = torch.empty(2, rows, -(-cols // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")
    B.fp8_quantize(x, rows_out=(q, sf))
    for m in range(2):
        _, e = ops.fp8_quantize(f64(x[m]), "e4m3")
        assert (sf[m].cpu().numpy() == ops.fp8_scales(e)).all()
