"""Rotary positions taken from inside a table of positions, as a decoding step takes them."""

import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod
from rank_bottleneck_online_gb300.block import Rotary

from ops_parity import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def freq(pairs):
    return 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T", [1, 3, 50])
@pytest.mark.parametrize("first", [0, 1, 2, 3, 4, 5, 70])
def test_slices_of_a_vector(first, T, dtype):
    table = torch.randint(0, 9000, (200,), dtype=dtype, device="cuda")
    q, k, w = normal(1, T, 4, 64), normal(2, T, 2, 64), freq(32)
    got = B.rope(q, k, table[first:first + T], w)
    want = B.rope(q, k, table[first:first + T].clone(), w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T", [1, 3, 50])
@pytest.mark.parametrize("first", [0, 1, 70])
def test_columns_of_a_table_with_several_axes(first, T, dtype):
    table = torch.randint(0, 9000, (3, 201), dtype=dtype, device="cuda")
    part = table[:, first:first + T]
    q, w = normal(1, T, 4, 64), freq(32)
    got, _ = B.rope(q, None, part, w, sections=[8, 12, 12])
    want, _ = B.rope(q, None, part.clone().contiguous(), w, sections=[8, 12, 12])
    assert torch.equal(got, want)


def test_a_decoding_step_of_the_layers_positions():
    rotary = Rotary(64)
    table = torch.arange(32, dtype=torch.int32, device="cuda")
    q = normal(4, 32, 256)
    want, _ = rotary(q, None, table)
    for t in range(32):
        got, _ = rotary(q[t:t + 1], None, table[t:t + 1])
        assert torch.equal(got, want[t:t + 1])


def test_refuses_other_strides():
    q, w = normal(5, 10, 2, 64), freq(32)
    table = torch.zeros(2, 40, dtype=torch.int32, device="cuda")
    for bad in (table[0, :20:2], table[:, :20:2], table[0, :1].expand(10), table[:1, :10].expand(2, 10)):
        with pytest.raises(ValueError):
            B.rope(q, None, bad, w)
