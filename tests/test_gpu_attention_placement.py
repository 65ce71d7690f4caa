"""Attention's operands in one buffer, unequal numbers of queries and keys: outputs between inputs,
which share no element, and overlaps, which are refused."""

import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from attention_parity import Case
from ops_parity import BF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


@pytest.mark.parametrize("nq,nk", [(1, 300), (10, 300), (300, 10), (140, 140)])
def test_gradients_side_by_side_head_by_head(nq, nk):
    """dq, then dk, then dv in the rows of one [heads, nq + 2 nk, dim] buffer."""
    heads, dim = 2, 64
    c = Case([(nq, nk)], heads, heads, dim, seed=nq)
    out, lse = c.forward()
    want = c.backward(out, lse)
    whole = torch.zeros(heads, nq + 2 * nk, dim, dtype=BF, device="cuda").transpose(0, 1)
    got = B.attention_bwd(c.q, c.k, c.v, out, lse, c.dout, c.ws, dq=whole[:nq],
                          dk=whole[nq:nq + nk], dv=whole[nq + nk:], **c.args)
    B.check(c.ws)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("by_heads", [True, False])
def test_a_cache_with_the_new_tokens_rows_behind_it(by_heads):
    """Keys, values, queries and their result in rows of one buffer."""
    nq, nk, heads, dim = 3, 200, 2, 64
    c = Case([(nq, nk)], heads, heads, dim, seed=4)
    want = c.forward()
    rows = 2 * nk + 2 * nq
    whole = torch.zeros((heads, rows, dim) if by_heads else (rows, heads, dim), dtype=BF, device="cuda")
    if by_heads:
        whole = whole.transpose(0, 1)
    k, v, q, out = whole.split([nk, nk, nq, nq])
    for to, t in ((k, c.k), (v, c.v), (q, c.q)):
        to.copy_(t)
    got = B.attention(q, k, v, c.ws, out=out, **c.args)
    B.check(c.ws)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for row in (0, 1, nk - nq, nk - 1, nk, 2 * nk - 1, 2 * nk):
        with pytest.raises(B.BoostError):
            B.attention(q, k, v, c.ws, out=whole[row:row + nq], **c.args)
