"""Attention over many sequences: single tokens over ragged contexts, and more sequences than a
warp has lanes (tolerances: attention_parity)."""

import numpy as np
import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from attention_parity import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def ragged(n, most, seed):
    """`n` lengths from 1 to `most`, spread over their logarithm, the extremes among them."""
    rng = np.random.default_rng(seed)
    return [1, most, *(int(v) for v in np.exp(rng.uniform(0, np.log(most), n - 2)))]


@pytest.mark.parametrize("sequences", [25, 26, 32, 33, 64])
@pytest.mark.parametrize("hq,hk", [(10, 2), (8, 8), (33, 1), (48, 1)])
def test_one_token_of_many_sequences(hq, hk, sequences):
    """On both sides of the queries that one tile holds."""
    c = Case([(1, n) for n in ragged(sequences, 1500, sequences)], hq, hk, 64, seed=hq)
    out, lse = c.forward()
    c.check_forward(out, lse, c.want())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sequences", [31, 32, 33, 65])
def test_more_sequences_than_lanes(sequences, dim, causal):
    """Of none to a few tiles each, queries and keys of their own lengths."""
    q, k = (ragged(sequences, 300, seed) for seed in (1, 2))
    lengths = list(zip(q[::-1], k))
    lengths[5], lengths[9], lengths[20] = (0, 40), (150, 0), (0, 0)
    Case(lengths, 2, 1, dim, causal=causal, tail=30, seed=dim).check()
