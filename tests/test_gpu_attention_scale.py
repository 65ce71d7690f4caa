"""The scale of attention's scores, in whatever form a caller has it."""

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


@pytest.mark.parametrize("make", [torch.tensor, np.float32, np.array])
def test_a_scale_that_is_no_plain_number(make):
    """The value at the time of the call counts, also of one that has changed since another call."""
    c = Case([(50, 70)], 2, 1, 64, seed=3)
    scale = make(0.5)
    for value in (0.5, 0.25):
        if isinstance(scale, np.float32):
            scale = make(value)
        else:
            scale[...] = value
        c.scale = value
        want = c.forward()
        want = (*want, *c.backward(*want))
        c.scale = scale
        got = c.forward()
        got = (*got, *c.backward(*got))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
