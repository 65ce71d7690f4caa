"""Rotary positions of q and k that are packed head by head, in place."""

import pytest
import torch

from rank_bottleneck_online_gb300 import binding as B
from rank_bottleneck_online_gb300 import build as build_mod

from ops_parity import BF, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    B.lib()


def parts(layout, whole, T, H, D):
    """q, k and v [T, H, D] as they lie in one buffer."""
    shape = {"token_head_part": (T, H, 3, D), "head_part_token": (H, 3, T, D),
             "part_token_head": (3, T, H, D), "token_part_head": (T, 3, H, D),
             "part_head_token": (3, H, T, D), "head_token_part": (H, T, 3, D)}[layout]
    names = layout.split("_")
    order = [names.index(n) for n in ("part", "token", "head")] + [3]
    return whole.view(shape).permute(order).unbind(0)


LAYOUTS = ("token_head_part", "head_part_token", "part_token_head", "token_part_head",
           "part_head_token", "head_token_part")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H", [(1, 1), (1, 5), (37, 1), (37, 4)])
def test_in_place(layout, T, H):
    D = 64
    whole = normal(1, T * H * 3 * D)
    q, k, v = parts(layout, whole, T, H, D)
    pos = torch.arange(7, 7 + T, dtype=torch.int32, device="cuda")
    w = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    want = B.rope(q, k, pos, w)
    value = v.clone()
    B.rope(q, k, pos, w, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, value)


@pytest.mark.parametrize("T", [1, 20])
def test_into_the_other_parts(T):
    """Outputs between the heads of their inputs; one key head among several query heads."""
    H, D = 4, 64
    whole = normal(2, T * H * 3 * D)
    q, k, v = parts("token_head_part", whole, T, H, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    w = torch.linspace(0, 1, D // 2, dtype=torch.float64, device="cuda")
    want = B.rope(q, k[:, :1], pos, w)
    before = k.clone()
    B.rope(q, k[:, :1], pos, w, q_out=v, k_out=k[:, 1:2])
    assert torch.equal(v, want[0]) and torch.equal(k[:, 1:2], want[1])
    assert torch.equal(k[:, ::2], before[:, ::2])


def test_still_refuses_what_shares_elements():
    T, H, D = 20, 4, 64
    whole = normal(3, T * H * 3 * D + 64)
    q, k, _ = parts("token_head_part", whole[:-64], T, H, D)
    shifted = parts("token_head_part", whole[8:-56], T, H, D)
    later = parts("token_head_part", whole[192 * H:][:T // 2 * H * 3 * D], T // 2, H, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    w = torch.ones(D // 2, dtype=torch.float64, device="cuda")
    for q_out, k_out in ((k, q), (shifted[0], k), (q, shifted[1]), (q, q), (shifted[2], k)):
        with pytest.raises(B.BoostError):
            B.rope(q, k, pos, w, q_out=q_out, k_out=k_out)
    with pytest.raises(B.BoostError):                  # a token further on in the same buffer
        B.rope(q[:T // 2], None, pos[:T // 2], w, q_out=later[0])
