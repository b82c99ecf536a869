"""That the row by row check of the backward pass sees what it is for: mistakes planted in the oracle."""

import pytest
import torch

from tests import _backward_sums as B
from tests import _layer_ref as R

SCALE = 576 ** -0.5


def case(seed, T, H, K, num, dead=0.2):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    q, cache, dout = normal(T, H, 576), normal(num, 576), normal(T, H, 512)
    slots = torch.full((T, K), -1, dtype=torch.int32)
    for t in range(T):
        m = min(K, num)
        slots[t, :m] = torch.randperm(num, generator=g)[:m].to(torch.int32)
    slots[torch.rand((T, K), generator=g) < dead] = -1
    out, lse = torch.zeros(T, H, 512), torch.full((T, H), -float("inf"))
    for t in range(T):
        at = slots[t][slots[t] >= 0].long()
        if len(at):
            o, l = R.attention(q[t].double(), cache[at].double(), SCALE)
            out[t], lse[t] = o.float(), l.float()
    return q, cache, slots, SCALE, out.to(torch.bfloat16), lse, dout


@pytest.mark.parametrize("T,H,K,num", [(60, 16, 300, 350), (40, 66, 129, 200), (3, 1, 5, 8)])
def test_the_stated_roundings_pass(T, H, K, num):
    args = case(1, T, H, K, num)
    dq, dkv, tq, tkv = B.rows(*args)
    gq, gkv, _, _ = B.rows(*args, bf16_operands=True)
    assert B.off(gq, dq, tq)[0] == 0 and B.off(gkv, dkv, tkv)[0] == 0


@pytest.mark.parametrize("columns", [slice(0, 576), slice(0, 512), slice(128, 160), slice(512, 576)])
def test_one_lost_addition_does_not(columns):
    """Of about 130 additions to a cache row, one whole, its latent columns, 32 of them, or its rope columns."""
    args = case(2, 160, 16, 300, 300)
    slots = args[2]
    t, entry = 77, int(torch.nonzero(slots[77] >= 0)[40])
    none = slice(0, 0)
    _, dkv, _, tol = B.rows(*args)
    _, got, _, _ = B.rows(*args, bf16_operands=True, skip=lambda a, b: columns if (a, b) == (t, entry) else none)
    err = (got - dkv).norm(dim=-1) > tol
    assert err.nonzero().flatten().tolist() == [int(slots[t, entry])]
