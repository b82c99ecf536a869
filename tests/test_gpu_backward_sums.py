"""The sums of the attention's backward pass, row by row: where many CTAs add to the same cache rows, a
missing or doubled addition shows."""

import pytest
import torch

from sparse_mla_attention_top_gb300 import workloads as W
from tests import _backward_sums as B

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_mla_attention_top_gb300 as S
    from sparse_mla_attention_top_gb300 import build

    build.build()
    return S


def check(S, q, cache, slots, dout, dlse=None, runs=3):
    n = cache.shape[0]
    kv = S.KVCache(cache.cuda(), n, 1, W.KV_BF16)
    qd, td, dd = q.cuda(), slots.cuda(), dout.cuda()
    out, lse = S.sparse_mla_decode(qd, kv, td, SCALE, num_splits=1)
    ws = S.Workspace()
    got = [S.sparse_mla_backward(qd, kv, td, SCALE, out, lse, dd, dlse=None if dlse is None else dlse.cuda(), ws=ws)
           for _ in range(runs)]
    assert ws.read_status() == 0
    dq, dkv, tq, tkv = B.rows(q, cache, slots, SCALE, out.cpu(), lse.cpu(), dout, dlse)
    for gq, gkv, _ in got:
        for name, g, ref, tol in (("dq", gq, dq, tq), ("dkv", gkv, dkv, tkv)):
            bad, worst = B.off(g, ref, tol)
            assert bad == 0, f"{name}: {bad} rows off, the worst by {worst:.3g} tolerances"
            # all rows together: the roundings' root mean square, 1.2 for its spread over the mantissas' steps
            rms = float(((g.double().cpu() - ref) ** 2).sum().sqrt())
            assert rms <= 1.2 * float((tol ** 2).sum().sqrt()) / 3


def lists(seed, T, K, num, dead=0.2, ordered=False):
    g = torch.Generator().manual_seed(seed)
    out = torch.full((T, K), -1, dtype=torch.int32)
    for t in range(T):
        m = min(K, num)
        pick = torch.randperm(num, generator=g)[:m]
        out[t, :m] = (pick.sort().values if ordered else pick).to(torch.int32)
    out[torch.rand((T, K), generator=g) < dead] = -1
    return out


@pytest.mark.parametrize("ordered", [False, True])
@pytest.mark.parametrize("T,H,K,num", [
    (170, 16, 600, 700), (190, 32, 129, 1200), (37, 33, 1100, 1200), (200, 128, 130, 300), (321, 64, 70, 90),
    (64, 65, 200, 200), (300, 8, 64, 64), (153, 1, 64, 700)])
def test_backward_sums_of_many_lists(S, T, H, K, num, ordered):
    g = torch.Generator().manual_seed(7)
    normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    q, cache, dout = normal(T, H, 576), normal(num, 576), normal(T, H, 512)
    check(S, q, cache, lists(8, T, K, num, ordered=ordered), dout, torch.randn((T, H), generator=g))


def test_backward_sums_of_a_row_that_every_list_holds(S):
    """One cache row in all of 2000 lists, and one in each list alone."""
    T, H = 2000, 16
    g = torch.Generator().manual_seed(9)
    normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    slots = torch.stack([torch.zeros(T, dtype=torch.int32), torch.arange(1, T + 1, dtype=torch.int32)], 1)
    check(S, normal(T, H, 576), normal(T + 1, 576), slots, normal(T, H, 512))
