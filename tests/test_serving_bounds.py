"""The bounds of the serving operators' tests: mistakes planted in the oracle, on the CPU, that they have to tell."""

import numpy as np
import pytest
import torch

from tests import _serving_ref as R

SCALE = 2.0 ** -8


def inputs(kind, n, T=6, H=5, seed=0):
    g = torch.Generator()
    g.manual_seed(seed)
    if kind == "bf16":
        cache = torch.randn((n, 576), generator=g).to(torch.bfloat16).view(torch.uint8)
    else:
        cache = torch.cat([torch.randn((n, 512), generator=g).to(torch.float8_e4m3fn).view(torch.uint8),
                           (torch.rand((n, 4), generator=g) * 1.5 + 0.5).view(torch.uint8),
                           torch.randn((n, 64), generator=g).to(torch.bfloat16).view(torch.uint8)], 1).contiguous()
    q, cache = R.whole_numbers(torch.randn((T, H, 576), generator=g), cache, kind)
    return q, cache, [np.arange(n)] * T


def lse_in_32_bits(q, cache, lists, kind, parts=1):
    """As the operator computes it: block sums, their scales in fp32, base 2."""
    f, lse = torch.float32, []
    for t, ls in enumerate(lists):
        k = cache[torch.as_tensor(ls)]
        if kind == "bf16":
            s = q[t].to(f) @ k.view(torch.bfloat16).to(f).T
        else:
            codes, sc = k[:, :512].view(torch.float8_e4m3fn).to(f), k[:, 512:528].view(f)
            s = torch.zeros((q.shape[1], len(ls)))
            for c in range(4):
                s = s + (q[t, :, 128 * c:128 * c + 128].to(f) @ codes[:, 128 * c:128 * c + 128].T) * sc[:, c]
            s = s + q[t, :, 512:].to(f) @ k[:, 528:].view(torch.bfloat16).to(f).T
        y = s * torch.tensor(SCALE * 1.4426950408889634, dtype=f)
        ends = []
        for part in y.chunk(parts, 1):
            m = part.amax(1, keepdim=True)
            ends.append(m[:, 0] + torch.log2(torch.exp2(part - m).sum(1)))
        e = torch.stack(ends, 1)
        m = e.amax(1, keepdim=True)
        lse.append((m[:, 0] + torch.log2(torch.exp2(e - m).sum(1))) * torch.tensor(0.69314718055994530942, dtype=f))
    return torch.stack(lse).double()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 10, 500, 5000])
def test_the_bound_of_an_lse_holds_and_tells_a_row_less(kind, n):
    q, cache, lists = inputs(kind, n, seed=n)
    want, bound = R.lse_of_whole_numbers(q, R.cache_rows(cache, kind), lists, SCALE, kind)
    assert float(bound.max()) < 2.5e-5
    for parts in (1, 2) if n > 1 else (1,):
        assert bool(((lse_in_32_bits(q, cache, lists, kind, parts) - want).abs() <= bound).all())
    if n > 1:
        less = lse_in_32_bits(q, cache, [ls[:-1] for ls in lists], kind)
        assert float(((less - want).abs() > bound).double().mean()) > 0.8


@pytest.mark.parametrize("n", [1, 10, 100])
def test_the_bound_of_an_lse_tells_codes_times_scales_in_f16(n):
    q, cache, lists = inputs("e4m3", n, T=40, seed=n)
    want, bound = R.lse_of_whole_numbers(q, R.cache_rows(cache, "e4m3"), lists, SCALE, "e4m3")
    rows = R.cache_rows(cache, "e4m3")
    rows[:, :512] = rows[:, :512].to(torch.float16).double()
    off = R.lse_of_whole_numbers(q, rows, lists, SCALE, "e4m3")[0]
    assert float(((off - want).abs() > bound).double().mean()) > 0.5


def test_the_bound_of_the_normalisers_tells_one_running_sum_in_32_bits():
    r = np.random.default_rng(0)
    x = (r.standard_normal((16, 131072)) * 3).astype(np.float32)
    logits = torch.from_numpy(x)[:, None]
    scores = (torch.logsumexp(logits.double(), 2) - logits.double().amax(2)).float()
    e = np.exp((x - x.max(1, keepdims=True)).astype(np.float64))
    by_threads = e.astype(np.float32).reshape(16, -1, 256).cumsum(1, dtype=np.float32)[:, -1].astype(np.float64).sum(1)
    exact = scores.double() - torch.from_numpy(np.log(by_threads))[:, None]
    assert R.normaliser_error(exact, logits, scores) < R.NORMALISER
    running = e.astype(np.float32).cumsum(1, dtype=np.float32)[:, -1].astype(np.float64)
    assert R.normaliser_error(scores.double() - torch.from_numpy(np.log(running))[:, None], logits, scores) > R.NORMALISER
    assert R.normaliser_error(exact + 2.0 ** -19, logits, scores) > R.NORMALISER
