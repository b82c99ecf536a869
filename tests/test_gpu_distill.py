"""The distillation loss on a teacher's top entries and its gradient, against fp64."""

import math

import pytest
import torch

from tests import _layer_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_mla_attention_top_gb300 as S
    from sparse_mla_attention_top_gb300 import build

    build.build()
    return S


def case(seed, T, N, K, dtype=torch.float32, kind="weights", ragged=True):
    g = torch.Generator().manual_seed(seed)
    scores = (torch.randn((T, N), generator=g) * 3).to(dtype)
    lens = torch.randint(0, N + 1, (T,), generator=g, dtype=torch.int32) if ragged else None
    if ragged:
        lens[-1] = N
        lens[0] = min(N, 1)
    topk = torch.full((T, K), -1, dtype=torch.int32)
    for t in range(T):
        n = N if lens is None else int(lens[t])
        m = min(K, n)
        topk[t, :m] = torch.randperm(n, generator=g)[:m].to(torch.int32)
    value = torch.randn((T, K), generator=g) * 2
    return scores, lens, topk, torch.exp(value) if kind == "weights" else value


def check(S, scores, lens, topk, teacher, kind="weights", scope="candidates", temperature=1.0, row_weight=None,
          scores_dev=None, dscores=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    loss, grad = S.distill_topk(dev(scores) if scores_dev is None else scores_dev, dev(topk), dev(teacher), lens=dev(lens),
                                temperature=temperature, teacher_kind=kind, over=scope, row_weight=dev(row_weight),
                                dscores=dscores)
    (rl, rg), (bl, bg) = R.distill(scores, lens, topk, teacher, kind, scope, temperature, row_weight)
    R.within(loss, rl, bl, "loss")
    half = R.HALF[scores.dtype]
    # a value below the type's normal range is held to its smallest step (fp32 and bf16: 2^-126)
    R.within(grad, rg, bg + half * (rg.abs() + bg) + 2.0 ** -126, "gradient")
    return loss, grad


@pytest.mark.parametrize("scope", ["candidates", "listed"])
@pytest.mark.parametrize("kind", ["weights", "logits"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (3, 5, 8), (7, 333, 40), (5, 4096, 512), (2, 20000, 2048)])
def test_distill(S, scope, kind, dtype, T, N, K):
    s, lens, topk, w = case(T * N, T, N, K, dtype, kind)
    rw = torch.linspace(-0.5, 2.0, T)
    check(S, s, lens, topk, w, kind, scope, 0.7, rw)


@pytest.mark.parametrize("scope", ["candidates", "listed"])
@pytest.mark.parametrize("T,N", [(400, 16384), (400, 16390), (1, 131072), (2, 140001), (330, 33000)])
def test_distill_whole_rows_and_rows_beyond_shared_memory(S, scope, T, N):
    """One CTA a row up to 16384 scores, up to eight of them, and rows longer than eight parts."""
    g = torch.Generator().manual_seed(5)
    s = torch.randn((T, N), generator=g)
    topk = torch.randint(0, N, (T, 33), generator=g, dtype=torch.int32).sort(1).values
    w = torch.rand((T, 33), generator=g)
    lens = torch.full((T,), N, dtype=torch.int32)
    lens[T // 2] = N // 2
    loss, grad = S.distill_topk(s.cuda(), topk.cuda(), w.cuda(), lens=lens.cuda(), over=scope)
    pick = sorted({0, T // 2, T - 1})
    (rl, rg), (bl, bg) = R.distill(s[pick], lens[pick], topk[pick], w[pick], "weights", scope, 1.0)
    R.within(loss[pick], rl, bl, "loss")
    R.within(grad[pick], rg, bg + 2.0 ** -24 * rg.abs() + 2.0 ** -126, "gradient")


def test_distill_no_lens_no_row_weight_and_loss_or_gradient_alone(S):
    s, _, topk, w = case(1, 6, 777, 30, ragged=False)
    loss, grad = check(S, s, None, topk, w)
    only, none = S.distill_topk(s.cuda(), topk.cuda(), w.cuda(), need_grad=False)
    assert none is None and torch.equal(only, loss)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_distill_strided_rows_leave_what_lies_between(S, dtype):
    s, lens, topk, w = case(2, 6, 130, 20, dtype)
    for lead, stride in ((0, 136), (1, 139), (4, 160)):
        wide = torch.zeros(6, stride, dtype=dtype, device="cuda")
        wide[:, lead:lead + 130] = s.cuda()
        out = torch.full((6, stride), 9.0, dtype=dtype, device="cuda")
        check(S, s, lens, topk, w, scores_dev=wide[:, lead:lead + 130], dscores=out[:, lead:lead + 130])
        out[:, lead:lead + 130] = 9
        assert bool((out == 9).all())


@pytest.mark.parametrize("scope", ["candidates", "listed"])
def test_distill_rows_with_nothing(S, scope):
    T, N, K = 6, 50, 4
    s = torch.randn(T, N, generator=torch.Generator().manual_seed(3))
    topk = torch.tensor([[0, 1, 2, 3]] * T, dtype=torch.int32)
    w = torch.ones(T, K)
    lens = torch.tensor([0, 50, 50, 50, 50, -3], dtype=torch.int32)
    topk[1] = -1                     # no entry
    w[2] = 0                         # no weight
    topk[3] = torch.tensor([50, 60, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)  # all outside
    s[4] = -math.inf                 # no score
    loss, grad = check(S, s, lens, topk, w, scope=scope)
    assert not loss.any() and not grad.any()
    logits = torch.full((T, K), -math.inf)
    loss, grad = check(S, s, lens, topk, logits, kind="logits", scope=scope)
    assert not loss.any() and not grad.any()


@pytest.mark.parametrize("scope", ["candidates", "listed"])
def test_distill_masked_scores_and_weights(S, scope):
    T, N, K = 3, 100, 6
    s = torch.randn(T, N, generator=torch.Generator().manual_seed(4))
    topk = torch.arange(6, dtype=torch.int32).repeat(T, 1)
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(5)) + 0.1
    s[0, 10:] = -math.inf
    s[0, 2] = -math.inf
    w[0, 2] = 0.0                    # a masked score whose weight is 0 costs nothing
    s[1, 3:5] = torch.finfo(torch.float32).min
    w[1, 3:5] = 0.0
    s[2, 50] = 80.0
    check(S, s, None, topk, w, scope=scope, temperature=2.0)
    w[0, 2] = 1.0                    # with a weight, it costs everything, in its own row alone
    loss, grad = S.distill_topk(s.cuda(), topk.cuda(), w.cuda(), over=scope)
    assert math.isinf(loss[0]) and bool(torch.isfinite(loss[1:]).all()) and bool(torch.isfinite(grad).all())
    s[1, 1] = math.nan
    loss, grad = S.distill_topk(s.cuda(), topk.cuda(), w.cuda(), over=scope)
    assert math.isnan(loss[1]) and math.isfinite(loss[2]) and bool(torch.isfinite(grad[2]).all())


@pytest.mark.parametrize("scope", ["candidates", "listed"])
def test_distill_positions_listed_twice_count_twice(S, scope):
    s, _, _, _ = case(6, 2, 40, 6, ragged=False)
    topk = torch.tensor([[5, 5, 7, -1, 5, 9], [39, 0, 0, 39, 1, 1]], dtype=torch.int32)
    check(S, s, None, topk, torch.rand(2, 6, generator=torch.Generator().manual_seed(7)), scope=scope)


@pytest.mark.parametrize("scope", ["candidates", "listed"])
def test_distill_gradient_matches_differences(S, scope):
    """The fp64 loss along a direction, by a central difference of step h = 1e-4: its own error is h^2 / 6
    times a third derivative below 10 |d|^3, and 2^-50 / h."""
    s, lens, topk, w = case(8, 5, 200, 20)
    rw = torch.rand(5, generator=torch.Generator().manual_seed(9))
    d = torch.randn(5, 200, generator=torch.Generator().manual_seed(10)).double()
    _, grad = S.distill_topk(s.cuda(), topk.cuda(), w.cuda(), lens=lens.cuda(), row_weight=rw.cuda(), over=scope)
    h = 1e-4
    up, down = (R.distill(s.double() + z * h * d, lens, topk, w, "weights", scope, 1.0)[0][0] for z in (1, -1))
    num = ((up - down) / (2 * h) * rw.double()).sum()
    ana = (grad.double().cpu() * d).sum()
    assert abs(float(num - ana)) <= 2.0 ** -18 * float((grad.double().cpu() * d).abs().sum()) + 1e-6


def test_distill_in_a_graph(S):
    s, lens, topk, w = case(11, 8, 3000, 64)
    a, b, c, n = s.cuda(), topk.cuda(), w.cuda(), lens.cuda()
    S.distill_topk(a, b, c, lens=n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, grad = S.distill_topk(a, b, c, lens=n)
    s2, lens2, topk2, w2 = case(12, 8, 3000, 64)
    for x, y in ((a, s2), (b, topk2), (c, w2), (n, lens2)):
        x.copy_(y)
    g.replay()
    want = S.distill_topk(a, b, c, lens=n)
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])


def test_distill_empty_sizes(S):
    for T, N in ((0, 5), (3, 0)):
        loss, grad = S.distill_topk(torch.zeros((T, N), device="cuda"), torch.zeros((T, 2), dtype=torch.int32, device="cuda"),
                                    torch.ones((T, 2), device="cuda"))
        assert loss.shape == (T,) and grad.shape == (T, N) and not loss.any()


@pytest.mark.parametrize("scope", ["candidates", "listed"])
@pytest.mark.parametrize("kind", ["weights", "logits"])
def test_distill_lists_longer_than_the_registers_hold(S, scope, kind):
    s, lens, topk, w = case(13, 3, 6000, 5000, torch.float32, kind)
    check(S, s, lens, topk, w, kind, scope, 1.3)


def test_distill_a_small_loss_keeps_its_digits(S):
    """A student next to its teacher: the loss is a small difference of logarithms. Each entry's difference
    is rounded to fp32 (values up to 8, differences of a few hundredths), the sums' logarithms to 2^-23."""
    g = torch.Generator().manual_seed(14)
    s = torch.randn((64, 900), generator=g) * 2
    topk = torch.argsort(torch.rand((64, 900), generator=g), 1)[:, :8].sort(1).values.to(torch.int32)
    v = s.gather(1, topk.long()) + 0.05 * torch.randn((64, 8), generator=g)
    loss, _ = S.distill_topk(s.cuda(), topk.cuda(), v.cuda(), teacher_kind="logits", over="listed")
    (ref, _), _ = R.distill(s, None, topk, v, "logits", "listed", 1.0)
    assert float(ref.max()) < 0.02
    assert float((loss.double().cpu() - ref).abs().max()) <= 2.0 ** -21


def test_distill_on_two_streams_at_once(S):
    made = [case(15 + i, 40, 20000, 300) for i in range(2)]
    dev = [[None if t is None else t.cuda() for t in m] for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        got = []
        for st, (s, lens, topk, w) in zip(streams, dev):
            with torch.cuda.stream(st):
                got.append(S.distill_topk(s, topk, w, lens=lens))
    torch.cuda.synchronize()
    for (s, lens, topk, w), (loss, grad) in zip(made, got):
        (rl, rg), (bl, bg) = R.distill(s, lens, topk, w, "weights", "candidates", 1.0)
        R.within(loss, rl, bl)
        R.within(grad, rg, bg + 2.0 ** -24 * rg.abs() + 2.0 ** -126)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["weights", "logits"])
@pytest.mark.parametrize("N", [50, 20000, 200000])
def test_distill_a_choice_of_one_costs_exactly_nothing(S, dtype, kind, N):
    """One live entry among the listed, or one candidate: p = q = 1."""
    g = torch.Generator().manual_seed(16)
    s = (torch.randn((4, N), generator=g) * 5).to(dtype).cuda()
    topk = torch.randint(0, N, (4, 3), generator=g, dtype=torch.int32).cuda()
    topk[:, 1:] = -1
    w = torch.rand((4, 3), generator=g).cuda() * 7 + 0.1
    loss, grad = S.distill_topk(s, topk, w, teacher_kind=kind, over="listed", temperature=1.7)
    assert not loss.any() and not grad.any()
    topk[:] = 0
    topk[:, 1:] = torch.tensor([1, 77], dtype=torch.int32)  # dead: there is one candidate
    lens = torch.ones(4, dtype=torch.int32, device="cuda")
    loss, grad = S.distill_topk(s, topk, w, lens=lens, teacher_kind=kind, temperature=0.3)
    assert not loss.any() and not grad.any()


@pytest.mark.parametrize("scope", ["candidates", "listed"])
def test_distill_weights_of_any_size(S, scope):
    s, lens, topk, w = case(17, 6, 3000, 40)
    check(S, s, lens, topk, w * 1e36, scope=scope)
    check(S, s, lens, topk, w * 1e-36, scope=scope)
    s[:, ::3] = -math.inf
    w[topk % 3 == 0] = 0.0
    check(S, s, lens, topk, w, scope=scope)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_distill_nan_among_masked_scores_of_a_long_row_stays_nan(S, dtype):
    """Rows so long that a CTA reads its share in pieces; in the first piece nothing but -inf and one NaN."""
    N, K = 140_000, 16
    scores, lens, topk, teacher = case(70, 3, N, K, dtype, ragged=False)
    scores[0, :16384] = -math.inf
    scores[0, 100] = math.nan
    scores[2, :16384] = -math.inf  # the same row without the NaN
    topk[:] += 20_000 * (topk < 20_000).to(torch.int32)
    loss, grad = S.distill_topk(scores.cuda(), topk.cuda(), teacher.cuda())
    assert bool(loss[0].isnan()) and bool(grad[0].isnan().all())
    (rl, rg), (bl, bg) = R.distill(scores[1:], None, topk[1:], teacher[1:], "weights", "candidates", 1.0)
    R.within(loss[1:], rl, bl, "loss")
    R.within(grad[1:], rg, bg + R.HALF[dtype] * (rg.abs() + bg) + 2.0 ** -126, "gradient")


@pytest.mark.parametrize("scope,nan_listed", [("candidates", False), ("candidates", True), ("listed", True)])
@pytest.mark.parametrize("N,K", [(100, 8), (9000, 8), (9000, 2100), (140_000, 8)])
def test_distill_nan_beside_a_weighted_score_of_minus_infinity(S, scope, nan_listed, N, K):
    """A NaN makes the row NaN also where a listed score of -inf alone would make its loss infinite."""
    scores, lens, topk, teacher = case(71, 3, N, K, ragged=False)
    free = [n for n in range(K + 1) if n not in topk[0].tolist()][0]
    scores[0, topk[0, 0] if nan_listed else free], scores[0, topk[0, 1]] = math.nan, -math.inf
    scores[1, topk[1, 1]] = -math.inf
    loss, grad = S.distill_topk(scores.cuda(), topk.cuda(), teacher.cuda(), over=scope)
    assert bool(loss[0].isnan()) and float(loss[1]) == math.inf and bool(loss[2].isfinite())
    assert bool(grad[0, topk[0].long().cuda()].isnan().all()) and bool(grad[1:].isfinite().all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scope", ["candidates", "listed"])
@pytest.mark.parametrize("kind", ["weights", "logits"])
@pytest.mark.parametrize("N,K", [(64, 6), (9000, 6), (9000, 2100)])
def test_distill_listed_scores_of_the_lowest_value(S, dtype, scope, kind, N, K):
    """Masks of the type's lowest value instead of -inf: a weighted one costs its share of 3.4e38, a finite
    loss. Its fp32 terms: the difference of scores, c = log2 e / tau (two roundings), the product, the weight
    (2 ulp and a division), the logarithm below it, W, the quotient and ln 2, each within 2^-23, and sums of
    at most 2100 / 512 + 64 steps of 2^-24: below 2^-17."""
    low = torch.finfo(dtype).min
    scores, lens, topk, teacher = case(72, 4, N, K, dtype, kind, ragged=False)
    masked = K // 2
    for t in (0, 1):
        scores[t, topk[t, :masked].long()] = low
    scores[2] = low  # every score the same: a uniform softmax
    if kind == "weights":
        teacher = teacher * 0.25 + 0.5
    for tau in (1.0, 8.0):
        loss, grad = S.distill_topk(scores.cuda(), topk.cuda(), teacher.cuda(), teacher_kind=kind, over=scope, temperature=tau)
        # (relative to the row's largest: fp64 would lose ln N beside 3.4e38)
        shifted = scores.double() - scores.double().amax(1, keepdim=True)
        (rl, rg), _ = R.distill(shifted, None, topk, teacher, kind, scope, tau)
        assert 1e36 < float(rl[0]) < 3.3e38 and float(rl[2]) < 20
        off = (loss.double().cpu() - rl).abs()
        assert bool((off[:2] <= 2.0 ** -17 * rl[:2]).all()), (loss, rl)
        assert bool((off[2:] <= 1e-4).all()), (loss, rl)
        assert float((grad.double().cpu() - rg).abs().max()) <= (2.0 ** -17 + R.HALF[dtype]) / tau
