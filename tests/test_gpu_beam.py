"""svt_beam_select against fp64 sums and a sort."""

import numpy as np
import pytest
import torch

import sparse_mla_attention_top_gb300 as S
from tests import _serving_ref as R

pytestmark = pytest.mark.gpu
INF = float("inf")


# What a normaliser may be off by. Its sum has positive terms: each exponential is off by at most 2^-22 (ex2.approx) and,
# by the roundings of its argument y = (x - max) log2 e, 2^-23 |y| 2^-|y| <= 2^-23.9 of the sum. A thread takes at most 32
# rounds (131072 tokens of fp32 by one CTA); a term goes through at most 8 additions in its round, 2 that join the round's parts
# and 32 rounds (2^-24 each; sums of threads are integers), and a rescaling by an exponential in each and at the end (2^-22 +
# 2^-23.9 + 2^-24; slices, which are joined by another, have half the rounds). The logarithm's mantissa is rounded, and it
# itself (2.5 * 2^-24). 2^-22 + 2^-23.9 + 42 * 2^-24 + 33 * 6.1 * 2^-24 + 2.5 * 2^-24 < 2^-16.
DELTA = 2.0 ** -16


def check(logits, scores, K, finished=None, end_token=0):
    """Values within the normalisers' error, and the order of the exact values: within a beam always, between beams that do not
    have the same logits and scores where the values are further apart than two such errors."""
    value, parent, token = S.beam_select(logits, scores, K, finished=finished, end_token=end_token)
    everything = R.beam(logits, scores, logits.shape[1] * logits.shape[2], finished, end_token)
    for b, (v, p, t) in enumerate(everything):
        n = min(K, len(v))
        got = value[b].double().cpu().numpy(), parent[b].cpu().numpy(), token[b].cpu().numpy()
        assert (got[1][n:] == -1).all() and (got[2][n:] == -1).all() and np.isneginf(got[0][n:]).all()
        picked = list(zip(got[1][:n].tolist(), got[2][:n].tolist()))
        assert len(set(picked)) == n
        exact = {(int(pp), int(tt)): float(vv) for vv, pp, tt in zip(v, p, t)}
        mine = np.array([exact[x] for x in picked])
        assert (np.abs(got[0][:n] - mine) <= np.abs(mine) * 2.0 ** -24 + DELTA).all(), b
        differ = np.array([x != (int(pp), int(tt)) for x, pp, tt in zip(picked, p, t)], bool)
        assert (np.abs(mine - v[:n])[differ] <= 2 * DELTA).all(), b
        of = [[tt for pp, tt in picked if pp == w] for w in range(logits.shape[1])]
        for w, ours in enumerate(of):  # a beam's own candidates: its first ones, in order
            assert ours == t[p == w][:len(ours)].tolist(), (b, w)
            for u in range(w):  # equal beams: a candidate of the first comes before the other's
                if finished is None and scores[b, u] == scores[b, w] and torch.equal(logits[b, u], logits[b, w]):
                    assert of[u][:len(ours)] == ours and all(picked.index((u, x)) < picked.index((w, x)) for x in ours)
    return value, parent, token


def draw(B, W, V, dtype, seed=0, scale=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return ((torch.randn((B, W, V), generator=g, device="cuda") * scale).to(dtype),
            -torch.rand((B, W), generator=g, device="cuda") * 20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 100, 1000, 8191, 8192, 50257, 131072])
def test_vocabularies(dtype, V):
    logits, scores = draw(3, 4, V, dtype, V)
    check(logits, scores, 8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W, K", [(1, 1), (1, 128), (2, 128), (5, 3), (16, 32), (64, 128), (128, 64)])
def test_widths(dtype, W, K):
    logits, scores = draw(2, W, 3001, dtype, W)
    check(logits, scores, K)


def test_a_small_vocabulary_has_few_candidates():
    logits, scores = draw(2, 3, 4, torch.float32)
    value, parent, _ = check(logits, scores, 20)
    assert (parent[:, 12:] == -1).all() and torch.isneginf(value[:, 12:]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [300, 9000, 70001])
def test_ties_go_to_the_first(dtype, V):
    logits = torch.zeros((2, 3, V), dtype=dtype, device="cuda")
    scores = torch.tensor([[0.0, 0.0, 0.0], [-2.0, -1.0, -1.0]], device="cuda")
    _, parent, token = check(logits, scores, 5)
    assert token.tolist() == [[0, 1, 2, 3, 4]] * 2 and parent.tolist() == [[0] * 5, [1] * 5]
    logits[:, :, V // 2] = 1
    logits[:, :, V - 1] = 1
    _, _, token = check(logits, scores, 7)
    assert token[0].tolist() == [V // 2, V - 1] * 3 + [0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_in_order(dtype):
    # each round of a CTA's loads beats all before it; and steps of equal values
    up = torch.linspace(-30, 30, 60000, device="cuda")
    logits = torch.stack([up, up.flip(0), (up * 0.2).round()]).to(dtype)[None].contiguous()
    check(logits, torch.zeros((1, 3), device="cuda"), 40)


def test_signed_zeroes_are_equal():
    logits = torch.zeros((1, 1, 64), device="cuda")
    logits[0, 0, ::2] = -0.0
    assert check(logits, torch.zeros((1, 1), device="cuda"), 4)[2].tolist() == [[0, 1, 2, 3]]


def test_the_first_step_of_a_search():
    # one live beam, the others at -inf
    logits, scores = draw(4, 5, 5003, torch.bfloat16, 1)
    scores[:, 1:] = -INF
    scores[:, 0] = 0
    _, parent, _ = check(logits, scores, 5)
    assert (parent == 0).all()


@pytest.mark.parametrize("low", [-1e9, -1e30, torch.finfo(torch.float32).min])
def test_the_first_step_with_low_scores_for_the_others(low):
    logits, scores = draw(3, 6, 4001, torch.float32, 11)
    scores[:, 1:] = low
    scores[:, 0] = 0
    _, parent, _ = check(logits, scores, 12)
    assert (parent == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W, V", [(64, 500), (3, 40000)])
def test_many_equal_candidates(dtype, W, V):
    # more of them than a warp or a CTA keeps: each slice's first K, then the beams' in order
    logits = torch.full((2, W, V), 3.25, dtype=dtype, device="cuda")
    logits[1, :, : V // 2] = torch.finfo(dtype).min
    scores = torch.zeros((2, W), device="cuda")
    _, parent, token = S.beam_select(logits, scores, 128)
    assert (parent == 0).all()
    assert token.tolist() == [list(range(128)), list(range(V // 2, V // 2 + 128))]


def test_one_beam_above_all_others():
    logits, scores = draw(3, 16, 9000, torch.float32, 12)
    scores[:, 5] = 1000
    _, parent, _ = check(logits, scores, 128)
    assert (parent == 5).all()


def test_beams_that_share_their_logits():
    # (a stride of 0)
    logits, scores = draw(2, 1, 2000, torch.bfloat16, 13)
    check(logits.expand(2, 4, 2000), scores[:, :1].expand(2, 4).contiguous(), 9)


@pytest.mark.parametrize("off", range(8))
def test_equal_rows_have_equal_sums_wherever_they_lie(off):
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    row = (torch.randn(5003, generator=g, device="cuda") * 2).to(torch.bfloat16)
    flat = torch.zeros(3 * 5100 + 8, dtype=torch.bfloat16, device="cuda")
    x = flat[off:off + 3 * 5097].view(1, 3, 5097)[:, :, :5003]  # (an odd stride: another alignment for each)
    x[:] = row
    value, parent, token = check(x, torch.zeros((1, 3), device="cuda"), 12)
    # (equal values within the row, too: those of a beam together)
    assert torch.bincount(parent[0]).tolist() == [4, 4, 4]
    for w in (1, 2):
        assert torch.equal(token[parent == 0], token[parent == w]) and torch.equal(value[parent == 0], value[parent == w])


def test_two_graphs_at_once():
    cases = [draw(3, 4, 30000, torch.bfloat16, 15), draw(3, 4, 30000, torch.bfloat16, 16)]
    wants = [S.beam_select(*c, 8) for c in cases]
    graphs, outs = [], []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(S.beam_select(*c, 8))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_finished_beams_keep_their_score():
    logits, scores = draw(6, 4, 20000, torch.float32, 2)
    finished = torch.rand((6, 4), device="cuda") < 0.5
    finished[0] = True
    finished[1] = False
    logits[finished] = float("nan")  # (not read)
    for kind in (torch.bool, torch.uint8):
        value, parent, token = check(logits, scores, 9, finished.to(kind), 77)
    assert (parent[0, 4:] == -1).all() and (token[0, :4] == 77).all()
    assert torch.equal(value[0, :4], scores[0].sort(descending=True).values)


def test_masked_logits():
    for dtype in (torch.bfloat16, torch.float32):
        logits, scores = draw(3, 3, 9001, dtype, 3)
        logits[:, :, 5:] = -INF          # five candidates a beam
        logits[1, 0] = -INF              # none
        low = torch.finfo(dtype).min
        logits[2, 1, 5:] = low           # masks of the type's lowest value are numbers
        logits[2, 2] = low
        check(logits, scores, 16)


def test_nan_and_infinite_logits_leave_their_beam_without_candidates():
    logits, scores = draw(4, 3, 40001, torch.float32, 4)
    logits[0, 1, 39999] = float("nan")
    logits[1, 0, 3] = INF
    logits[2] = float("nan")
    scores[3, 0] = float("nan")
    _, parent, _ = check(logits, scores, 6)
    assert not (parent[0] == 1).any() and not (parent[1] == 0).any() and (parent[2] == -1).all()
    assert not (parent[3] == 0).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(dtype):
    big = draw(5, 6, 1013, dtype, 5)[0]
    scores = draw(2, 3, 1, dtype)[1]
    for x in (big[1:3, 2:5, 3:1003], big[::3][:2, ::2, :1000], big.transpose(0, 1)[:2, :3, 1:]):
        check(x, scores, 6)


def test_large_logits():
    logits, scores = draw(2, 2, 3000, torch.float32, 6, scale=1e4)
    value, parent, token = S.beam_select(logits, scores, 4)
    for b, (v, p, t) in enumerate(R.beam(logits, scores, 4)):
        assert parent[b].tolist() == p.tolist() and token[b].tolist() == t.tolist()


def test_graph_and_empty_batch():
    logits, scores = draw(3, 4, 30000, torch.bfloat16, 7)
    ws = S.Workspace()
    want = S.beam_select(logits, scores, 8, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = S.beam_select(logits, scores, 8, ws=ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert [x.shape for x in S.beam_select(logits[:0], scores[:0], 8)] == [(0, 8)] * 3


def test_refused_tensors():
    logits, scores = draw(2, 3, 50, torch.float32)
    with pytest.raises(TypeError):
        S.beam_select(logits.half(), scores, 2)
    with pytest.raises(TypeError):
        S.beam_select(logits, scores.double(), 2)
    with pytest.raises(TypeError):
        S.beam_select(logits, scores[:1], 2)
    with pytest.raises(TypeError):
        S.beam_select(logits, scores, 2, finished=scores)
    with pytest.raises(S.SvtError):
        S.beam_select(logits, scores, 0)
    with pytest.raises(S.SvtError):
        S.beam_select(logits, scores, 129)
    with pytest.raises(S.SvtError):
        S.beam_select(logits, scores, 2, finished=scores > 0, end_token=50)


@pytest.mark.parametrize("dtype, V", [(torch.float32, 50001), (torch.bfloat16, 100001)])
@pytest.mark.parametrize("K", [1, 100])
def test_rounds_that_overflow_one_after_another(dtype, V, K):
    # so many beams that each is one CTA's, over several rankings: all values of a round above those before, steps of equal
    # ones, and both in turn; time and again, as warps run ahead of one another as they like
    up = torch.arange(V, device="cuda", dtype=torch.float32)
    rows = torch.stack([up * 2.0 ** -12, (up / 3000).floor(), torch.where(up % 20000 < 10000, up * 2.0 ** -12, 1.0)]).to(dtype)
    B = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    logits = rows.repeat(B // 3, 1)[:, None]
    scores = torch.zeros((B, 1), device="cuda")
    want = torch.sort(rows.double(), dim=1, descending=True, stable=True).indices[:, :K].to(torch.int32).repeat(B // 3, 1)
    first = S.beam_select(logits, scores, K)
    assert torch.equal(first[2], want)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(S.beam_select(logits, scores, K), first))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B, V", [(64, 50257), (600, 32003), (512, 131072)])
def test_normalisers(dtype, B, V):
    # rows cut in slices and rows of one CTA; scores that leave the values near 0, where their own rounding is none
    logits, _ = draw(B, 1, V, dtype, 17)
    x = logits.double()
    scores = (x.logsumexp(2) - x.amax(2)).float()
    value, _, _ = S.beam_select(logits, scores, 1)
    assert R.normaliser_error(value, logits, scores) < R.NORMALISER
