"""The attention's backward pass against fp64, with bounds from the stated roundings."""

import math

import pytest
import torch

from sparse_mla_attention_top_gb300 import workloads as W
from tests import _layer_ref as R

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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(seed, *shape):
    return torch.randn(shape, generator=gen(seed)).to(torch.bfloat16)


def lists(seed, T, K, num, dead=0.2):
    """Distinct slots per query in random order, some entries -1 anywhere."""
    g = gen(seed)
    out = torch.full((T, K), -1, dtype=torch.int32)
    for t in range(T):
        m = min(K, num)
        out[t, :m] = torch.randperm(num, generator=g)[:m].to(torch.int32)
    out[torch.rand((T, K), generator=g) < dead] = -1
    return out


def forward(S, q, kv, topk, scale=SCALE, **kw):
    out, lse = S.sparse_mla_decode(q, kv, topk, scale, num_splits=1, **kw)
    return out, lse


def check(S, q, cache, slots, dout, dlse=None, scale=SCALE, stride=0, fwd=None, **kw):
    """q, cache [n, 576] and dout on the CPU; slots [T, K] the resolved lists; kw: how the call names them."""
    n = cache.shape[0]
    if stride:
        wide = torch.full((n, stride // 2), float("nan"), dtype=torch.bfloat16)
        wide[:, :576] = cache
        data = wide.cuda()
    else:
        data = cache.cuda()
    page = kw.pop("page_size", 1)
    kv = S.KVCache(data, n // page, page, W.KV_BF16, row_stride_bytes=stride)
    topk = kw.pop("topk", slots).cuda()
    kw = {k: v.cuda() for k, v in kw.items()}
    qd, dd = q.cuda(), dout.cuda()
    out, lse = forward(S, qd, kv, topk, scale, **kw) if fwd is None else fwd
    ws = S.Workspace()
    dq, dkv, w = S.sparse_mla_backward(qd, kv, topk, scale, out, lse, dd, dlse=None if dlse is None else dlse.cuda(),
                                       return_weights=True, ws=ws, **kw)
    assert ws.read_status() == 0
    ref, bound = R.backward(q, cache, slots.long(), scale, out.cpu(), lse.cpu(), dout, dlse)
    for name, a, b, c in zip(("dq", "dkv", "weights"), (dq, dkv, w), ref, bound):
        R.within(a, b, c, name)
    return dq, dkv, w


@pytest.mark.parametrize("T,H,K,num", [
    (1, 1, 1, 1), (1, 8, 64, 256), (3, 5, 70, 90), (2, 64, 64, 64), (2, 65, 63, 100), (1, 128, 129, 300),
    (5, 16, 200, 333), (2, 64, 128, 129), (7, 33, 65, 70), (1, 64, 2048, 3000), (2, 128, 1000, 1024)])
def test_backward(S, T, H, K, num):
    check(S, normal(1, T, H, 576), normal(2, num, 576), lists(3, T, K, num), normal(4, T, H, 512),
          dlse=torch.randn((T, H), generator=gen(5)))


@pytest.mark.parametrize("T,H,K", [(200, 128, 130), (170, 16, 600), (321, 64, 70), (153, 1, 64), (150, 64, 129)])
def test_backward_more_queries_than_sms(S, T, H, K):
    check(S, normal(1, T, H, 576), normal(2, 700, 576), lists(3, T, K, 700), normal(4, T, H, 512))


@pytest.mark.parametrize("H", [15, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 63), (3, 65), (190, 129), (37, 1100)])
def test_backward_around_32_heads(S, T, H, K):
    """Row-sets of 32 and of 64 heads: lists of one tile and of many, cut between CTAs and whole, dead tiles."""
    slots = lists(102, T, K, 1200)
    if T > 2:
        slots[1] = -1
        slots[2, : K // 2] = -1
    dq, dkv, w = check(S, normal(103, T, H, 576), normal(104, 1200, 576), slots, normal(105, T, H, 512))
    if T > 2:
        assert not dq[1].any() and not w[1].any()


@pytest.mark.parametrize("T,H,K,live", [(1, 4, 9000, 9000), (2, 16, 5000, 2049), (3, 1, 4097, 1), (2, 70, 4096, 0)])
def test_backward_lists_of_several_pieces(S, T, H, K, live):
    """Long lists, their live entries ending in any piece of them (or missing, or only at the very end)."""
    slots = lists(98, T, K, 9500, dead=0.0)
    slots[:, live:] = -1
    if live == 1:
        slots[0, 0], slots[0, K - 1] = -1, 77
    check(S, normal(99, T, H, 576), normal(100, 9500, 576), slots, normal(101, T, H, 512))


def test_backward_paged_requests_counts_and_padded_rows(S):
    T, H, K, P = 6, 12, 40, 16
    n = 10 * P
    g = gen(7)
    bt = torch.tensor([[3, 9, 0, -1], [5, 1, 2, 8]], dtype=torch.int32)
    seq = torch.tensor([41, 64], dtype=torch.int32)
    req = torch.tensor([1, 0, 0, 1, 1, 0], dtype=torch.int32)
    count = torch.tensor([40, 30, 0, 1, 40, 17], dtype=torch.int32)
    topk = torch.full((T, K), -1, dtype=torch.int32)
    slots = torch.full((T, K), -1, dtype=torch.int32)
    for t in range(T):
        perm = torch.randperm(int(seq[req[t]]), generator=g)[:K].to(torch.int32)
        topk[t, :len(perm)] = perm
        for j in range(int(count[t])):
            if topk[t, j] >= 0:
                slots[t, j] = bt[req[t], topk[t, j] // P] * P + topk[t, j] % P
    for stride in (0, 1216):
        check(S, normal(8, T, H, 576), normal(9, n, 576), slots, normal(10, T, H, 512), stride=stride, topk=topk,
              block_table=bt, seq_lens=seq, req_of_token=req, topk_len=count, page_size=P)


def test_backward_rows_with_nothing_and_rows_nobody_lists(S):
    T, H, n = 4, 16, 200
    slots = lists(11, T, 100, 150, dead=0.1)
    slots[1] = -1
    slots[3, 5:] = -1
    cache = normal(12, n, 576)
    cache[150:] = float("nan")   # behind every list: must not be read into anything
    q, dout = normal(13, T, H, 576), normal(14, T, H, 512)
    kv = S.KVCache(cache.cuda(), n, 1, W.KV_BF16)
    out, lse = forward(S, q.cuda(), kv, slots.cuda())
    dq, dkv, w = S.sparse_mla_backward(q.cuda(), kv, slots.cuda(), SCALE, out, lse, dout.cuda(), return_weights=True,
                                       ws=S.Workspace())
    assert not dq[1].any() and not w[1].any() and not dkv[150:].any()
    assert not w[3, 5:].any() and not w[slots.cuda() < 0].any()
    clean = cache.clone()
    clean[150:] = 0
    ref, bound = R.backward(q, clean, slots.long(), SCALE, out.cpu(), lse.cpu(), dout)
    for a, b, c in zip((dq, dkv, w), ref, bound):
        R.within(a, b, c)


def test_backward_bad_values_stay_with_their_query(S):
    """A query with NaN and infinities spoils its own gradient and the rows it lists, nothing else."""
    T, H = 3, 16
    slots = torch.stack([torch.arange(0, 70), torch.arange(70, 140), torch.arange(140, 210)]).to(torch.int32)
    q, dout, cache = normal(15, T, H, 576), normal(16, T, H, 512), normal(17, 210, 576)
    kv = S.KVCache(cache.cuda(), 210, 1, W.KV_BF16)
    out, lse = forward(S, q.cuda(), kv, slots.cuda())
    q[1, 3, 7], q[1, 4, 8], dout[1, 5, 9] = math.nan, math.inf, math.nan
    dq, dkv, w = S.sparse_mla_backward(q.cuda(), kv, slots.cuda(), SCALE, out, lse, dout.cuda(), return_weights=True,
                                       ws=S.Workspace())
    ref, bound = R.backward(q[::2], cache, slots[::2].long(), SCALE, out[::2].cpu(), lse[::2].cpu(), dout[::2])
    R.within(dq[::2], ref[0], bound[0])
    keep = torch.cat([torch.arange(70), torch.arange(140, 210)])
    R.within(dkv.cpu()[keep], ref[1][keep], bound[1][keep])
    assert dkv[70:140].isnan().any()


def test_backward_entries_listed_twice_count_twice(S):
    slots = torch.tensor([[3, 3, 5, 3, 0, 5, -1, 9]] * 2, dtype=torch.int32)
    check(S, normal(18, 2, 16, 576), normal(19, 10, 576), slots, normal(20, 2, 16, 512))


def test_backward_out_of_range_entries_are_dead_and_reported(S):
    q, dout, cache = normal(21, 2, 8, 576), normal(22, 2, 8, 512), normal(23, 64, 576)
    good = torch.tensor([[1, 2, -1, 3], [4, -1, 5, 6]], dtype=torch.int32)
    bad = good.clone()
    bad[0, 2], bad[1, 1] = 64, 2 ** 31 - 1
    kv = S.KVCache(cache.cuda(), 64, 1, W.KV_BF16)
    out, lse = forward(S, q.cuda(), kv, good.cuda())
    ws = S.Workspace()
    got = S.sparse_mla_backward(q.cuda(), kv, bad.cuda(), SCALE, out, lse, dout.cuda(), return_weights=True, ws=ws)
    assert ws.read_status() == S.svt.DEV_ERR_INDEX_RANGE and ws.read_status() == 0
    want = S.sparse_mla_backward(q.cuda(), kv, good.cuda(), SCALE, out, lse, dout.cuda(), return_weights=True, ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]) and torch.equal(got[1], want[1])


def test_backward_large_scores(S):
    """Logits of +-60: the probabilities underflow cleanly and the largest stay exact."""
    q, cache = normal(24, 2, 16, 576) * 4, normal(25, 300, 576) * 4
    check(S, q, cache, lists(26, 2, 256, 300), normal(27, 2, 16, 512))


def test_backward_empty_calls(S):
    cache = normal(28, 32, 576).cuda()
    kv = S.KVCache(cache, 32, 1, W.KV_BF16)
    e = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    dkv = torch.full((32, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    S.sparse_mla_backward(e(0, 4, 576), kv, e(0, 8, d=torch.int32), SCALE, e(0, 4, 512), e(0, 4, d=torch.float32),
                          e(0, 4, 512), dkv=dkv, ws=S.Workspace())
    assert not dkv.any()
    dq = torch.full((2, 4, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    S.sparse_mla_backward(e(2, 4, 576), kv, e(2, 0, d=torch.int32), SCALE, e(2, 4, 512),
                          torch.full((2, 4), -math.inf, device="cuda"), e(2, 4, 512), dq=dq, dkv=dkv, ws=S.Workspace())
    assert not dq.any() and not dkv.any()


def test_backward_matches_differences_of_the_forward(S):
    """L = sum(out . dout) + sum(lse . dlse) in fp64, along one direction in q and the cache by a central
    difference; the gradient's own bound along that direction is the tolerance, with 1e-6 of L's size
    for the difference (h = 1e-4, third derivatives of order one; out enters delta rounded to bf16,
    which moves delta by at most 2^-8 sum |out dout|)."""
    T, H, K, n = 3, 8, 90, 120
    q, cache, dout = normal(30, T, H, 576), normal(31, n, 576), normal(32, T, H, 512)
    dlse = torch.randn((T, H), generator=gen(33))
    slots = lists(34, T, K, n)
    dq, dkv, _ = check(S, q, cache, slots, dout, dlse)
    ref_out = torch.zeros(T, H, 512, dtype=torch.float64)

    def loss(qq, cc):
        total = 0.0
        for t in range(T):
            o, l = R.attention(qq[t], cc[slots[t][slots[t] >= 0].long()], SCALE)
            ref_out[t] = o
            total += (o * dout[t].double()).sum() + (l * dlse[t].double()).sum()
        return float(total)
    vq, vk = torch.randn(q.shape, generator=gen(35)).double(), torch.randn(cache.shape, generator=gen(36)).double()
    h = 1e-4
    num = (loss(q.double() + h * vq, cache.double() + h * vk) - loss(q.double() - h * vq, cache.double() - h * vk)) / (2 * h)
    loss(q.double(), cache.double())
    ana = float((dq.double().cpu() * vq).sum() + (dkv.double().cpu() * vk).sum())
    lse = torch.stack([R.attention(q[t].double(), cache[slots[t][slots[t] >= 0].long()].double(), SCALE)[1] for t in range(T)])
    (rq, rk, _), (bq, bk, _) = R.backward(q, cache, slots.long(), SCALE, ref_out, lse, dout, dlse)
    slack = float((bq * vq.abs()).sum() + (bk * vk.abs()).sum())
    moved = float((ref_out.abs() * dout.double().abs()).sum()) * 2.0 ** -8 * SCALE
    reach = max(float((cache.double() @ vq.reshape(-1, 576).T).abs().max()), float((q.reshape(-1, 576).double() @ vk.T).abs().max()))
    assert abs(num - ana) <= slack + moved * reach + 1e-6 * (abs(num) + 1)


def test_backward_is_repeatable_but_for_the_cache_sums(S):
    q, cache, dout = normal(40, 50, 16, 576).cuda(), normal(41, 500, 576).cuda(), normal(42, 50, 16, 512).cuda()
    slots = lists(43, 50, 300, 500).cuda()
    kv = S.KVCache(cache, 500, 1, W.KV_BF16)
    out, lse = forward(S, q, kv, slots)
    ws = S.Workspace()
    a = S.sparse_mla_backward(q, kv, slots, SCALE, out, lse, dout, return_weights=True, ws=ws)
    b = S.sparse_mla_backward(q, kv, slots, SCALE, out, lse, dout, return_weights=True, ws=ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_backward_in_graphs_and_on_two_streams(S):
    """Two captured graphs with a workspace each, replayed on two streams at once, on inputs that changed
    after the capture, against eager calls."""
    T, H, K, n = 20, 64, 200, 400
    kv = [S.KVCache(normal(50 + i, n, 576).cuda(), n, 1, W.KV_BF16) for i in range(2)]
    q = [normal(52 + i, T, H, 576).cuda() for i in range(2)]
    slots = [lists(54 + i, T, K, n).cuda() for i in range(2)]
    dout = [normal(56 + i, T, H, 512).cuda() for i in range(2)]
    fw = [forward(S, q[i], kv[i], slots[i]) for i in range(2)]
    ws = [S.Workspace(nbytes=S.svt.lib().svt_sparse_mla_backward_workspace_size(T, H, K, n)) for _ in range(2)]
    run = lambda i: S.sparse_mla_backward(q[i], kv[i], slots[i], SCALE, *fw[i], dout[i], return_weights=True, ws=ws[i])  # noqa: E731
    graphs, got = [], []
    for i in range(2):
        run(i)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(run(i))
        graphs.append(g)
    for i in range(2):
        dout[i].copy_(normal(58 + i, T, H, 512))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert ws[i].read_status() == 0
        ref, bound = R.backward(q[i].cpu(), kv[i].data.cpu(), slots[i].cpu().long(), SCALE, fw[i][0].cpu(), fw[i][1].cpu(),
                                dout[i].cpu())
        for a, b, c in zip(got[i], ref, bound):
            R.within(a, b, c)


def test_backward_after_other_calls_in_the_same_workspace(S):
    """The workspace is shared with the forward's split decode and comes back larger or dirty."""
    T, H, K, n = 4, 64, 500, 600
    kv = S.KVCache(normal(60, n, 576).cuda(), n, 1, W.KV_BF16)
    q, dout, slots = normal(61, T, H, 576).cuda(), normal(62, T, H, 512).cuda(), lists(63, T, K, n).cuda()
    ws = S.Workspace()
    outs = []
    for _ in range(2):
        out, lse = S.sparse_mla_decode(q, kv, slots, SCALE, num_splits=3, ws=ws)
        dq, dkv, w = S.sparse_mla_backward(q, kv, slots, SCALE, out, lse, dout, return_weights=True, ws=ws)
        outs.append((out, lse, dq, w))
    assert ws.read_status() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    ref, bound = R.backward(q.cpu(), kv.data.cpu(), slots.cpu().long(), SCALE, out.cpu(), lse.cpu(), dout.cpu())
    for a, b, c in zip((dq, dkv, w), ref, bound):
        R.within(a, b, c)


def test_backward_refuses_an_e4m3_cache(S):
    kv = S.KVCache(torch.zeros(8, 656, dtype=torch.uint8, device="cuda"), 8, 1, W.KV_FP8_E4M3)
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    with pytest.raises(S.SvtError) as e:
        S.sparse_mla_backward(z(1, 4, 576), kv, z(1, 2, d=torch.int32), SCALE, z(1, 4, 512), z(1, 4, d=torch.float32),
                              z(1, 4, 512), ws=S.Workspace())
    assert e.value.status == S.svt.SVT_ERR_UNSUPPORTED


def test_backward_graphs_that_share_a_workspace_replay_in_turn(S):
    """Two graphs of different sizes captured on one workspace, replayed one after another, the workspace
    outgrown in between by an eager call."""
    T, H, K, n = 6, 32, 150, 260
    ws = S.Workspace()
    made = []
    for i, (t, k) in enumerate(((T, K), (2 * T, K // 2))):
        kv = S.KVCache(normal(70 + i, n, 576).cuda(), n, 1, W.KV_BF16)
        q, dout, slots = normal(72 + i, t, H, 576).cuda(), normal(74 + i, t, H, 512).cuda(), lists(76 + i, t, k, n).cuda()
        out, lse = forward(S, q, kv, slots)
        run = lambda kv=kv, q=q, dout=dout, slots=slots, out=out, lse=lse: S.sparse_mla_backward(  # noqa: E731
            q, kv, slots, SCALE, out, lse, dout, return_weights=True, ws=ws)
        want = run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        made.append((g, got, want, (q, kv, slots, out, lse, dout)))
    big = S.KVCache(normal(80, 5000, 576).cuda(), 5000, 1, W.KV_BF16)
    q, kv, slots, out, lse, dout = made[0][3]
    S.sparse_mla_backward(q, big, slots, SCALE, out, lse, dout, ws=ws)
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]  # over what was freed, if it was
    for _ in range(2):
        for g, got, want, _ in made:
            for x in got:
                x.fill_(7)
            g.replay()
        torch.cuda.synchronize()
        for g, got, want, (q, kv, slots, out, lse, dout) in made:
            assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
            ref, bound = R.backward(q.cpu(), kv.data.cpu(), slots.cpu().long(), SCALE, out.cpu(), lse.cpu(), dout.cpu())
            R.within(got[1], ref[1], bound[1])
    del junk


def test_backward_and_append_past_32_bit_offsets(S):
    """A cache of 4.6 GB: rows at both ends, and beyond 2^31 and 2^32 bytes."""
    n, H, T = 4_000_000, 16, 2
    cache = torch.zeros((n, 576), dtype=torch.bfloat16, device="cuda")
    kv = S.KVCache(cache, n // 64, 64, W.KV_BF16)
    spots = torch.tensor([0, 1, (1 << 31) // 1152 + 1, (1 << 32) // 1152 + 1, n - 2, n - 1], dtype=torch.int32)
    lat, kr = normal(90, 6, 512), normal(91, 6, 64)
    f = S.rope_frequencies(64)
    ws = S.Workspace()
    pos = torch.arange(6, dtype=torch.int32)
    S.rope_append(lat.cuda(), kr.cuda(), pos.cuda(), spots.cuda(), kv, f, ws=ws)
    rows = cache[spots.long().cuda()].cpu()
    assert torch.equal(rows[:, :512], lat)
    assert int(torch.count_nonzero(cache[:, 0])) <= 6
    q, dout = normal(92, T, H, 576).cuda(), normal(93, T, H, 512).cuda()
    topk = torch.stack([spots, spots.flip(0)]).cuda()
    out, lse = forward(S, q, kv, topk)
    dq, dkv, w = S.sparse_mla_backward(q, kv, topk, SCALE, out, lse, dout, return_weights=True, ws=ws)
    assert ws.read_status() == 0
    small = torch.arange(6).repeat(T, 1)
    small[1] = small[1].flip(0)
    ref, bound = R.backward(q.cpu(), rows, small, SCALE, out.cpu(), lse.cpu(), dout.cpu())
    for a, b, c in zip((dq, dkv[spots.long().cuda()], w), ref, bound):
        R.within(a, b, c)
    dkv[spots.long().cuda()] = 0
    assert not dkv.any()


def test_backward_wait_that_runs_out_is_reported_and_the_next_call_is_clean(S):
    T, H, K, n = 3, 40, 200, 300
    kv = S.KVCache(normal(94, n, 576).cuda(), n, 1, W.KV_BF16)
    q, dout, slots = normal(95, T, H, 576).cuda(), normal(96, T, H, 512).cuda(), lists(97, T, K, n).cuda()
    out, lse = forward(S, q, kv, slots)
    ws = S.Workspace()
    args = (q, kv, slots, SCALE, out, lse, dout)
    want = S.sparse_mla_backward(*args, return_weights=True, ws=ws)
    assert ws.read_status() == 0
    S.debug_pipeline_fault(1, 2_000_000)
    try:
        S.sparse_mla_backward(*args, return_weights=True, ws=ws)
        assert ws.read_status() == S.svt.DEV_ERR_TIMEOUT
    finally:
        S.debug_pipeline_fault()
    got = S.sparse_mla_backward(*args, return_weights=True, ws=ws)
    assert ws.read_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("T,H,K", [(40, 16, 700), (300, 32, 130), (40, 64, 700), (170, 128, 200)])
def test_backward_wait_that_runs_out_with_several_tiles_a_cta(S, T, H, K):
    """A CTA whose first wait gave up has tiles left to walk: it adds to no row that no list names, and writes
    nothing outside its outputs and its part of the workspace."""
    n, listed = 900, 800
    kv = S.KVCache(normal(110, n, 576).cuda(), n, 1, W.KV_BF16)
    q, dout, slots = normal(111, T, H, 576).cuda(), normal(112, T, H, 512).cuda(), lists(113, T, K, listed).cuda()
    out, lse = forward(S, q, kv, slots)
    need = S.svt.lib().svt_sparse_mla_backward_workspace_size(T, H, K, n)
    ws = S.Workspace(nbytes=need + (1 << 20))
    ws.buf[need:] = 90
    wide_q = torch.full((T + 2, H, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    wide_kv = torch.full((n + 2, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    run = lambda: S.sparse_mla_backward(  # noqa: E731
        q, kv, slots, SCALE, out, lse, dout, dq=wide_q[1:-1], dkv=wide_kv[1:-1], return_weights=True, ws=ws)
    want = [x.clone() for x in run()]
    assert ws.read_status() == 0
    S.debug_pipeline_fault(1, 2_000_000)
    try:
        _, dkv, _ = run()
        assert ws.read_status() == S.svt.DEV_ERR_TIMEOUT
    finally:
        S.debug_pipeline_fault()
    assert not dkv[listed:].any()
    for wide in (wide_q, wide_kv):
        assert bool((wide[0] == 3).all()) and bool((wide[-1] == 3).all())
    assert bool((ws.buf[need:] == 90).all())
    got = run()
    assert ws.read_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    ref, bound = R.backward(q.cpu(), kv.data.cpu(), slots.cpu().long(), SCALE, out.cpu(), lse.cpu(), dout.cpu())
    R.within(got[1], ref[1], bound[1])


def test_backward_refused_calls_allocate_nothing(S):
    """The library's refusal comes before the workspace grows and before dq and dkv are made."""
    n = 4096
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    good = S.KVCache(z(n, 576), n, 1, W.KV_BF16)
    e4m3 = S.KVCache(z(n, 656, d=torch.uint8), n, 1, W.KV_FP8_E4M3)
    # rows that no memory holds: page counts of 2^40, and of 2^62 pages of 4 (2^64 rows wrap to none)
    huge = S.KVCache(good.data, 1 << 40, 1, W.KV_BF16)
    wraps = S.KVCache(good.data, 1 << 62, 4, W.KV_BF16)
    unsupported, invalid = S.svt.SVT_ERR_UNSUPPORTED, S.svt.SVT_ERR_INVALID_ARG
    for kv, H, kw, status in ((e4m3, 4, {}, unsupported), (good, 129, {}, unsupported), (huge, 4, {}, unsupported),
                              (wraps, 4, {}, unsupported), (good, 4, dict(scale=math.inf), invalid)):
        args = (z(1, H, 576), kv, z(1, 2, d=torch.int32), kw.get("scale", SCALE), z(1, H, 512), z(1, H, d=torch.float32),
                z(1, H, 512))
        ws = S.Workspace()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with pytest.raises(S.SvtError) as e:
            S.sparse_mla_backward(*args, ws=ws)
        assert e.value.status == status
        assert ws.nbytes == 256 and torch.cuda.max_memory_allocated() == before


def test_backward_empty_block_table_is_refused(S):
    """A table of no requests, or of no pages, resolves nothing (and is not the same as none)."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    kv, i32 = S.KVCache(z(64, 576), 64, 1, W.KV_BF16), torch.int32
    for shape in ((0, 3), (2, 0)):
        bt = z(*shape, d=i32)
        for T, refused in ((1, True), (0, False)):
            q, topk, ws = z(T, 4, 576), z(T, 2, d=i32), S.Workspace()
            out, lse = z(T, 4, 512), z(T, 4, d=torch.float32)
            calls = (lambda: S.sparse_mla_decode(q, kv, topk, SCALE, block_table=bt, ws=ws),
                     lambda: S.resolve_topk_slots(topk, block_table=bt, num_pages=64, ws=ws),
                     lambda: S.sparse_mla_backward(q, kv, topk, SCALE, out, lse, out, block_table=bt, ws=ws))
            for call in calls:
                if refused:
                    with pytest.raises(S.SvtError, match="num_reqs"):
                        call()
                else:
                    call()
