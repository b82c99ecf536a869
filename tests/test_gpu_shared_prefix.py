"""svt_mla_decode_shared_prefix against 64-bit attention over each query's own rows."""

import numpy as np
import pytest
import torch

import sparse_mla_attention_top_gb300 as S
from sparse_mla_attention_top_gb300 import svt
from tests import _serving_ref as R

pytestmark = pytest.mark.gpu
SCALE = 576 ** -0.5


def dev():
    return torch.device("cuda", torch.cuda.current_device())


def make_cache(g, rows, kind):
    if kind == "bf16":
        return torch.randn((rows, 576), generator=g, device=dev()).to(torch.bfloat16).view(torch.uint8)
    codes = torch.randn((rows, 512), generator=g, device=dev()).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = (torch.rand((rows, 4), generator=g, device=dev()) * 1.5 + 0.5).view(torch.uint8)
    rope = torch.randn((rows, 64), generator=g, device=dev()).to(torch.bfloat16).view(torch.uint8)
    return torch.cat([codes, scales, rope], 1).contiguous()


class Case:
    """Groups of (queries' lengths, prefix length) over a pool of shuffled pages; unused rows of the pool are NaN."""

    def __init__(self, groups, H, page, kind="bf16", seed=0, gap=0, tail=0, q_scale=1.0, share_pages=True):
        g = torch.Generator(device=dev())
        g.manual_seed(seed)
        r = np.random.default_rng(seed)
        self.kind, self.page, self.H = kind, page, H
        lens = [0] * gap + [n for ls, _ in groups for n in ls] + [0] * tail
        T = len(lens)
        self.T, self.lens = T, lens
        need = sum(-(-max(n, p) // page) for ls, p in groups for n in ls + [p]) + 1
        blocks = max([1] + [-(-max([p] + ls) // page) for ls, p in groups])
        pages = r.permutation(need + 3)
        table, used = np.full((T, blocks), -1, np.int32), 0
        self.start, self.prefix = [gap], []
        first = gap
        lists = [[] for _ in range(T)]
        copies = []
        for ls, p in groups:
            n_pre = -(-min(p, max(ls + [0])) // page) if ls else 0
            base = pages[used:used + n_pre]
            used += n_pre
            for i, n in enumerate(ls):
                t = first + i
                full = min(p, n) // page if share_pages else 0
                own = max(0, -(-n // page) - full)
                table[t, :n_pre] = base
                if n > p or not share_pages:
                    mine = pages[used:used + own]
                    used += own
                    table[t, full:full + own] = mine
                    # content below the prefix is the same
                    for j in range(full, min(n_pre, full + own)):
                        copies.append((base[j], mine[j - full]))
                pos = np.arange(n)
                row = np.where(pos < p, base[np.minimum(pos // page, max(n_pre - 1, 0))] if n_pre else 0,
                               table[t, np.minimum(pos // page, blocks - 1)])
                lists[t] = row * page + pos % page
            if ls and n_pre:
                table[first, :n_pre] = np.where(np.arange(n_pre) < -(-max(ls[0], 0) // page), table[first, :n_pre], base)
            first += len(ls)
            self.start.append(first)
            self.prefix.append(p)
        num_pages = need + 3
        self.cache = make_cache(g, num_pages * page, kind)
        view = self.cache.view(num_pages, -1)
        for a, b in copies:
            view[int(b)] = view[int(a)]
        rows = R.cache_rows(self.cache, kind)
        # what no query attends to holds NaN
        live = np.zeros(num_pages * page, bool)
        for ls in lists:
            live[ls] = True
        for t in range(T):  # a first query's own copy of prefix rows is read in place of the base's
            for pos in range(lens[t]):
                pg = table[t, pos // page]
                if pg >= 0:
                    live[pg * page + pos % page] = True
        dead = torch.from_numpy(np.flatnonzero(~live)).to(dev())
        self.cache[dead] = 0xFF if kind == "bf16" else 0x7F
        self.rows, self.lists = rows, lists
        self.q = (torch.randn((T, H, 576), generator=g, device=dev()) * q_scale).to(torch.bfloat16)
        self.kv = S.KVCache(self.cache, num_pages, page, S.KV_BF16 if kind == "bf16" else S.KV_FP8_E4M3)
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev())  # noqa: E731
        self.table, self.len_t, self.start_t, self.prefix_t = i32(table), i32(lens), i32(self.start), i32(self.prefix)

    def run(self, ws=None, **kw):
        return S.mla_decode_shared_prefix(self.q, self.kv, self.table, self.len_t, self.start_t, self.prefix_t, SCALE,
                                          ws=ws, **kw)

    def want(self):
        return R.attention(self.q, self.rows, self.lists, SCALE, self.kind)

    def check(self):
        ws = S.Workspace()
        got = self.run(ws)
        assert ws.read_status() == 0
        R.check_attention(got, self.want())
        return got


def beams(n, prefix, own):
    return [prefix + (own * (i + 1)) // n for i in range(n)], prefix


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 16, 24, 64])
@pytest.mark.parametrize("prefix, own", [(128, 0), (127, 1), (129, 33), (500, 17), (16, 140), (1, 1)])
def test_one_group(kind, page, prefix, own):
    Case([beams(5, prefix, own)], 16, page, kind, seed=prefix + own).check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H", [1, 3, 8, 40, 64, 127, 128])
def test_heads(kind, H):
    Case([beams(6, 300, 40), beams(3, 70, 200)], H, 16, kind, seed=H).check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_single_tokens(kind):
    Case([([1], 0), ([1], 1), ([2], 1), ([17], 16)], 16, 16, kind).check()


def test_nothing_is_shared():
    Case([([700, 3, 128], 0)], 64, 64).check()


def test_everything_is_shared_and_lengths_are_causal():
    # the new tokens of one request: the prefix is all of it, each keeps to its own length
    Case([(list(range(190, 230)), 229)], 16, 64, seed=3).check()


def test_queries_shorter_than_the_prefix_and_empty_ones():
    Case([([0, 5, 300, 0, 299, 301, 16], 300), ([0, 0], 40), ([], 7), ([9], 100)], 16, 16, seed=4).check()


def test_all_queries_empty():
    c = Case([([0, 0, 0], 0), ([0], 5)], 64, 16)
    out, lse = c.check()
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_long_prefix_cut_between_ctas(kind):
    Case([beams(4, 9000, 100)], 16, 64, kind, seed=5).check()


def test_several_row_tiles_and_groups():
    Case([beams(9, 1500, 300), beams(1, 64, 0), beams(20, 640, 31), ([2000], 3)], 64, 64, seed=6).check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("groups", [[([20], 0)] * 1100, [beams(24, 6000, 300)],
                                    [beams(7, 5000, 900), ([4000], 0), beams(9, 100, 900), ([], 5), ([0], 3), ([6000] * 4, 6000)]],
                         ids=["short", "long", "mixed"])
def test_more_tiles_than_a_few_a_pair(kind, groups):
    # enough of them to be dealt out by what they cost: row tiles of a single tile, of a prefix and own rows, of either only
    Case(groups, 128, 64, kind, seed=26).check()


@pytest.mark.parametrize("page", [64, 128, 192])
@pytest.mark.parametrize("prefix", [0, 63, 500, 512, 1001])
def test_many_own_rows(page, prefix):
    # beside queries with few, and with none
    lens = [prefix + n for n in (255, 256, 257, 300, 0, 17, 511, 640)]
    Case([(lens, prefix), ([prefix + 400, prefix + 3], prefix)], 40, page, seed=prefix + page).check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pages_of_48_rows(kind):
    Case([beams(7, 700, 100), beams(2, 47, 2)], 16, 48, kind, seed=20).check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_query_for_each_row_of_a_tile(kind):
    Case([beams(130, 300, 40)], 1, 16, kind, seed=21).check()


def test_more_queries_than_the_plan_keeps_at_hand():
    Case([beams(700, 40, 9)] + [([3], 1)] * 500 + [beams(300, 16, 2)], 3, 16, seed=22).check()


def test_values_of_all_sizes_where_a_tile_is_cut():
    # the parts of a cut tile are f16 with a scale for each 128 channels: what f16 could not hold lies in two such blocks,
    # whose channels the scores do not see
    c = Case([beams(4, 9000, 100)], 16, 64, seed=23)
    c.q[..., :256] = 0
    v = c.cache.view(torch.bfloat16)
    v[:, :128] *= 2.0 ** 90
    v[:, 128:256] *= 2.0 ** -60
    c.rows = torch.cat([c.rows[:, :128] * 2.0 ** 90, c.rows[:, 128:256] * 2.0 ** -60, c.rows[:, 256:]], 1)
    ws = S.Workspace()
    got = c.run(ws)
    assert ws.read_status() == 0
    want = c.want()
    for sl in (slice(0, 128), slice(128, 256), slice(256, 512)):
        R.check_attention((got[0][..., sl], got[1]), (want[0][..., sl], want[1], want[2][..., sl], want[3]))


def test_two_graphs_at_once():
    cases = [Case([beams(8, 3000, 100)], 16, 64, seed=s) for s in (24, 25)]
    graphs, outs = [], []
    for c in cases:
        c.run()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(c.run())
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for c, got in zip(cases, outs):
        R.check_attention(got, c.want())


def test_queries_of_no_group_are_left():
    c = Case([beams(3, 100, 9), beams(2, 50, 50)], 16, 16, gap=2, tail=3, seed=7)
    out = torch.full((c.T, 16, 512), 7.0, dtype=torch.bfloat16, device=dev())
    lse = torch.full((c.T, 16), 7.0, device=dev())
    c.run(out=out, lse=lse)
    R.check_attention((out, lse), c.want(), slice(2, c.T - 3))
    for sel in (slice(0, 2), slice(c.T - 3, c.T)):
        assert (out[sel] == 7).all() and (lse[sel] == 7).all()


def test_requests_of_tokens_and_strided_rows():
    c = Case([beams(4, 200, 20), beams(3, 90, 5)], 16, 16, seed=8)
    order = torch.randperm(c.T, device=dev())
    table = c.table[order].contiguous()
    req = torch.argsort(order).to(torch.int32)
    wide = torch.zeros((c.cache.shape[0], 1184), dtype=torch.uint8, device=dev())
    wide[:, :1152] = c.cache
    kv = S.KVCache(wide, c.kv.num_pages, 16, S.KV_BF16, row_stride_bytes=1184)
    got = S.mla_decode_shared_prefix(c.q, kv, table, c.len_t, c.start_t, c.prefix_t, SCALE, req_of_token=req)
    R.check_attention(got, c.want())


def test_large_scores_move_the_reference():
    Case([beams(6, 700, 90)], 64, 64, seed=9, q_scale=12.0).check()


def test_lse_is_optional_and_outputs_repeat():
    c = Case([beams(40, 3000, 200)], 64, 64, seed=10)
    a, lse = c.run()
    b, none = c.run(return_lse=False)
    assert none is None and torch.equal(a, b)


def test_empty_call():
    c = Case([beams(2, 30, 3)], 16, 16)
    out, lse = S.mla_decode_shared_prefix(c.q[:0], c.kv, c.table, c.len_t[:0], c.start_t[:1] * 0, c.prefix_t[:0], SCALE)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)


def test_pages_and_lengths_out_of_range_are_reported():
    for edit, bit in (("page", 1), ("len", 1), ("start", 1), ("prefix", 1), ("req", 1)):
        c = Case([beams(3, 100, 40)], 16, 16, seed=11)
        want = c.want()
        ws, req, ok = S.Workspace(), None, [0, 1, 2]
        if edit == "page":  # a page of query 1's own rows
            c.table[1, 7] = 10 ** 6
            ok = [0, 2]
        elif edit == "len":
            c.len_t[1] = -5
            ok = [0, 2]
        elif edit == "start":
            c.start_t[1] = 99
        elif edit == "prefix":
            c.prefix_t[0] = -1
        else:
            req = torch.tensor([0, 77, 2], dtype=torch.int32, device=dev())
            ok = [0, 2]
        got = c.run(ws, req_of_token=req)
        assert ws.read_status() == bit, edit
        if edit in ("len", "req"):
            assert not got[0][1].any() and torch.isneginf(got[1][1]).all()
        if edit != "prefix":
            R.check_attention(got, want, ok)


def test_rows_of_a_page_out_of_range_are_left_out():
    c = Case([([64, 64], 64)], 16, 16, seed=12)
    c.table[:, 2] = -3
    keep = np.r_[0:32, 48:64]
    c.lists = [np.asarray(x)[keep] for x in c.lists]
    ws = S.Workspace()
    got = c.run(ws)
    assert ws.read_status() == svt.DEV_ERR_INDEX_RANGE
    R.check_attention(got, c.want())


def test_e4m3_values_beyond_f16_are_reported():
    c = Case([beams(3, 60, 4)], 16, 16, "e4m3", seed=13)
    c.cache[:, 512:516] = torch.tensor([200.0], device=dev()).view(torch.uint8)
    ws = S.Workspace()
    c.run(ws)
    assert ws.read_status() & svt.DEV_ERR_FP8_RANGE
    c = Case([beams(3, 60, 4)], 16, 16, "e4m3", seed=13)
    c.q[1, 3, 70] = 1e6
    c.run(ws)
    assert ws.read_status() == svt.DEV_ERR_FP8_RANGE


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    for kind in ("bf16", "e4m3"):
        c = Case([beams(4, 600, 40)], 16, 64, kind, seed=14)
        ws = S.Workspace()
        c.run(ws)
        torch.cuda.synchronize()
        assert ws.read_status() == 0
        S.debug_pipeline_fault(1, 1_000_000)
        try:
            c.run(ws)
            torch.cuda.synchronize()
        finally:
            S.debug_pipeline_fault(0, 0)
        assert ws.read_status() & svt.DEV_ERR_TIMEOUT
        got = c.run(ws)
        assert ws.read_status() == 0
        R.check_attention(got, c.want())


def test_graph_replays_and_streams():
    c = Case([beams(8, 2000, 100)], 16, 64, seed=15)
    want = c.want()
    ws = S.Workspace()
    out, lse = c.run(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = c.run()
    torch.cuda.current_stream().wait_stream(side)
    R.check_attention(other, want)
    graph = torch.cuda.CUDAGraph()
    out, lse = torch.empty_like(out), torch.empty_like(lse)
    with torch.cuda.graph(graph):
        c.run(ws, out=out, lse=lse)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    assert ws.read_status() == 0
    R.check_attention((out, lse), want)
    # the captured call reads its inputs when it runs
    c.len_t.sub_(1)
    c.lists = [x[:-1] for x in c.lists]
    graph.replay()
    R.check_attention((out, lse), c.want())


def test_rows_past_32_bit_offsets():
    # a pool of 2.5 GB: its last pages' rows lie past 2^31 bytes
    pages, page = 34000, 64
    free, _ = torch.cuda.mem_get_info()
    assert free > 6e9
    g = torch.Generator(device=dev())
    g.manual_seed(16)
    cache = torch.empty((pages * page, 576), dtype=torch.bfloat16, device=dev())
    at = torch.tensor([pages - 1, 31500, 5, pages - 7], device=dev())
    cache.view(pages, page, 576)[at] = torch.randn((4, page, 576), generator=g, device=dev()).to(torch.bfloat16)
    q = torch.randn((2, 16, 576), generator=g, device=dev()).to(torch.bfloat16)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev())  # noqa: E731
    kv = S.KVCache(cache.view(torch.uint8), pages, page, S.KV_BF16)
    table = torch.stack([at[[0, 1, 2]], at[[0, 1, 3]]]).to(torch.int32)
    got = S.mla_decode_shared_prefix(q, kv, table, i32([150, 192]), i32([0, 2]), i32([128]), SCALE)
    lists = [np.arange(150), np.r_[0:128, 192:256]]
    rows = cache.view(pages, page, 576)[at].reshape(-1, 576).double()
    R.check_attention(got, R.attention(q, rows, lists, SCALE, "bf16"))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -SCALE, -0.5, 1e-30])
@pytest.mark.parametrize("groups, page", [([([37, 0, 130, 1], 30), ([5], 0)], 16), ([beams(5, 129, 33)], 24),
                                          ([beams(4, 9000, 100)], 64)], ids=["short", "rows", "cut"])
def test_scales_of_zero_negative_and_tiny(kind, scale, groups, page):
    """Any finite scale has its softmax (0: the mean of V). Lists that end inside tiles: what is masked stays masked."""
    c = Case(groups, 16, page, kind, seed=27)
    ws = S.Workspace()
    got = S.mla_decode_shared_prefix(c.q, c.kv, c.table, c.len_t, c.start_t, c.prefix_t, scale, ws=ws)
    assert ws.read_status() == 0
    out, lse, d_out, d_lse = R.attention(c.q, c.rows, c.lists, scale, kind)
    # log2 of a sum of up to 2^14 terms is off by at most two of its ulp, 2^-19, whatever the scores are
    R.check_attention(got, (out, lse, d_out, d_lse + 2.0 ** -19))


@pytest.mark.parametrize("kind, page", [("bf16", 64), ("bf16", 24), ("e4m3", 64)])
def test_outputs_repeat_to_the_bit(kind, page):
    # units by TMA, by TMA with zeroes put in, and by threads; P and units of both CTAs of a pair are read by the MMAs of one
    c = Case([beams(30, 1500, 300), beams(9, 700, 33)], 64, page, kind, seed=28)
    out, lse = c.check()
    for _ in range(30):
        again = c.run()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_a_call_may_take_longer_than_one_wait():
    # some 9 ms of tiles, where a wait gives up after 2
    pages, page, H, T, n = 6250, 64, 128, 128, 400_000
    g = torch.Generator(device=dev())
    g.manual_seed(29)
    kv = S.KVCache(make_cache(g, pages * page, "bf16"), pages, page, S.KV_BF16)
    q = torch.randn((T, H, 576), generator=g, device=dev()).to(torch.bfloat16)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev())  # noqa: E731
    table = torch.arange(pages, dtype=torch.int32, device=dev())[None]
    call = lambda: S.mla_decode_shared_prefix(q, kv, table, i32([n] * T), i32([0, T]), i32([n]), SCALE,  # noqa: E731
                                              req_of_token=i32([0] * T), ws=ws)
    ws = S.Workspace()
    want = call()
    torch.cuda.synchronize()
    S.debug_pipeline_fault(0, 2_000_000)
    try:
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        got = call()
        end.record()
        torch.cuda.synchronize()
    finally:
        S.debug_pipeline_fault(0, 0)
    assert begin.elapsed_time(end) > 4
    assert ws.read_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_no_wait_runs_out_whatever_the_number_of_tiles(kind):
    # a kernel leaves when the last arrival on each of its barriers has landed: as many as its tiles make, 0 to 9 a CTA pair
    page = 64
    pages = 2 * (76 * 9 + 1)
    g = torch.Generator(device=dev())
    g.manual_seed(30)
    cache = make_cache(g, pages * page, kind)
    kv = S.KVCache(cache, pages, page, S.KV_BF16 if kind == "bf16" else S.KV_FP8_E4M3)
    rows = R.cache_rows(cache, kind)
    q = torch.randn((4, 16, 576), generator=g, device=dev()).to(torch.bfloat16)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev())  # noqa: E731
    table = torch.arange(pages, dtype=torch.int32, device=dev())[None]
    scores = q.flatten(0, 1).double() @ rows.T * SCALE
    ws = S.Workspace()
    S.debug_pipeline_fault(0, 100_000_000)
    try:
        for tiles in [1, 2, 3, 7, 75, 76, 77] + [76 * m + r for m in range(1, 10) for r in (0, 1, 38)][2:-2]:
            n = 128 * tiles - 5
            _, lse = S.mla_decode_shared_prefix(q, kv, table, i32([n] * 4), i32([0, 4]), i32([n]), SCALE,
                                                req_of_token=i32([0] * 4), ws=ws)
            assert ws.read_status() == 0, tiles
            bound = 1.2e-3 if kind == "bf16" else 2.5e-2  # (576 2^-23 and 2^-10 of sums of magnitudes of some 20)
            assert float((lse.flatten().double() - scores[:, :n].logsumexp(1)).abs().amax()) < bound, tiles
    finally:
        S.debug_pipeline_fault(0, 0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [-1, 99])
def test_a_group_whose_first_request_is_out_of_range(kind, bad):
    # only the first query is without rows: the others keep the prefix, in each of the group's row tiles
    c = Case([beams(9, 700, 60), ([200, 3, 0, 150], 160), beams(2, 90, 9)], 64, 16, kind, seed=31)
    first = [0, 9]
    req = torch.arange(c.T, dtype=torch.int32, device=dev())
    req[first] = bad
    ws = S.Workspace()
    got = c.run(ws, req_of_token=req)
    assert ws.read_status() == svt.DEV_ERR_INDEX_RANGE
    assert not got[0][first].any() and torch.isneginf(got[1][first]).all()
    R.check_attention(got, c.want(), [t for t in range(c.T) if t not in first])
    # a group of which nobody has a request
    req[9:13] = bad
    got = c.run(ws, req_of_token=req)
    assert ws.read_status() == svt.DEV_ERR_INDEX_RANGE
    assert not got[0][9:13].any() and torch.isneginf(got[1][9:13]).all()
    R.check_attention(got, c.want(), list(range(1, 9)) + [13, 14])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("groups, page", [([([1, 2, 9, 10, 17], 1)], 16), ([beams(7, 500, 300), beams(3, 33, 5)], 16),
                                          ([beams(5, 129, 33)], 24), ([beams(24, 3000, 100)], 64)],
                         ids=["few", "own", "rows", "cut"])
def test_lse_of_scores_without_rounding(kind, groups, page):
    # whole numbers: the scores' sums are exact, and what is left is a hundred-thousandth. A row too many or too few, or codes
    # times scales rounded to f16, is more (tests/test_serving_bounds.py)
    scale = 2.0 ** -8
    c = Case(groups, 16, page, kind, seed=32)
    c.q, cache = R.whole_numbers(c.q, c.cache, kind)
    c.cache.copy_(cache)
    ws = S.Workspace()
    _, lse = S.mla_decode_shared_prefix(c.q, c.kv, c.table, c.len_t, c.start_t, c.prefix_t, scale, ws=ws)
    assert ws.read_status() == 0
    want, bound = R.lse_of_whole_numbers(c.q, R.cache_rows(c.cache, kind), c.lists, scale, kind)
    assert bool(((lse.double() - want).abs() <= bound).all()), float(((lse.double() - want).abs() / bound).max())


def test_more_tiles_than_a_few_a_pair_in_pages_of_24_rows():
    # loaded by threads, whose tiles cost the same whether rows are shared or not
    Case([beams(7, 5000, 900), ([4000], 0), beams(9, 100, 900), ([], 5), ([0], 3), ([6000] * 4, 6000)], 128, 24, seed=33).check()
