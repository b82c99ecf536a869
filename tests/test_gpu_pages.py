"""svt_fork_pages and svt_compact_pages against a list of pages on the host."""

import numpy as np
import pytest
import torch

import sparse_mla_attention_top_gb300 as S
from sparse_mla_attention_top_gb300 import svt
from tests import _serving_ref as R

pytestmark = pytest.mark.gpu
KIND = {"bf16": (S.KV_BF16, 1152), "e4m3": (S.KV_FP8_E4M3, 656)}


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


class Pool:
    """Rows of the given lengths over shuffled pages; rows of one family share the pages before their `shared` tokens."""

    def __init__(self, families, page, spare, kind="bf16", seed=0, blocks=None, stride=0):
        r = np.random.default_rng(seed)
        need = sum(shared // page + sum(-(-n // page) - shared // page for n in lens) for shared, lens in families)
        self.pages, self.page, self.kind = need + spare, page, kind
        order, used = r.permutation(self.pages), 0
        self.lens = [n for _, lens in families for n in lens]
        self.blocks = blocks or max([1] + [-(-n // page) for n in self.lens])
        self.table = np.full((len(self.lens), self.blocks), -1, np.int32)
        row = 0
        for shared, lens in families:
            full = shared // page
            base = order[used:used + full]
            used += full
            for n in lens:
                more = -(-n // page) - full
                self.table[row, :full] = base
                self.table[row, full:full + more] = order[used:used + more]
                used += more
                row += 1
        self.refs = np.bincount(self.table[self.table >= 0], minlength=self.pages).astype(np.int32)
        self.dtype, self.row_bytes = KIND[kind]
        self.stride = stride
        self.data = torch.randint(0, 256, (self.pages * page, stride or self.row_bytes), dtype=torch.uint8, device="cuda")

    def kv(self, data):
        return S.KVCache(data, self.pages, self.page, self.dtype, row_stride_bytes=self.stride)

    def fork(self, parents, grow, max_grow=None, blocks=None, in_place=True, ws=None):
        data, refs = self.data.clone(), i32(self.refs)
        kw = {} if in_place else {"refs_out": torch.full_like(refs, -9)}
        each = grow if isinstance(grow, int) else i32(grow)
        got = S.fork_pages(self.kv(data), refs, i32(self.table), i32(self.lens), i32(parents),
                           grow=each, max_grow=max_grow, max_blocks=blocks, ws=ws, **kw)
        return got, refs, data

    def check_fork(self, parents, grow, blocks=None, in_place=True):
        parents = list(parents)
        each = [grow] * len(parents) if isinstance(grow, int) else list(grow)
        most = max([1] + each) if not isinstance(grow, int) else grow
        ws = S.Workspace()
        (table, lens, slots, refs), given, data = self.fork(parents, grow, None if isinstance(grow, int) else most, blocks,
                                                            in_place, ws)
        want = R.fork(self.refs, self.table, self.lens, parents, each, self.page, blocks or self.blocks, most)
        assert want is not None and ws.read_status() == 0
        for name, a, b in zip(("table", "lens", "slots", "refs"), (table, lens, slots, refs), want):
            assert np.array_equal(a.cpu().numpy(), b), name
        assert (refs is given) == in_place
        if not in_place:
            assert np.array_equal(given.cpu().numpy(), self.refs)
        rows = self.data.clone()
        for src, dst, n in want[4]:
            a, b = src * self.page, dst * self.page
            rows[b:b + n, :self.row_bytes] = self.data[a:a + n, :self.row_bytes]
        assert torch.equal(rows, data)
        counts = np.bincount(want[0][want[0] >= 0], minlength=self.pages)
        assert np.array_equal(want[3], counts)  # (all pages are this table's)
        return want


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
def test_a_step_of_a_beam_search(kind, page):
    p = Pool([(100, [105, 131, 100, 128]), (7, [9, 8, 7, 64])], page, 300, kind, seed=page)
    p.check_fork([1, 1, 0, 3, 7, 5, 5, 5], 1, blocks=140 // page + 2)


@pytest.mark.parametrize("in_place", [True, False])
def test_samples_admission_and_release(in_place):
    p = Pool([(0, [77]), (0, [1]), (0, [64]), (0, [0])], 16, 400, seed=1)
    r = np.random.default_rng(2)
    parents = [0] * 9 + [-1, 2, -1, 3] + [2] * 3
    p.check_fork(parents, r.integers(0, 90, len(parents)), blocks=20, in_place=in_place)


def test_pages_are_whole_and_rows_stay():
    p = Pool([(0, [32, 48])], 16, 0, seed=3)
    want = p.check_fork([0, 1, 1, 0], 0)
    assert not want[4] and np.array_equal(want[0], p.table[[0, 1, 1, 0]])


def test_a_begun_page_that_others_hold_is_copied_for_each():
    p = Pool([(0, [20, 20])], 16, 4, seed=4)
    p.table[1] = p.table[0]  # both rows hold the same two pages
    p.refs = np.bincount(p.table[p.table >= 0], minlength=p.pages).astype(np.int32)
    want = p.check_fork([0, 1], 1)
    assert len(want[4]) == 2


def test_everything_ends():
    p = Pool([(30, [40, 50, 33])], 8, 5, seed=5)
    want = p.check_fork([], 1)
    assert want[0].shape == (0, p.blocks) and not want[3].any()
    p.check_fork([-1, -1], 0)


def test_no_old_rows():
    p = Pool([], 16, 12, seed=6, blocks=4)
    p.check_fork([-1, -1, -1], [17, 0, 33], blocks=4)


def test_the_last_free_page():
    p = Pool([(0, [16, 16])], 16, 2, seed=7)
    p.check_fork([0, 1], 1, blocks=2)
    p.check_fork([0, 0], [16, 1], blocks=2)


def void(p, bit, *args, **kw):
    ws = S.Workspace()
    for in_place in (True, False):
        (table, lens, slots, refs), given, data = p.fork(*args, in_place=in_place, ws=ws, **kw)
        assert ws.read_status() == bit
        assert (table == -1).all() and (lens == 0).all() and (slots == -1).all()
        assert np.array_equal(refs.cpu().numpy(), p.refs) and torch.equal(data, p.data)


def test_too_few_pages_change_nothing():
    # a copy of row 1's begun page and a page for row 0's growth: one more than there are
    p = Pool([(0, [16, 20])], 16, 1, seed=8)
    void(p, svt.DEV_ERR_NO_PAGES, [1, 1, 0], 1, blocks=4)
    void(p, svt.DEV_ERR_NO_PAGES, [-1], 33, blocks=4)


def test_arguments_out_of_range_change_nothing():
    def pool():
        return Pool([(0, [16, 20, 3])], 16, 9, seed=9)
    bit = svt.DEV_ERR_INDEX_RANGE
    void(pool(), bit, [0, 3], 1, blocks=4)
    void(pool(), bit, [0, -2], 1, blocks=4)
    void(pool(), bit, [0, 1], [0, -1], max_grow=4, blocks=4)
    void(pool(), bit, [0, 1], [0, 5], max_grow=4, blocks=4)
    void(pool(), bit, [0, 1], [20, 0], max_grow=20, blocks=2)  # past the table's width
    for at, value in (((1, 1), -1), ((1, 1), 10 ** 6), ((2, 0), -7)):
        p = pool()
        p.table[at] = value
        void(p, bit, [0, 1], 1, blocks=4)
    for n in (-1, 33):
        p = pool()
        p.lens[2] = n
        void(p, bit, [0], 1, blocks=4)
    p = pool()
    p.refs[p.table[0, 0]] = 0  # a page in use without a count
    void(p, bit, [0], 1, blocks=4)


def test_many_rows():
    r = np.random.default_rng(10)
    p = Pool([(int(s), (s + r.integers(0, 40, 8)).tolist()) for s in r.integers(0, 300, 250)], 16, 9000, seed=10)
    p.check_fork(r.integers(-1, 2000, 3000), r.integers(0, 30, 3000), blocks=30)


def test_a_large_pool():
    # several words and chunks without a free page, several chunks in a CTA's share
    p = Pool([(0, [5000] * 60)], 1, 700_000, seed=11, kind="e4m3")
    want = p.check_fork(list(range(60)) + [0, 5], 3, blocks=5010)
    assert len(want[4]) == 0  # pages of one row are never begun


def test_strided_rows():
    p = Pool([(40, [45, 52])], 16, 20, seed=12, stride=1200)
    p.check_fork([0, 0, 1, 1, 1], 2, blocks=6)


# ------------------------------------------------------------------------------------ compacting

def check_compact(pages, refs, table, page, kind="bf16", in_place=True, stride=0):
    dtype, row = KIND[kind]
    data = torch.randint(0, 256, (pages * page, stride or row), dtype=torch.uint8, device="cuda")
    before = data.clone()
    r, t = i32(refs), i32(table)
    kw = {} if in_place else {"refs_out": torch.full_like(r, -9), "table_out": torch.full_like(t, -9)}
    ws = S.Workspace()
    got_t, got_r, mapping = S.compact_pages(S.KVCache(data, pages, page, dtype, row_stride_bytes=stride), r, t, ws=ws, **kw)
    want_t, want_r, want_m, moves = R.compact(refs, table)
    status = ws.read_status()
    assert np.array_equal(got_t.cpu().numpy(), want_t) and np.array_equal(mapping.cpu().numpy(), want_m)
    assert np.array_equal(got_r.cpu().numpy(), want_r)
    assert (got_t is t) == in_place and (got_r is r) == in_place
    view, old = data.view(pages, page, -1), before.view(pages, page, -1)
    if moves:
        src, dst = (torch.tensor([m[i] for m in moves], device="cuda") for i in (0, 1))
        old = old.clone()
        old[dst, :, :row] = before.view(pages, page, -1)[src][:, :, :row]
    assert torch.equal(view, old)
    return status


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("pages, page, live", [(1, 16, 1.0), (1, 1, 0.0), (33, 16, 0.5), (64, 3, 0.9), (1000, 64, 0.3),
                                               (5000, 1, 0.6), (40000, 1, 0.02), (2049, 16, 0.98)])
def test_compact(pages, page, live, kind, in_place):
    r = np.random.default_rng(pages)
    used = r.random(pages) < live
    refs = np.where(used, r.integers(1, 5, pages), 0).astype(np.int32)
    at = np.flatnonzero(used)
    table = np.full((7, 50), -1, np.int32)
    if len(at):
        table[:, :40] = r.choice(at, (7, 40))
    assert check_compact(pages, refs, table, page, kind, in_place) == 0


def test_compact_leaves_a_dense_pool_and_an_empty_one():
    assert check_compact(70, np.ones(70, np.int32), np.arange(70).reshape(7, 10), 16) == 0
    assert check_compact(70, np.zeros(70, np.int32), np.full((3, 2), -1), 16) == 0
    assert check_compact(70, np.r_[np.zeros(35), np.ones(35)].astype(np.int32), np.arange(35, 70), 16) == 0


def test_compact_reports_entries_that_are_no_live_pages():
    refs = np.array([0, 1, 0, 2, 1], np.int32)
    for bad in (0, 2, 5, 10 ** 6):
        assert check_compact(5, refs, np.array([[1, 3, bad, -4, 4]]), 16) == svt.DEV_ERR_INDEX_RANGE


def test_compact_strided_rows():
    refs = np.array([0, 1, 0, 2, 1, 0, 0, 3], np.int32)
    assert check_compact(8, refs, np.array([[1, 3, 4, 7]]), 16, stride=1168) == 0
    assert check_compact(8, refs, np.array([[1, 3, 4, 7]]), 16, "e4m3", stride=672) == 0


def test_without_a_table():
    refs = np.array([0, 1, 0, 2], np.int32)
    assert check_compact(4, refs, np.zeros((0, 5), np.int32), 16) == 0


def test_compact_a_large_pool():
    # moves past 2^31 bytes: 2.6 GB
    pages, page = 35000, 64
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[5:1000] = 0
    data = torch.zeros((pages, page * 1152), dtype=torch.uint8, device="cuda")
    data[:, 0] = torch.arange(pages, device="cuda").to(torch.uint8)
    data[:, -1] = (torch.arange(pages, device="cuda") // 256).to(torch.uint8)
    kv = S.KVCache(data.view(pages * page, 1152), pages, page, S.KV_BF16)
    table, refs, mapping = S.compact_pages(kv, refs, torch.arange(34000, pages, dtype=torch.int32, device="cuda"))
    src = torch.arange(34005, pages, device="cuda")
    assert torch.equal(data[5:1000, 0], src.to(torch.uint8))
    assert torch.equal(data[5:1000, -1], (src // 256).to(torch.uint8))
    assert int(refs.sum()) == 34005 and int((refs[34005:]).sum()) == 0
    assert torch.equal(table[5:], torch.arange(5, 1000, dtype=torch.int32, device="cuda"))


def test_graphs():
    p = Pool([(100, [105, 131, 100, 128])], 16, 50, seed=20)
    ws = S.Workspace()
    table, refs, lens, parents = i32(p.table), i32(p.refs), i32(p.lens), i32([2, 0, 0, 1])
    out = torch.empty_like(refs)
    kv = p.kv(p.data)
    first = S.fork_pages(kv, refs, table, lens, parents, grow=2, max_blocks=12, refs_out=out, ws=ws)
    first = [x.clone() for x in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        second = S.fork_pages(kv, refs, table, lens, parents, grow=2, max_blocks=12, refs_out=out, ws=ws)
        moved = S.compact_pages(kv, second[3], second[0], refs_out=torch.empty_like(refs),
                                table_out=torch.empty_like(second[0]), ws=ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second)) and ws.read_status() == 0
    want = R.compact(first[3].cpu().numpy(), first[0].cpu().numpy())
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(moved, want))


def test_refused_tensors():
    p = Pool([(0, [16, 20])], 16, 4)
    with pytest.raises(ValueError):
        S.fork_pages(p.kv(p.data), i32(p.refs), i32(p.table), i32(p.lens), i32([0]), grow=i32([1]))
    with pytest.raises(TypeError):
        S.fork_pages(p.kv(p.data), i32(p.refs)[:2], i32(p.table), i32(p.lens), i32([0]))
    with pytest.raises(TypeError):
        S.fork_pages(p.kv(p.data), i32(p.refs), i32(p.table).long(), i32(p.lens), i32([0]))
    for kw in (dict(grow=-1), dict(grow=2, max_grow=1), dict(max_blocks=-5), dict(grow=0, max_grow=-3)):
        with pytest.raises(S.SvtError):
            S.fork_pages(p.kv(p.data), i32(p.refs), i32(p.table), i32(p.lens), i32([0]), **kw)
    with pytest.raises(TypeError):
        S.compact_pages(p.kv(p.data), i32(p.refs), i32(p.table).t())


@pytest.mark.parametrize("rows, grow", [(1024, 1 << 21), (2048, 1 << 20), (2048, 1 << 21)])
def test_growths_beyond_32_bits_change_nothing(rows, grow):
    # pages of one token: rows x grow of them are 2^31 (in one round of the plan's sum, and in two) and 2^32, of 70 free ones
    free, _ = torch.cuda.mem_get_info()
    assert free > 12 * rows * grow
    p = Pool([(0, [16, 20])], 1, 70, seed=21)
    refs, data, ws = i32(p.refs), p.data.clone(), S.Workspace()
    table, lens, slots, _ = S.fork_pages(p.kv(data), refs, i32(p.table), i32(p.lens), i32([-1] * rows), grow=grow,
                                         max_blocks=grow, ws=ws)
    assert ws.read_status() == svt.DEV_ERR_NO_PAGES
    assert int(table.amax()) == int(table.amin()) == -1 and int(slots.amax()) == int(slots.amin()) == -1 and not lens.any()
    assert np.array_equal(refs.cpu().numpy(), p.refs) and torch.equal(data, p.data)
    del table, slots
    torch.cuda.empty_cache()
