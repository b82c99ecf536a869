"""Workspaces: calls that are given none, on streams, in threads and in graphs at once."""

import threading

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


class Step:
    """A split decode and its backward pass on inputs of a seed, with the results of calls made one by one."""

    def __init__(self, S, seed, T=24, H=64, K=300, n=500):
        g = torch.Generator().manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
        self.S = S
        self.kv = S.KVCache(normal(n, 576).cuda(), n, 1, W.KV_BF16)
        self.q, self.dout = normal(T, H, 576).cuda(), normal(T, H, 512).cuda()
        self.topk = torch.stack([torch.randperm(n, generator=g)[:K] for _ in range(T)]).to(torch.int32).cuda()
        self.want = self.run(S.Workspace())
        torch.cuda.synchronize()
        cpu = lambda t: t.cpu()  # noqa: E731
        self.ref, self.bound = R.backward(cpu(self.q), cpu(self.kv.data), cpu(self.topk).long(), SCALE, cpu(self.want[0]),
                                          cpu(self.want[1]), cpu(self.dout))

    def run(self, ws=None):
        out, lse = self.S.sparse_mla_decode(self.q, self.kv, self.topk, SCALE, num_splits=3, ws=ws)
        return out, lse, *self.S.sparse_mla_backward(self.q, self.kv, self.topk, SCALE, out, lse, self.dout,
                                                     return_weights=True, ws=ws)

    def check(self, got):
        for i in (0, 1, 2, 4):  # all but the cache rows' sums repeat exactly
            assert torch.equal(got[i], self.want[i]), i
        R.within(got[3], self.ref[1], self.bound[1])


def test_default_workspaces_on_two_streams_at_once(S):
    steps = [Step(S, 1), Step(S, 2, T=30, H=16, K=200)]
    streams = [torch.cuda.Stream() for _ in steps]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(8):
        for step, stream, out in zip(steps, streams, got):
            with torch.cuda.stream(stream):
                out.append(step.run())
    torch.cuda.synchronize()
    for step, stream, out in zip(steps, streams, got):
        for x in out:
            step.check(x)
        with torch.cuda.stream(stream):
            assert S.svt.default_workspace().read_status() == 0


def test_default_workspace_of_threads_on_one_stream(S):
    steps = [Step(S, 3), Step(S, 4, T=30, H=16, K=200), Step(S, 5, T=7, H=128, K=400)]
    got, errors = [[] for _ in steps], []

    def loop(step, out):
        try:
            for _ in range(8):
                out.append(step.run())
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=loop, args=a) for a in zip(steps, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for step, out in zip(steps, got):
        for x in out:
            step.check(x)
    assert S.svt.default_workspace().read_status() == 0


def test_default_workspaces_of_graphs_replayed_at_once(S):
    """Captured by the same stream, as torch.cuda.graph does; the second graph is the larger one."""
    steps = [Step(S, 6), Step(S, 7, T=60, H=64, K=400)]
    graphs, got = [], []
    for step in steps:
        step.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(step.run())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(4):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        steps[0].run()  # beside them, on the current stream
    torch.cuda.synchronize()
    for step, x in zip(steps, got):
        step.check(x)


def test_outgrown_buffers_are_kept_for_captured_calls_alone(S):
    step = Step(S, 8)
    ws = S.Workspace()
    torch.cuda.synchronize()
    for n in (1 << 20, 1 << 28, (1 << 28) + 1):
        before = torch.cuda.memory_allocated() - ws.nbytes
        ws.ensure(n)
        assert ws.nbytes == n and torch.cuda.memory_allocated() - n <= before + 512
    ws = S.Workspace()
    step.run(ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step.run(ws)
    used, bad = ws.buf.data_ptr(), torch.tensor([500, -1, 3], dtype=torch.int32, device="cuda")
    ws.ensure(ws.nbytes + (1 << 20))
    junk = [torch.full((1 << 18,), 7, device="cuda") for _ in range(16)]  # over what was freed, if it was
    for x in got:
        x.fill_(5)
    g.replay()
    step.check(got)
    assert ws.buf.data_ptr() != used and ws.read_status() == 0
    # what a replay reports is read with the workspace, though it lies in the buffer of the capture
    step.topk[0, :3] = bad
    g.replay()
    assert ws.read_status() == S.svt.DEV_ERR_INDEX_RANGE and ws.read_status() == 0
    del junk


@pytest.mark.parametrize("name", ["decode", "split", "unsplit", "prefill", "backward"])
def test_the_first_call_of_a_thread(S, name):
    """A new thread that has made no CUDA call of its own."""
    step = Step(S, 9, T=8, H=16)
    ws = S.Workspace(nbytes=1 << 24)
    out = torch.empty_like(step.want[0]), torch.empty_like(step.want[1])
    enc, lens = S.build_group_union(step.topk, 8, step.kv.num_slots, ws=ws)
    decode = lambda n: S.sparse_mla_decode(step.q, step.kv, step.topk, SCALE, num_splits=n, out=out[0], lse=out[1], ws=ws)  # noqa: E731
    call = {"decode": lambda: decode(0), "split": lambda: decode(3), "unsplit": lambda: decode(1),
            "prefill": lambda: S.sparse_mla_prefill_grouped(step.q, 8, step.kv, enc, lens, 300, SCALE, out=out[0], lse=out[1],
                                                            ws=ws),
            "backward": lambda: S.sparse_mla_backward(step.q, step.kv, step.topk, SCALE, *step.want[:2], step.dout, ws=ws)}[name]
    errors = []

    def run():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors
    if name != "backward":
        assert float((out[1] - step.want[1]).abs().max()) <= 1e-3


@pytest.mark.parametrize("fill", [0xFF, 0x7F, 0x3C])
def test_workspaces_may_hold_anything_behind_the_header(S, fill):
    """NaN, large numbers, valid indices: no call reads what it has not written."""
    T, H, K = 24, 16, 300
    step = Step(S, 10, T=T, H=H, K=K)
    step.topk[3] = -1
    step.topk[5, 10:] = -1
    G = 8

    def calls(ws):
        got = []
        for n in (0, 1, 2, 3, 5, 8):
            got += S.sparse_mla_decode(step.q, step.kv, step.topk, SCALE, num_splits=n, ws=ws(
                S.svt.lib().svt_sparse_mla_decode_workspace_size(T, H, K, n)))
        got.append(S.resolve_topk_slots(step.topk, num_pages=500, ws=ws(0)))
        enc, lens = S.build_group_union(step.topk, G, 500, ws=ws(0))
        got.append(lens)
        for tile in (False, True):
            got += S.sparse_mla_prefill_grouped(step.q, G, step.kv, enc, lens, K, SCALE, union_tile=tile, ws=ws(
                S.svt.lib().svt_sparse_mla_prefill_grouped_workspace_size(T, H, G)))
        dq, _, w = S.sparse_mla_backward(step.q, step.kv, step.topk, SCALE, got[0], got[1], step.dout, return_weights=True,
                                         ws=ws(S.svt.lib().svt_sparse_mla_backward_workspace_size(T, H, K, 500)))
        return got + [dq, w]

    def dirty(nbytes):
        ws = S.Workspace(nbytes=nbytes)
        ws.buf[256:] = fill
        return ws

    def clean(nbytes):
        ws = S.Workspace(nbytes=nbytes)
        ws.buf.zero_()
        return ws
    for a, b in zip(calls(dirty), calls(clean)):
        assert torch.equal(a, b)
