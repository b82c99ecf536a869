"""Shared-prefix attention, beam selection and page operations, as far as a machine without a GPU can check them: arguments
that are refused (before anything reaches a device) and workspace sizes."""

import ctypes

import pytest

from sparse_mla_attention_top_gb300 import build as B
from sparse_mla_attention_top_gb300 import svt

A = ctypes.c_void_p(0x10000)
OUT = ctypes.c_void_p(0x40000)
ODD = ctypes.c_void_p(0x10008)
WS = ctypes.c_void_p(0x100000)
BIG = 1 << 40
OK, BAD, UNS, SMALL = svt.SVT_OK, svt.SVT_ERR_INVALID_ARG, svt.SVT_ERR_UNSUPPORTED, svt.SVT_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    B.build()
    return svt.lib()


def _kv(dtype=0, pages=4, page_size=64, stride=0, data=0x10000):
    return svt._KV(data, pages, page_size, stride, dtype)


def test_shared_prefix_refusals(L):
    def call(q=A, T=3, H=64, kv=None, bt=A, nr=3, mb=4, req=None, lens=A, start=A, pre=A, G=2, scale=0.04, out=OUT, ws=WS,
             n=BIG):
        return L.svt_mla_decode_shared_prefix(q, T, H, ctypes.byref(kv or _kv()), bt, nr, mb, req, lens, start, pre, G,
                                              ctypes.c_float(scale), out, None, ws, n, None)
    assert call(T=-1) == BAD and call(G=-1) == BAD and call(H=0) == BAD and call(H=129) == UNS
    assert call(scale=float("nan")) == BAD and call(scale=float("inf")) == BAD
    assert call(T=1 << 24) == UNS and call(G=(1 << 24) + 1) == UNS
    assert call(kv=_kv(dtype=2)) == UNS and call(kv=_kv(pages=0)) == BAD and call(kv=_kv(data=0x10008)) == BAD
    assert call(kv=_kv(stride=1160)) == BAD and call(kv=_kv(pages=1 << 26)) == UNS
    assert call(bt=None) == BAD and call(nr=0) == BAD and call(mb=0) == BAD and call(mb=1 << 25) == UNS
    assert call(nr=2) == BAD and "req_of_token" in L.svt_last_error_string().decode()
    for name in ("q", "lens", "start", "pre", "out"):
        assert call(**{name: None}) == BAD, name
    assert call(q=ODD) == BAD and call(out=ODD) == BAD
    assert call(ws=None) == BAD and call(ws=ctypes.c_void_p(0x100010)) == BAD
    need = L.svt_mla_decode_shared_prefix_workspace_size(3, 64, 2)
    assert need > 256 and call(n=need - 1) == SMALL
    assert call(T=0, q=None, out=None, bt=None, lens=None) == OK and call(G=0) == OK
    assert L.svt_mla_decode_shared_prefix_workspace_size(-1, 64, 2) == 256
    assert L.svt_mla_decode_shared_prefix_workspace_size(3, 129, 2) == 256


def test_beam_refusals(L):
    def call(x=A, dt=0, b=2, w=4, v=100, sb=400, sw=100, scores=A, done=None, end=0, k=4, o=OUT, p=OUT, t=OUT, ws=WS, n=BIG):
        return L.svt_beam_select(x, dt, b, w, v, sb, sw, scores, done, end, k, o, p, t, ws, n, None)
    assert call(dt=2) == UNS and call(b=-1) == BAD and call(w=0) == BAD and call(v=0) == BAD and call(k=0) == BAD
    assert call(w=129) == UNS and call(k=129) == UNS and call(w=128, k=65) == UNS
    assert call(w=128, v=1 << 24) == UNS and call(b=1 << 23) == UNS
    assert call(done=A, end=100) == BAD and call(done=A, end=-1) == BAD
    for name in ("x", "scores", "o", "p", "t"):
        assert call(**{name: None}) == BAD, name
    assert call(x=ctypes.c_void_p(0x10001)) == BAD and call(dt=1, x=ctypes.c_void_p(0x10002)) == BAD
    assert call(ws=None) == BAD
    need = L.svt_beam_select_workspace_size(2, 4, 100, 4)
    assert need > 256 and call(n=need - 1) == SMALL
    assert call(b=0, x=None) == OK and L.svt_beam_select_workspace_size(2, 4, 100, 500) == 256


def test_fork_refusals(L):
    def call(kv=None, refs=A, ro=A, bt=A, R=3, M=4, lens=A, par=A, N=5, grow=None, every=1, most=1, bo=OUT, Mo=4, lo=OUT,
             slots=OUT, ws=WS, n=BIG):
        return L.svt_fork_pages(ctypes.byref(kv or _kv()), refs, ro, bt, R, M, lens, par, N, grow, every, most, bo, Mo, lo,
                                slots, ws, n, None)
    assert call(kv=_kv(pages=0)) == BAD and call(kv=_kv(dtype=9)) == UNS and call(kv=_kv(stride=8)) == BAD
    assert call(refs=None) == BAD and call(ro=None) == BAD
    assert call(R=-1) == BAD and call(N=-1) == BAD and call(M=-1) == BAD and call(Mo=-1) == BAD
    assert call(R=16385) == UNS and call(N=16385) == UNS and call(M=1 << 25) == UNS and call(Mo=1 << 25) == UNS
    assert call(every=2) == BAD and call(every=-1) == BAD and call(most=-1, every=0) == BAD
    for name in ("bt", "lens", "par", "bo", "lo", "slots"):
        assert call(**{name: None}) == BAD, name
    assert call(bo=A) == BAD and call(bo=ctypes.c_void_p(0x10000 + 3 * 4 * 4 - 4)) == BAD
    assert "overlap" in L.svt_last_error_string().decode()
    assert call(lo=A) == BAD
    assert call(kv=_kv(pages=1, page_size=1 << 21)) == UNS
    need = L.svt_fork_pages_workspace_size(4, 3, 5)
    assert need > 256 and call(n=need - 1) == SMALL and call(ws=None) == BAD
    assert L.svt_fork_pages_workspace_size(0, 3, 5) == 256 and L.svt_fork_pages_workspace_size(4, 16385, 5) == 256


def test_compact_refusals(L):
    def call(kv=None, refs=A, ro=A, bt=A, e=7, bo=A, m=None, ws=WS, n=BIG):
        return L.svt_compact_pages(ctypes.byref(kv or _kv()), refs, ro, bt, e, bo, m, ws, n, None)
    assert call(kv=_kv(pages=-1)) == BAD and call(refs=None) == BAD and call(ro=None) == BAD and call(e=-1) == BAD
    assert call(bt=None) == BAD and call(bo=None) == BAD
    need = L.svt_compact_pages_workspace_size(4)
    assert need > 256 and call(n=need - 1) == SMALL and call(ws=None) == BAD
    assert L.svt_compact_pages_workspace_size(0) == 256 and L.svt_compact_pages_workspace_size(1 << 31) == 256


def test_a_pool_of_any_size_has_a_workspace_of_a_quarter_byte_a_page(L):
    for pages in (1, 33, 1024, 1025, 524288, 524289, 10_000_019, (1 << 31) - 1):
        n = L.svt_compact_pages_workspace_size(pages)
        assert pages / 4 <= n <= pages / 4 + 4096, pages


def test_the_documented_search_step_leaves_missing_candidates_without_a_parent():
    """The example of a search step, run up to its fork: an item with fewer candidates than beams names no other item's row."""
    import pathlib
    from unittest import mock

    import torch

    text = pathlib.Path(__file__).resolve().parents[1].joinpath("README.md").read_text()
    block = next(b for b in text.split("```python")[1:] if "S.beam_select" in b).split("```")[0]
    seen = {}

    class Names(dict):
        def __missing__(self, name):
            return mock.MagicMock()

    B, W = 3, 4
    parents = torch.tensor([[3, 0, 0, 1], [2, 2, -1, -1], [-1, -1, -1, -1]], dtype=torch.int32)
    S = mock.MagicMock()
    S.beam_select.return_value = (torch.zeros(B, W), parents, torch.zeros(B, W, dtype=torch.int32))

    def fork(kv, refs, bt, seq, rows, **kw):
        seen["rows"] = rows
        return (mock.MagicMock(),) * 4

    S.fork_pages.side_effect = fork
    S.mla_decode_shared_prefix.return_value = (None, None)
    S.compact_pages.return_value = (None, None, None)
    exec(compile(block, "README.md", "exec"), {}, Names(S=S, torch=torch, B=B, W=W))
    assert seen["rows"].dtype == torch.int32
    assert seen["rows"].tolist() == [3, 0, 0, 1, 6, 6, -1, -1, -1, -1, -1, -1]


def test_shared_prefix_lists_beyond_32_bits_are_refused(L):
    # a row tile of 128 (query, head) rows counts its list in pieces of 16 positions: H = 1 has 128 queries in one
    def call(T, H, mb, page=64):
        kv = _kv(page_size=page)
        return L.svt_mla_decode_shared_prefix(A, T, H, ctypes.byref(kv), A, T, mb, None, A, A, A, 2, ctypes.c_float(0.04),
                                              OUT, None, WS, 300, None)
    most = (1 << 30) // 64
    assert call(128, 1, most) == UNS and "2^35" in L.svt_last_error_string().decode()
    assert call(31, 1, most) == UNS and call(30, 1, most) == SMALL
    assert call(4096, 4, most) == UNS and call(4096, 5, most) == SMALL and call(4096, 128, most) == SMALL
    assert call(128, 1, most // 8) == SMALL and call(128, 1, (1 << 30) // 7, page=7) == UNS
