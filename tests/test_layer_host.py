"""The operators around the attention, as far as a machine without a GPU can check them: rope
frequencies against their formulas, and refused arguments (every refusal happens before anything
reaches a device)."""

import ctypes
import gc
import math
import threading
import weakref

import pytest
import torch

import sparse_mla_attention_top_gb300 as S
from sparse_mla_attention_top_gb300 import build as B
from sparse_mla_attention_top_gb300 import svt

A = ctypes.c_void_p(0x10000)
WS = ctypes.c_void_p(0x100000)


@pytest.fixture(scope="module")
def L():
    B.build()
    return svt.lib()


def err(L):
    return L.svt_last_error_string().decode()


def freqs(dim, **kw):
    return S.rope_frequencies(dim, device="cpu", **kw)


def test_frequencies(L):
    base = torch.tensor([500.0 ** (-2 * i / 8) for i in range(4)], dtype=torch.float64)
    assert torch.allclose(freqs(8, base=500.0), base, rtol=1e-15, atol=0)
    assert torch.allclose(freqs(8, base=500.0, scaling="linear", factor=4.0), base / 4, rtol=1e-15, atol=0)


def test_frequencies_by_parts_keep_fast_pairs_and_divide_slow_ones(L):
    dim, orig, factor, fast, slow = 64, 4096, 40.0, 32.0, 1.0
    plain = freqs(dim)
    f = freqs(dim, scaling="by_parts", factor=factor, original_len=orig, fast=fast, slow=slow)
    turns = plain * orig / (2 * math.pi)
    share = (1 - f / plain) / (1 - 1 / factor)  # 0 = kept, 1 = divided
    assert torch.all(share[turns > 1.5 * fast].abs() < 1e-12)
    assert torch.all((share[turns < slow / 1.5] - 1).abs() < 1e-12)
    inside = share[(share > 1e-9) & (share < 1 - 1e-9)]
    assert len(inside) > 3
    step = inside[1:] - inside[:-1]  # a linear ramp over the pair index
    assert torch.allclose(step, step[:1].expand_as(step), atol=1e-12)


def test_frequencies_by_wavelength(L):
    dim, orig, factor, fast, slow = 128, 8192, 8.0, 4.0, 1.0
    plain = freqs(dim, base=500000.0)
    f = freqs(dim, base=500000.0, scaling="by_wavelength", factor=factor, original_len=orig, fast=fast, slow=slow)
    for a, b in zip(plain.tolist(), f.tolist()):
        wave = 2 * math.pi / a
        if wave < orig / fast:
            want = a
        elif wave > orig / slow:
            want = a / factor
        else:
            keep = (orig / wave - slow) / (fast - slow)
            want = (1 - keep) * a / factor + keep * a
        assert abs(b - want) <= 1e-14 * want


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=7), dict(dim=514), dict(dim=8, base=0.0), dict(dim=8, base=float("inf")),
    dict(dim=8, scaling="linear", factor=0.0), dict(dim=8, scaling="by_parts", factor=2.0),
    dict(dim=8, scaling="by_wavelength", factor=2.0, original_len=10.0, fast=1.0, slow=1.0),
    dict(dim=8, scaling="by_parts", factor=2.0, original_len=10.0, base=1.0)])
def test_frequencies_refusals(L, kw):
    with pytest.raises(S.SvtError):
        freqs(kw.pop("dim"), **kw)
    with pytest.raises(ValueError):
        freqs(8, scaling="other")


def test_rope_refusals(L):
    def call(x=A, out=ctypes.c_void_p(0x80000), dt=0, T=3, H=4, D=64, st=256, sh=64, ot=256, oh=64, pos=A, fr=A, dim=64,
             off=0, layout=0, amp=1.0):
        return L.svt_rope(x, out, dt, T, H, D, st, sh, ot, oh, pos, fr, dim, off, layout, ctypes.c_float(amp), 0, None)
    bad, uns = svt.SVT_ERR_INVALID_ARG, svt.SVT_ERR_UNSUPPORTED
    assert call(dt=2) == uns
    assert call(dim=63) == bad and call(dim=0) == bad
    assert call(dim=514, D=600) == uns
    assert call(layout=2) == bad
    assert call(amp=float("nan")) == bad
    assert call(fr=None) == bad and call(pos=None) == bad
    assert call(x=None) == bad and call(out=None) == bad
    assert call(x=ctypes.c_void_p(0x10001)) == bad
    assert call(off=2) == bad and call(off=-2, D=128) == bad and "columns" in err(L)
    assert call(T=-1) == bad
    assert call(H=20000) == uns
    assert call(T=1 << 20, H=1 << 12) == uns
    assert call(oh=32) == bad and "overlap" in err(L)
    assert call(ot=64) == bad and call(ot=0) == bad
    assert call(out=A, st=512) == bad and "in place" in err(L)
    assert call(T=0, x=None, out=None, pos=None) == svt.SVT_OK


def _kv(dtype=0, pages=4, page_size=64, stride=0, data=0x10000):
    return svt._KV(data, pages, page_size, stride, dtype)


def test_rope_append_refusals(L):
    def call(lat=A, ls=512, kr=A, krs=64, pos=A, slots=A, T=3, kv=None, fr=A, layout=0, amp=1.0, q=None, H=0, qt=0, qh=0,
             qo=None, ot=0, oh=0, ws=WS, n=256):
        return L.svt_rope_append(lat, ls, kr, krs, pos, slots, T, ctypes.byref(kv or _kv()), fr, layout,
                                 ctypes.c_float(amp), q, H, qt, qh, qo, ot, oh, ws, n, None)
    bad, uns = svt.SVT_ERR_INVALID_ARG, svt.SVT_ERR_UNSUPPORTED
    assert call(lat=None) == bad and call(kr=None) == bad and call(pos=None) == bad and call(slots=None) == bad
    assert call(lat=ctypes.c_void_p(0x10008)) == bad and call(ls=516) == bad and "16-byte" in err(L)
    assert call(T=(1 << 30) + 1) == uns
    assert call(T=-1) == bad and call(fr=None) == bad and call(layout=5) == bad and call(amp=float("inf")) == bad
    assert call(kv=_kv(dtype=3)) == uns and call(kv=_kv(pages=0)) == bad and call(kv=_kv(stride=100)) == bad
    assert call(ws=None) == bad and call(n=128) == svt.SVT_ERR_WORKSPACE
    assert call(q=A, H=4, qt=256, qh=64) == bad  # q without q_out
    assert call(q=A, qo=ctypes.c_void_p(0x20000), H=4, qt=256, qh=64, ot=256, oh=32) == bad and "overlap" in err(L)
    assert call(q=A, qo=A, H=4, qt=256, qh=64, ot=512, oh=64) == bad
    assert call(T=0, lat=None, kr=None, pos=None, slots=None) == svt.SVT_OK


def test_backward_refusals(L):
    big = 1 << 40

    def call(q=A, T=2, H=64, kv=None, bt=None, nr=0, mb=0, topk=A, K=128, scale=0.04, out=A, lse=A, dout=A, dq=A, dkv=A,
             ws=WS, n=big):
        return L.svt_sparse_mla_backward(q, T, H, ctypes.byref(kv or _kv()), bt, nr, mb, None, None, topk, K, None,
                                         ctypes.c_float(scale), out, lse, dout, None, dq, dkv, None, ws, n, None)
    bad, uns = svt.SVT_ERR_INVALID_ARG, svt.SVT_ERR_UNSUPPORTED
    odd = ctypes.c_void_p(0x10008)
    assert call(T=-1) == bad and call(K=-1) == bad and call(H=0) == bad and call(H=129) == uns
    assert call(scale=float("nan")) == bad
    assert call(kv=_kv(dtype=1)) == uns and "bf16" in err(L)
    assert call(kv=_kv(pages=1 << 26)) == uns and call(kv=_kv(data=0x10008)) == bad
    assert call(bt=A) == bad
    assert call(T=1 << 26, K=1 << 20) == uns and call(K=(1 << 30) + 1) == uns and call(T=1 << 24) == uns
    for name in ("q", "out", "dout", "dq", "dkv"):
        assert call(**{name: None}) == bad and call(**{name: odd}) == bad, name
    assert call(lse=None) == bad and call(topk=None) == bad
    assert call(ws=ctypes.c_void_p(0x100010)) == bad
    need = L.svt_sparse_mla_backward_workspace_size(2, 64, 128, 256)
    assert need >= 256 + 2 * 128 * 4 + 256 * 576 * 4 and call(n=need - 1) == svt.SVT_ERR_WORKSPACE
    assert L.svt_sparse_mla_backward_workspace_size(-1, 64, 128, 256) == 256


def test_distill_refusals(L):
    def call(x=A, dt=1, T=2, N=100, st=100, topk=A, w=A, K=8, kind=0, scope=0, tau=1.0, loss=A,
             dx=ctypes.c_void_p(0x40000), ds=100):
        return L.svt_distill_topk(x, dt, T, N, st, None, topk, w, K, kind, scope, ctypes.c_float(tau), None, loss, dx, ds,
                                  None)
    bad, uns = svt.SVT_ERR_INVALID_ARG, svt.SVT_ERR_UNSUPPORTED
    assert call(dt=2) == uns and call(N=1 << 30 | 1, st=1 << 31, ds=1 << 31) == uns
    assert call(K=(1 << 30) + 1) == uns and call(T=(1 << 27) + 1) == uns
    assert call(T=-1) == bad and call(N=-1) == bad and call(K=0) == bad
    assert call(kind=2) == bad and call(scope=2) == bad
    for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-7, 1e7):
        assert call(tau=tau) == bad
    assert call(st=99) == bad and call(ds=99) == bad and "stride" in err(L)
    assert call(loss=None, dx=None) == bad and call(x=None) == bad and call(topk=None) == bad and call(w=None) == bad
    assert call(x=ctypes.c_void_p(0x10002)) == bad and call(dx=A) == bad
    assert call(T=0, x=None, topk=None, w=None) == svt.SVT_OK


def test_bindings_refuse_tensors_the_kernels_cannot_take(L):
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    for call in (lambda: S.rope(x.half(), pos, f), lambda: S.rope(x.transpose(0, 2), pos, f),
                 lambda: S.rope(x, pos, f.float()), lambda: S.rope(x, pos, f),  # CPU tensors
                 lambda: S.rope(x, pos, f, out=x.float()),
                 lambda: S.distill_topk(x[0].half(), pos[None], x[0].float()),
                 lambda: S.distill_topk(x[0].float().t(), pos[None], x[0].float())):
        with pytest.raises(TypeError):
            call()


def test_frequencies_on_a_negative_or_fractional_base(L):
    assert torch.allclose(freqs(4, base=0.25), torch.tensor([1.0, 2.0], dtype=torch.float64), rtol=1e-15, atol=0)
    with pytest.raises(S.SvtError):
        freqs(4, base=-2.0)


def test_the_binding_refuses_what_is_no_tensor(L):
    for args in ((None,) * 8, (1, 2, 3, 0, 0, False, 1.0, None)):
        with pytest.raises(TypeError):
            svt._binding().rope(*args)
    with pytest.raises(TypeError):
        svt._binding().rope(torch.zeros(1, 1, 2))
    with pytest.raises(ValueError):
        S.rope(torch.zeros(1, 1, 2), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.float64), layout="x")


def test_default_workspaces_are_one_a_stream_and_one_a_capture(monkeypatch):
    """A workspace is scratch for one stream: calls on two streams, or in two graphs, may overlap."""
    at = [0, 0, 0]
    monkeypatch.setattr(svt, "_fast", type("B", (), {"where": staticmethod(lambda: tuple(at))}))
    made = svt.Workspace
    monkeypatch.setattr(svt, "Workspace", lambda: made("cpu"))
    monkeypatch.setattr(svt, "_default_ws", {})

    def ws(device=0, stream=0, capture=0):
        at[:] = device, stream, capture
        return svt.default_workspace()
    plain = ws()
    assert ws() is plain and ws(stream=7) is ws(stream=7)
    recorded = ws(stream=7, capture=3)
    assert ws(stream=7, capture=3) is recorded
    others = [plain, ws(stream=7), ws(device=1), recorded, ws(stream=8, capture=3), ws(stream=7, capture=4)]
    assert len({id(w) for w in others}) == len(others)


def test_threads_share_a_growing_workspace(monkeypatch):
    """A call sees the address and the size of one buffer, whatever other threads ask for meanwhile."""
    ws = svt.Workspace("cpu")
    seen, stop = [], threading.Event()

    def grow():
        for n in range(1000, 200_000, 1000):
            ws.ensure(n)
        stop.set()
    t = threading.Thread(target=grow)
    t.start()
    while not stop.is_set():
        with ws.lock:
            p, n = ws.buf.data_ptr(), ws.nbytes
            seen.append(p == ws.ptr.value and n == ws.buf.numel())
    t.join()
    assert all(seen) and ws.nbytes >= 199_000


def test_outgrown_workspace_buffers_go_back():
    ws = svt.Workspace("cpu")
    ws.buf[0] = 2  # a pending status bit
    before = [weakref.ref(ws.buf)]
    for n in (1000, 5000, 5001):
        ws.ensure(n)
        assert ws.nbytes == n and ws.buf[0] == 2
        before.append(weakref.ref(ws.buf))
    gc.collect()
    assert [r() is None for r in before] == [True, True, True, False]


def test_page_counts_whose_rows_wrap_round_are_refused(L):
    """2^62 pages of 4 rows are 2^64 rows, no rows in 64 bits; and the border of 2^31 rows."""
    uns = svt.SVT_ERR_UNSUPPORTED
    for pages, size, ok in ((1 << 62, 4, False), (1 << 32, 1 << 30, False), ((1 << 63) - 1, 2, False), (1 << 31, 1, False),
                            (1, (1 << 31) - 1, True), ((1 << 31) - 1, 1, True), (1 << 25, 64, False), ((1 << 25) - 1, 64, True)):
        want = svt.SVT_OK if ok else uns
        kv = ctypes.byref(_kv(pages=pages, page_size=size))
        assert L.svt_sparse_mla_decode(None, 0, 8, kv, None, 0, 0, None, None, None, 0, None, ctypes.c_float(1), None, None, 0,
                                       WS, 256, None) == want
        assert L.svt_rope_append(None, 512, None, 64, None, None, 0, kv, A, 0, ctypes.c_float(1), None, 0, 0, 0, None, 0, 0,
                                 WS, 256, None) == want
        # no output, and a workspace of any size: refused in any case, for its rows or for that
        assert L.svt_sparse_mla_backward(None, 0, 8, kv, None, 0, 0, None, None, None, 0, None, ctypes.c_float(1), None, None,
                                         None, None, None, None, None, WS, 1 << 50, None) == (svt.SVT_ERR_INVALID_ARG if ok else uns)
        assert L.svt_resolve_topk_slots(None, 0, 0, None, None, None, 0, 0, None, size, pages, None, WS, 256, None) in (
            (svt.SVT_OK, svt.SVT_ERR_CUDA) if ok else (uns,))


def test_a_binding_for_another_torch_is_stale(L, monkeypatch):
    """Its file times say nothing of what it was compiled against."""
    assert B.binding_up_to_date() and svt._binding().target == B.binding_target()
    for name in ("2.1", B.binding_target() + "1", B.binding_target()[:-1]):
        monkeypatch.setattr(B, "binding_target", lambda: name)
        assert not B.binding_up_to_date()
        monkeypatch.setattr(svt, "_fast", None)
        with pytest.raises(RuntimeError, match="built for"):
            svt._binding()
