"""Thin Python binding of libsvt.so (ctypes, and csrc/binding.cpp for the short calls).

Argument marshalling only: every function takes torch tensors on the current CUDA device,
checks dtypes and shapes, passes raw pointers and the current stream to the C ABI, and
raises SvtError on a non-OK status. All computation happens in the library's kernels; there
is no fallback. The names follow the C entry points in include/svt.h.
"""

from __future__ import annotations

import ctypes
import threading
from dataclasses import dataclass
from pathlib import Path
from typing import Optional

import torch

_LIB_PATH = Path(__file__).resolve().parent / "libsvt.so"
_lib = None

SVT_OK, SVT_ERR_INVALID_ARG, SVT_ERR_UNSUPPORTED, SVT_ERR_WORKSPACE, SVT_ERR_CUDA = range(5)
STATUS_NAMES = {0: "SVT_OK", 1: "SVT_ERR_INVALID_ARG", 2: "SVT_ERR_UNSUPPORTED", 3: "SVT_ERR_WORKSPACE",
                4: "SVT_ERR_CUDA"}
DEV_ERR_INDEX_RANGE = 0x1
DEV_ERR_TIMEOUT = 0x2
DEV_ERR_FP8_RANGE = 0x4
DEV_ERR_NO_PAGES = 0x8
KV_BF16 = 0
KV_FP8_E4M3 = 1
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "by_parts": 2, "by_wavelength": 3}
TEACHER_KINDS = {"weights": 0, "logits": 1}
DISTILL_SCOPES = {"candidates": 0, "listed": 1}
ROW_BYTES = {KV_BF16: 1152, KV_FP8_E4M3: 656}

EXPORTED = [
    "svt_last_error_string", "svt_workspace_init", "svt_read_status", "svt_resolve_workspace_size",
    "svt_resolve_topk_slots", "svt_sparse_mla_decode_workspace_size", "svt_sparse_mla_decode",
    "svt_build_group_union_workspace_size", "svt_build_group_union",
    "svt_sparse_mla_prefill_grouped_workspace_size", "svt_sparse_mla_prefill_grouped",
    "svt_sparse_mla_prefill_grouped_union_tile", "svt_merge_splits",
    "svt_topk_select",
    "svt_rope_frequencies", "svt_rope", "svt_rope_append", "svt_sparse_mla_backward_workspace_size",
    "svt_sparse_mla_backward", "svt_distill_topk",
    "svt_mla_decode_shared_prefix_workspace_size", "svt_mla_decode_shared_prefix", "svt_beam_select_workspace_size",
    "svt_beam_select", "svt_fork_pages_workspace_size", "svt_fork_pages", "svt_compact_pages_workspace_size",
    "svt_compact_pages",
    "svt_sparse_mla_decode_noalloc", "svt_debug_pipeline_fault", "svt_gather_probe", "svt_tensor_probe",
]


class SvtError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class _KV(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("row_stride_bytes", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("fast", ctypes.c_double), ("slow", ctypes.c_double)]


def library_path() -> Path:
    return _LIB_PATH


def use_library(path) -> None:
    """Loads the library from `path` instead of libsvt.so (the phase-trace build, for
    profiling); must come before the first call into the library."""
    global _LIB_PATH
    if _lib is not None:
        raise RuntimeError("the library is already loaded")
    _LIB_PATH = Path(path)


def lib():
    """The loaded library; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not _LIB_PATH.exists():
            raise RuntimeError(f"{_LIB_PATH} is missing: build it first (sparse_mla_attention_top_gb300.build)")
        L = ctypes.CDLL(str(_LIB_PATH))
        P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        L.svt_last_error_string.restype = ctypes.c_char_p
        L.svt_workspace_init.argtypes = [P, sz, P]
        L.svt_read_status.argtypes = [P, P, P]
        L.svt_resolve_workspace_size.restype = sz
        L.svt_resolve_topk_slots.argtypes = [P, i32, i32, P, P, P, i32, i32, P, i32, i64, P, P, sz, P]
        L.svt_sparse_mla_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        L.svt_sparse_mla_decode_workspace_size.restype = sz
        L.svt_sparse_mla_decode.argtypes = [P, i32, i32, ctypes.POINTER(_KV), P, i32, i32, P, P, P, i32, P, f32, P, P,
                                            i32, P, sz, P]
        L.svt_build_group_union_workspace_size.argtypes = [i32, i32, i32]
        L.svt_build_group_union_workspace_size.restype = sz
        L.svt_build_group_union.argtypes = [P, P, i32, i32, i32, i64, P, P, P, sz, P]
        L.svt_sparse_mla_prefill_grouped_workspace_size.argtypes = [i32, i32, i32]
        L.svt_sparse_mla_prefill_grouped_workspace_size.restype = sz
        L.svt_sparse_mla_prefill_grouped.argtypes = [P, i32, i32, i32, ctypes.POINTER(_KV), P, P, i32, f32, P, P, P,
                                                     sz, P]
        L.svt_sparse_mla_prefill_grouped_union_tile.argtypes = L.svt_sparse_mla_prefill_grouped.argtypes
        L.svt_merge_splits.argtypes = [P, P, i32, i32, i32, P, P, P]
        L.svt_topk_select.argtypes = [P, i32, i32, i64, P, i32, P, P]
        L.svt_rope_frequencies.argtypes = [i32, ctypes.c_double, ctypes.POINTER(_RopeScaling), P]
        L.svt_rope.argtypes = [P, P, i32, i32, i32, i32, i64, i64, i64, i64, P, P, i32, i32, i32, f32, i32, P]
        L.svt_rope_append.argtypes = [P, i64, P, i64, P, P, i32, ctypes.POINTER(_KV), P, i32, f32, P, i32, i64, i64, P,
                                      i64, i64, P, sz, P]
        L.svt_sparse_mla_backward_workspace_size.argtypes = [i32, i32, i32, i64]
        L.svt_sparse_mla_backward_workspace_size.restype = sz
        L.svt_sparse_mla_backward.argtypes = [P, i32, i32, ctypes.POINTER(_KV), P, i32, i32, P, P, P, i32, P, f32, P, P,
                                              P, P, P, P, P, P, sz, P]
        L.svt_distill_topk.argtypes = [P, i32, i32, i32, i64, P, P, P, i32, i32, i32, f32, P, P, P, i64, P]
        L.svt_mla_decode_shared_prefix_workspace_size.argtypes = [i32, i32, i32]
        L.svt_mla_decode_shared_prefix_workspace_size.restype = sz
        L.svt_mla_decode_shared_prefix.argtypes = [P, i32, i32, ctypes.POINTER(_KV), P, i32, i32, P, P, P, P, i32, f32, P, P,
                                                   P, sz, P]
        L.svt_beam_select_workspace_size.argtypes = [i32, i32, i32, i32]
        L.svt_beam_select_workspace_size.restype = sz
        L.svt_beam_select.argtypes = [P, i32, i32, i32, i32, i64, i64, P, P, i32, i32, P, P, P, P, sz, P]
        L.svt_fork_pages_workspace_size.argtypes = [i64, i32, i32]
        L.svt_fork_pages_workspace_size.restype = sz
        L.svt_fork_pages.argtypes = [ctypes.POINTER(_KV), P, P, P, i32, i32, P, P, i32, P, i32, i32, P, i32, P, P, P, sz, P]
        L.svt_compact_pages_workspace_size.argtypes = [i64]
        L.svt_compact_pages_workspace_size.restype = sz
        L.svt_compact_pages.argtypes = [ctypes.POINTER(_KV), P, P, P, i64, P, P, P, sz, P]
        L.svt_sparse_mla_decode_noalloc.argtypes = [P, i32, i32, ctypes.POINTER(_KV), P, i32, i32, P, P, P, i32, P, f32,
                                                    P, P, i32, P, P]
        L.svt_debug_pipeline_fault.argtypes = [i32, i64]
        L.svt_gather_probe.argtypes = [ctypes.POINTER(_KV), P, i64, i32, P, P, sz, P]
        L.svt_tensor_probe.argtypes = [P, P, P, i32, i32, P, P, P, P, sz, P]
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != SVT_OK:
        msg = lib().svt_last_error_string()
        raise SvtError(status, where, msg.decode() if msg else "")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _i32(t: Optional[torch.Tensor], name: str) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    return t


def _table(bt: Optional[torch.Tensor], T: int):
    """The address of a block table. An empty one has none, which would read positions as slots: for queries
    to resolve it gets an address that is never read, and the library refuses its sizes."""
    return ctypes.c_void_p(256) if bt is not None and bt.numel() == 0 and T > 0 else _ptr(bt)


@dataclass
class KVCache:
    """A paged latent cache in device memory: `data` is uint8 [num_pages * page_size, row_bytes]
    (or any contiguous tensor with those bytes); dtype KV_BF16 or KV_FP8_E4M3."""
    data: torch.Tensor
    num_pages: int
    page_size: int
    dtype: int = KV_BF16
    row_stride_bytes: int = 0

    def _c(self) -> _KV:
        if not self.data.is_cuda or not self.data.is_contiguous():
            raise TypeError("kv data must be a contiguous CUDA tensor")
        return _KV(self.data.data_ptr(), int(self.num_pages), int(self.page_size), int(self.row_stride_bytes),
                   int(self.dtype))

    @property
    def num_slots(self) -> int:
        return int(self.num_pages) * int(self.page_size)


class Workspace:
    """Caller-owned scratch for one stream: a 256-byte status header plus per-call space.
    Grows on demand, to the size asked for (allocation happens here, in torch, never inside the library).
    An outgrown buffer goes back to torch, unless a call that used it was captured: the graph goes on using
    it, so it is kept, and its status is read with the workspace's. A call holds `lock` while it sizes the
    workspace and enqueues its kernels, so that threads can share one on their common stream."""

    def __init__(self, device=None, nbytes: int = 256):
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.buf = self._new(max(256, nbytes))
        self.buf[:256].zero_()
        self._captured = False  # whether a captured call uses buf
        self._kept = []
        self.lock = threading.RLock()

    def _new(self, nbytes: int) -> torch.Tensor:
        """Only the status header needs a value."""
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def ensure(self, nbytes: int) -> "Workspace":
        """At least nbytes."""
        with self.lock:
            self._size_to(nbytes, self.buf.is_cuda and torch.cuda.is_current_stream_capturing())
        return self

    def _size_to(self, nbytes: int, capturing: bool) -> None:
        """What a call makes of its workspace, under the lock, before it takes ptr and nbytes."""
        if nbytes > self.buf.numel():
            old = self.buf
            self.buf = self._new(nbytes)
            if self._captured or capturing:
                self.buf[:256].zero_()
                self._kept.append(old)
            else:
                self.buf[:256].copy_(old[:256])  # keep pending status bits
                if old.is_cuda:
                    old.record_stream(torch.cuda.current_stream())  # earlier calls may still run
            self._captured = False
        if capturing:
            self._captured = True

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    @property
    def nbytes(self) -> int:
        return self.buf.numel()

    def read_status(self, stream=None) -> int:
        bits = 0
        for buf in (self.buf, *self._kept):
            out = ctypes.c_int32(0)
            _check(lib().svt_read_status(_ptr(buf), _stream(stream), ctypes.byref(out)), "svt_read_status")
            bits |= int(out.value)
        return bits


_default_ws = {}  # (device, stream, capture or 0) -> Workspace
_default_lock = threading.Lock()


def _workspace(ws: Optional[Workspace]):
    """The workspace of a call (the given one, or the default), whether the call is captured, and the
    address of its stream."""
    at = (_fast or _binding()).where()
    if ws is None:
        ws = _default_ws.get(at)
        if ws is None:
            with _default_lock:
                ws = _default_ws.get(at)
                if ws is None:
                    if at[2]:  # a stream's last capture is over, and its graph's memory the graph's own
                        for key in [k for k in _default_ws if k[:2] == at[:2] and k[2]]:
                            del _default_ws[key]
                    ws = _default_ws[at] = Workspace()
    return ws, at[2] != 0, at[1]


def default_workspace() -> Workspace:
    """The workspace of calls that are given none: one for each stream of each device, as calls on two
    streams may overlap. While the stream is being captured it is one of that capture's own, as two graphs
    may be replayed at once: it lies in the graph's memory, and each replay begins by clearing its status.
    Give captured calls a workspace where their status is to be read."""
    return _workspace(None)[0]


def resolve_topk_slots(topk_pos, *, block_table=None, seq_lens=None, req_of_token=None, topk_len=None,
                       page_size: int = 1, num_pages: int, out=None, ws: Optional[Workspace] = None):
    """svt_resolve_topk_slots: [T, K] positions -> [T, K] int32 slots (-1 for dead entries)."""
    topk_pos = _i32(topk_pos, "topk_pos")
    T, K = topk_pos.shape
    bt = _i32(block_table, "block_table")
    out = torch.empty((T, K), dtype=torch.int32, device=topk_pos.device) if out is None else out
    ws, capturing, stream = _workspace(ws)
    with ws.lock:
        ws._size_to(lib().svt_resolve_workspace_size(), capturing)
        _check(lib().svt_resolve_topk_slots(_ptr(topk_pos), T, K, _ptr(_i32(topk_len, "topk_len")),
                                            _ptr(_i32(req_of_token, "req_of_token")), _table(bt, T),
                                            0 if bt is None else bt.shape[0], 0 if bt is None else bt.shape[1],
                                            _ptr(_i32(seq_lens, "seq_lens")), int(page_size), int(num_pages), _ptr(out),
                                            ws.ptr, ws.nbytes, stream), "svt_resolve_topk_slots")
    return out


def sparse_mla_decode(q, kv: KVCache, topk, softmax_scale: float, *, block_table=None, seq_lens=None,
                      req_of_token=None, topk_len=None, num_splits: int = 0, out=None, lse=None,
                      return_lse: bool = True, ws: Optional[Workspace] = None):
    """svt_sparse_mla_decode. q [T, H, 576] bf16; topk [T, K] int32 positions (slots when
    block_table is None). Returns (out [T, H, 512] bf16, lse [T, H] fp32 or None)."""
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[2] != 576 or not q.is_contiguous():
        raise TypeError("q must be a contiguous bf16 [T, H, 576] tensor")
    T, H, _ = q.shape
    topk = _i32(topk, "topk")
    K = topk.shape[1]
    bt = _i32(block_table, "block_table")
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    ws, capturing, stream = _workspace(ws)
    kvc = kv._c()
    with ws.lock:
        ws._size_to(lib().svt_sparse_mla_decode_workspace_size(T, H, K, num_splits), capturing)
        _check(lib().svt_sparse_mla_decode(_ptr(q), T, H, ctypes.byref(kvc), _table(bt, T), 0 if bt is None else bt.shape[0],
                                           0 if bt is None else bt.shape[1], _ptr(_i32(req_of_token, "req_of_token")),
                                           _ptr(_i32(seq_lens, "seq_lens")), _ptr(topk), K,
                                           _ptr(_i32(topk_len, "topk_len")), float(softmax_scale), _ptr(out), _ptr(lse),
                                           int(num_splits), ws.ptr, ws.nbytes, stream), "svt_sparse_mla_decode")
    return out, lse


def build_group_union(slots, G: int, num_slots: int, *, topk_len=None, enc=None, lens=None,
                      ws: Optional[Workspace] = None):
    """svt_build_group_union: slots [T, K] int32 -> (enc [ceil(T/G), G*K] int32, lens [ceil(T/G)] int32)."""
    slots = _i32(slots, "slots")
    T, K = slots.shape
    groups = (T + G - 1) // G
    if enc is None:
        enc = torch.empty((groups, G * K), dtype=torch.int32, device=slots.device)
    if lens is None:
        lens = torch.empty((groups,), dtype=torch.int32, device=slots.device)
    ws, capturing, stream = _workspace(ws)
    with ws.lock:
        ws._size_to(lib().svt_build_group_union_workspace_size(T, K, G), capturing)
        _check(lib().svt_build_group_union(_ptr(slots), _ptr(_i32(topk_len, "topk_len")), T, K, int(G), int(num_slots),
                                           _ptr(enc), _ptr(lens), ws.ptr, ws.nbytes, stream), "svt_build_group_union")
    return enc, lens


def sparse_mla_prefill_grouped(q, G: int, kv: KVCache, enc, lens, K: int, softmax_scale: float, *, out=None,
                               lse=None, return_lse: bool = True, ws: Optional[Workspace] = None,
                               union_tile: bool = False):
    """svt_sparse_mla_prefill_grouped (or, with union_tile, svt_sparse_mla_prefill_grouped_union_tile).
    q [T, H, 576] bf16 token-major, H * G = 128."""
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[2] != 576 or not q.is_contiguous():
        raise TypeError("q must be a contiguous bf16 [T, H, 576] tensor")
    T, H, _ = q.shape
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    ws, capturing, stream = _workspace(ws)
    kvc = kv._c()
    name = "svt_sparse_mla_prefill_grouped_union_tile" if union_tile else "svt_sparse_mla_prefill_grouped"
    with ws.lock:
        ws._size_to(lib().svt_sparse_mla_prefill_grouped_workspace_size(T, H, G), capturing)
        _check(getattr(lib(), name)(_ptr(q), T, H, int(G), ctypes.byref(kvc), _ptr(_i32(enc, "enc")),
                                    _ptr(_i32(lens, "lens")), int(K), float(softmax_scale), _ptr(out), _ptr(lse), ws.ptr,
                                    ws.nbytes, stream), name)
    return out, lse


def merge_splits(o_part, lse_part, *, out=None, lse=None, return_lse: bool = True):
    """svt_merge_splits: o_part [S, T, H, 512] fp32, lse_part [S, T, H] fp32 -> (out bf16, lse fp32)."""
    if o_part.dtype != torch.float32 or lse_part.dtype != torch.float32:
        raise TypeError("partials must be fp32")
    S, T, H, _ = o_part.shape
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=o_part.device)
    if lse is None and return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=o_part.device)
    if not (o_part.is_contiguous() and lse_part.is_contiguous()):
        raise TypeError("partials must be contiguous")
    _check(lib().svt_merge_splits(_ptr(o_part), _ptr(lse_part), S, T, H, _ptr(out),
                                  _ptr(lse), _stream()), "svt_merge_splits")
    return out, lse


def topk_select(scores, K: int, *, lens=None, out=None):
    """svt_topk_select: scores [T, N] fp32 (rows may be strided) -> [T, K] int32 positions,
    ascending, -1 padded."""
    if scores.dtype != torch.float32 or scores.dim() != 2 or scores.stride(1) != 1:
        raise TypeError("scores must be a [T, N] fp32 tensor with unit column stride")
    T, N = scores.shape
    if lens is not None:
        lens = _i32(lens, "lens")
    if out is None:
        out = torch.empty((T, K), dtype=torch.int32, device=scores.device)
    stride = scores.stride(0) if T > 1 else N  # a single row's stride is meaningless (can be 0)
    _check(lib().svt_topk_select(_ptr(scores), T, N, stride, _ptr(lens), int(K), _ptr(out), _stream()),
           "svt_topk_select")
    return out


_fast = None


def _binding():
    """The compiled binding (csrc/binding.cpp) of the short calls below, bound to the loaded library. It
    makes the checks of tensors: types, shapes, and that all are on the current CUDA device."""
    global _fast
    if _fast is None:
        L = lib()
        from . import build
        try:
            from . import _binding as fast
        except ImportError as e:
            raise RuntimeError("_binding.so is missing or stale: build it first "
                               "(sparse_mla_attention_top_gb300.build)") from e
        here = build.binding_target()
        if getattr(fast, "target", None) != here:
            raise RuntimeError(f"_binding.so was built for {getattr(fast, 'target', 'another torch')}, this is {here}: "
                               "build it again (sparse_mla_attention_top_gb300.build)")
        fast.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.svt_rope, L.svt_rope_append, L.svt_sparse_mla_backward_workspace_size, L.svt_sparse_mla_backward,
            L.svt_distill_topk, L.svt_mla_decode_shared_prefix_workspace_size, L.svt_mla_decode_shared_prefix,
            L.svt_beam_select_workspace_size, L.svt_beam_select, L.svt_fork_pages_workspace_size, L.svt_fork_pages,
            L.svt_compact_pages_workspace_size, L.svt_compact_pages)))
        _fast = fast
    return _fast


def _choice(value: str, choices: dict, name: str) -> int:
    code = choices.get(value)
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(choices)}, got {value!r}")
    return code


def rope_frequencies(dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original_len: float = 0.0, fast: float = 32.0, slow: float = 1.0, device=None):
    """svt_rope_frequencies: the [dim / 2] fp64 frequencies (radians per position) that rope and
    rope_append take, on the device. scaling: "none", "linear", "by_parts" or "by_wavelength"."""
    host = torch.empty(max(0, int(dim) // 2), dtype=torch.float64)
    s = _RopeScaling(_choice(scaling, ROPE_SCALINGS, "scaling"), float(factor), float(original_len), float(fast),
                     float(slow))
    _check(lib().svt_rope_frequencies(int(dim), float(base), ctypes.byref(s), _ptr(host)), "svt_rope_frequencies")
    return host.to(torch.device("cuda", torch.cuda.current_device()) if device is None else device)


def rope(x, positions, freqs, *, offset: int = 0, layout: str = "interleaved", inverse: bool = False,
         amplitude: float = 1.0, out=None):
    """svt_rope: rotates columns offset .. offset + 2 len(freqs) - 1 of x ([T, H, D] or [T, D], bf16
    or fp32, rows may be strided) by its tokens' positions; the other columns are copied. out=x
    rotates in place. inverse=True turns back: it maps the gradient of the result to x's."""
    r = (_fast or _binding()).rope(x, positions, freqs, offset, _choice(layout, ROPE_LAYOUTS, "layout"), inverse, amplitude,
                                   out)
    if type(r) is int:
        _check(r, "svt_rope")
    return r


def rope_append(latent, k_rope, positions, slots, kv: KVCache, freqs, *, layout: str = "interleaved",
                amplitude: float = 1.0, q_rope=None, q_out=None, ws: Optional[Workspace] = None):
    """svt_rope_append: writes latent [T, 512] and the rotated k_rope [T, 64] (bf16, rows may be
    strided) to cache rows slots [T] (negative: skipped); with q_rope [T, H, 64] it rotates the
    queries' rope columns into q_out (a new tensor when None; q[..., 512:] of a [T, H, 576] q fits)
    in the same launch. Returns q_out."""
    ws, capturing, _ = _workspace(ws)
    with ws.lock:
        ws._captured |= capturing
        r = (_fast or _binding()).rope_append(latent, k_rope, positions, slots, kv.data, kv.num_pages, kv.page_size,
                                              kv.row_stride_bytes, kv.dtype, freqs, _choice(layout, ROPE_LAYOUTS, "layout"),
                                              amplitude, q_rope, q_out, ws.buf)
    if type(r) is int:
        _check(r, "svt_rope_append")
    return r


def sparse_mla_backward(q, kv: KVCache, topk, softmax_scale: float, out, lse, dout, *, dlse=None, block_table=None,
                        seq_lens=None, req_of_token=None, topk_len=None, dq=None, dkv=None,
                        return_weights: bool = False, ws: Optional[Workspace] = None):
    """svt_sparse_mla_backward: the gradients of sparse_mla_decode (or of a grouped prefill, with each
    query's own list). out and lse are the forward's; dout (and dlse) their gradients. Returns
    (dq [T, H, 576] bf16, dkv [num_slots, 576] bf16, weights [T, K] fp32 or None)."""
    ws, capturing, _ = _workspace(ws)
    with ws.lock:
        ws._captured |= capturing
        for _ in range(2):
            r = (_fast or _binding()).sparse_mla_backward(
                q, kv.data, kv.num_pages, kv.page_size, kv.row_stride_bytes, kv.dtype, topk, softmax_scale, out, lse, dout,
                dlse, block_table, seq_lens, req_of_token, topk_len, dq, dkv, return_weights, ws.buf)
            if type(r) is not int:
                return r
            if r >= 0:
                break
            ws._size_to(-r, capturing)
    _check(r, "svt_sparse_mla_backward")


def distill_topk(scores, topk, teacher, *, lens=None, temperature: float = 1.0, teacher_kind: str = "weights",
                 over: str = "candidates", row_weight=None, need_grad: bool = True, dscores=None):
    """svt_distill_topk: per query, KL(teacher's top entries || softmax of scores) and the gradient of
    row_weight . loss. scores [T, N] fp32 or bf16 (rows may be strided), topk [T, K] positions (-1 =
    none), teacher [T, K] fp32 weights or logits. Returns (loss [T], dscores [T, N] or None)."""
    r = (_fast or _binding()).distill_topk(scores, topk, teacher, lens, temperature,
                                           _choice(teacher_kind, TEACHER_KINDS, "teacher_kind"),
                                           _choice(over, DISTILL_SCOPES, "over"), row_weight, need_grad, dscores)
    if type(r) is int:
        _check(r, "svt_distill_topk")
    return r


def _with_workspace(ws: Optional[Workspace], where: str, call):
    """call(workspace tensor) until it does not answer with minus the bytes that it needs; its outputs."""
    ws, capturing, _ = _workspace(ws)
    with ws.lock:
        ws._captured |= capturing
        for _ in range(2):
            r = call(ws.buf)
            if type(r) is not int:
                return r
            if r >= 0:
                break
            ws._size_to(-r, capturing)
    _check(r, where)


def mla_decode_shared_prefix(q, kv: KVCache, block_table, lens, group_start, prefix_lens, softmax_scale: float, *,
                             req_of_token=None, out=None, lse=None, return_lse: bool = True,
                             ws: Optional[Workspace] = None):
    """svt_mla_decode_shared_prefix: dense decode attention; query t attends to positions 0 .. lens[t] - 1 of its request, and
    the queries of a group (group_start [G + 1], consecutive) share the rows of its first prefix_lens [G] positions, which
    are read once for all. q [T, H, 576] bf16. Returns (out [T, H, 512] bf16, lse [T, H] fp32 or None); rows of queries
    in no group are not written."""
    return _with_workspace(ws, "svt_mla_decode_shared_prefix", lambda buf: (_fast or _binding()).mla_decode_shared_prefix(
        q, kv.data, kv.num_pages, kv.page_size, kv.row_stride_bytes, kv.dtype, block_table, req_of_token, lens,
        group_start, prefix_lens, softmax_scale, out, lse, return_lse, buf))


def beam_select(logits, scores, K: int, *, finished=None, end_token: int = 0, ws: Optional[Workspace] = None):
    """svt_beam_select: the K best continuations of each batch item's beams. logits [B, W, V] fp32 or bf16 (unit column
    stride), scores [B, W] fp32, finished [B, W] bool or uint8. Returns (scores [B, K] fp32, parents [B, K] int32, tokens
    [B, K] int32) in descending order, (-inf, -1, -1) where there are fewer: a parent of -1 stays -1 where parents become
    rows of a table for fork_pages (b * W - 1 is another item's)."""
    return _with_workspace(ws, "svt_beam_select", lambda buf: (_fast or _binding()).beam_select(
        logits, scores, K, finished, end_token, buf))


def fork_pages(kv: KVCache, refs, block_table, seq_lens, parents, *, grow=0, max_grow: Optional[int] = None,
               max_blocks: Optional[int] = None, refs_out=None, ws: Optional[Workspace] = None):
    """svt_fork_pages: new rows that continue rows `parents` [N] (-1: none) of block_table [R, M], each grown by `grow` tokens
    (an int, or int32 [N] with max_grow); the old rows are given up. refs [num_pages] int32 counts the entries that hold
    each page and is updated in place, or into refs_out. Returns (block_table [N, max_blocks or M], seq_lens [N], slots [N,
    max_grow], refs)."""
    if isinstance(grow, torch.Tensor):
        if max_grow is None:
            raise ValueError("a tensor of growths needs max_grow")
        each, every = grow, 0
    else:
        each, every = None, int(grow)
        max_grow = every if max_grow is None else max_grow
    return _with_workspace(ws, "svt_fork_pages", lambda buf: (_fast or _binding()).fork_pages(
        kv.data, kv.num_pages, kv.page_size, kv.row_stride_bytes, kv.dtype, refs, refs_out, block_table, seq_lens,
        parents, each, every, max_grow, -1 if max_blocks is None else max_blocks, buf))


def compact_pages(kv: KVCache, refs, block_table, *, refs_out=None, table_out=None, ws: Optional[Workspace] = None):
    """svt_compact_pages: moves the live pages to the lowest numbers and rewrites the page numbers of block_table (int32, any
    shape), in place or into table_out, and the counts, in place or into refs_out. Returns (block_table, refs, mapping):
    mapping [num_pages] int32 is each page's new number, -1 for a free one."""
    return _with_workspace(ws, "svt_compact_pages", lambda buf: (_fast or _binding()).compact_pages(
        kv.data, kv.num_pages, kv.page_size, kv.row_stride_bytes, kv.dtype, refs, refs_out, block_table, table_out, buf))


def debug_pipeline_fault(fault: int = 0, wait_limit_ns: int = 0) -> None:
    """Failure-detection hook for tests (svt_debug_pipeline_fault): plant a withheld arrival
    in the attention kernels launched afterwards and/or shorten their wait limit; (0, 0)
    restores ordinary behaviour."""
    _check(lib().svt_debug_pipeline_fault(int(fault), int(wait_limit_ns)), "svt_debug_pipeline_fault")


def gather_probe(kv: KVCache, slots, mode: int = 0, *, out=None, ws: Optional[Workspace] = None):
    """Reads the cache rows of `slots` ([n] int32) the way the decode's gather does, with no
    arithmetic (svt_gather_probe); returns each row's XOR of 32-bit words as int32 [n]."""
    slots = _i32(slots, "slots")
    n = slots.numel()
    if out is None:
        out = torch.empty((n,), dtype=torch.int32, device=slots.device)
    ws, capturing, stream = _workspace(ws)
    kvc = kv._c()
    with ws.lock:
        ws._size_to(256, capturing)
        _check(lib().svt_gather_probe(ctypes.byref(kvc), _ptr(slots), n, int(mode), _ptr(out), ws.ptr, ws.nbytes,
                                      stream), "svt_gather_probe")
    return out


def tensor_probe(k_rows, q, pt, reps: int = 1, grid: int = 1, *, ws: Optional[Workspace] = None):
    """Issues one half-tile's S^T and PV MMA group of the attention kernels `reps` times on
    `grid` CTAs (svt_tensor_probe). k_rows, q: [64, 576] bf16; pt: [64, 64] bf16 (P^T).
    Returns (S^T [64, 64] fp32, O^T [512, 64] fp32 = reps * V^T P^T, cycles [grid] int64)."""
    for name, t, shape in (("k_rows", k_rows, (64, 576)), ("q", q, (64, 576)), ("pt", pt, (64, 64))):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous() or not t.is_cuda:
            raise SvtError(f"{name} must be a contiguous CUDA bf16 tensor of shape {shape}")
    dev = k_rows.device
    s_out = torch.empty((64, 64), dtype=torch.float32, device=dev)
    o_out = torch.empty((512, 64), dtype=torch.float32, device=dev)
    cycles = torch.empty((int(grid),), dtype=torch.int64, device=dev)
    ws, capturing, stream = _workspace(ws)
    with ws.lock:
        ws._size_to(256, capturing)
        _check(lib().svt_tensor_probe(_ptr(k_rows), _ptr(q), _ptr(pt), int(reps), int(grid), _ptr(s_out), _ptr(o_out),
                                      _ptr(cycles), ws.ptr, ws.nbytes, stream), "svt_tensor_probe")
    return s_out, o_out, cycles
