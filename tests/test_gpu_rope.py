"""Rotary positions and cache writes on the GPU against an fp64 statement."""

import math
from fractions import Fraction

import pytest
import torch

from sparse_mla_attention_top_gb300 import workloads as W
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


def normal(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def positions(seed, T, far=1 << 17):
    p = torch.randint(0, far, (T,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    p[:1] = 0
    if T > 3:
        p[1], p[2], p[3] = 2 ** 31 - 1, -5, 1_000_003
    return p


def check(S, x, pos, f, layout, inverse=False, amplitude=1.0, offset=0, out=None, x_dev=None):
    dim = 2 * f.numel()
    xd = x.cuda() if x_dev is None else x_dev
    got = S.rope(xd, pos.cuda(), f.cuda(), offset=offset, layout=layout, inverse=inverse, amplitude=amplitude, out=out)
    x3 = x if x.dim() == 3 else x[:, None]
    g3 = got if x.dim() == 3 else got[:, None]
    lo, hi = offset, offset + dim
    ref = R.rotate(x3[..., lo:hi], pos, f, layout, inverse, amplitude)
    R.within(g3[..., lo:hi], ref, R.rotate_bound(x3[..., lo:hi], ref, layout, x.dtype, amplitude, pos, f), "rotated")
    assert torch.equal(g3[..., :lo].cpu(), x3[..., :lo]) and torch.equal(g3[..., hi:].cpu(), x3[..., hi:])
    return got


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,dim,offset", [
    (1, 1, 64, 64, 0), (1, 128, 64, 64, 0), (7, 5, 192, 64, 128), (64, 16, 96, 32, 32), (3, 2, 10, 2, 4),
    (5, 3, 71, 6, 65), (129, 1, 576, 64, 512), (1000, 3, 100, 98, 1), (2, 300, 512, 512, 0), (4100, 1, 40, 24, 8)])
def test_rope(S, layout, dtype, T, H, D, dim, offset):
    x = normal(T + H, T, H, D, dtype=dtype)
    f = S.rope_frequencies(dim, device="cpu")
    check(S, x, positions(T, T), f, layout, offset=offset)
    check(S, x, positions(T, T), f, layout, inverse=True, amplitude=1.37, offset=offset)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_scaled_frequencies_at_far_positions(S, layout):
    f = S.rope_frequencies(64, scaling="by_parts", factor=40.0, original_len=4096, device="cpu")
    x = normal(1, 50, 4, 64, dtype=torch.float32)
    check(S, x, positions(2, 50, 2 ** 31 - 1), f, layout)
    check(S, x, positions(2, 50, 2 ** 31 - 1), torch.full((32,), 7.25, dtype=torch.float64), layout)  # over a turn


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_rope_strided_views_and_in_place(S, layout, off):
    f, pos = S.rope_frequencies(64, device="cpu"), positions(3, 9)
    base = normal(4, 9, 6, 584)
    dev = base.cuda()
    view = dev[:, ::2, off:off + 192]
    got = check(S, base[:, ::2, off:off + 192], pos, f, layout, offset=128, x_dev=view, out=view)
    assert got.data_ptr() == view.data_ptr()
    after = dev.cpu()
    assert torch.equal(after[:, 1::2], base[:, 1::2])  # the heads between, and the columns around, as they were
    assert torch.equal(after[:, ::2, :off + 128], base[:, ::2, :off + 128])
    assert torch.equal(after[:, ::2, off + 192:], base[:, ::2, off + 192:])
    # tokens and heads exchanged in memory, into a strided place
    x = normal(5, 6, 9, 64)
    q = torch.zeros(9, 6, 576, dtype=torch.bfloat16, device="cuda")
    check(S, x.transpose(0, 1), pos, f, layout, x_dev=x.cuda().transpose(0, 1), out=q[..., 512:])
    assert not q[..., :512].any()


def test_rope_two_dimensional_and_empty(S):
    f = S.rope_frequencies(64, device="cpu")
    check(S, normal(6, 33, 64), positions(6, 33), f, "half")
    for shape in ((0, 4, 64), (4, 0, 64)):
        x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        assert S.rope(x, torch.zeros(shape[0], dtype=torch.int32, device="cuda"), f.cuda()).shape == shape


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_inverse_is_the_gradient(S, layout):
    """<rope(x + h d) - rope(x - h d), y> / 2h = <d, inverse(y)>: the map is linear, so the difference is
    exact up to the fp32 rounding of the three results (2^-20 of the sum of magnitudes covers it)."""
    f, pos = S.rope_frequencies(96, device="cuda"), positions(7, 40).cuda()
    x, d, y = (normal(s, 40, 3, 96, dtype=torch.float32).cuda() for s in (8, 9, 10))
    kw = dict(layout=layout, amplitude=0.8)
    up, down = S.rope(x + 0.5 * d, pos, f, **kw), S.rope(x - 0.5 * d, pos, f, **kw)
    left = ((up.double() - down.double()) * y.double()).sum()
    right = (d.double() * S.rope(y, pos, f, inverse=True, **kw).double()).sum()
    scale = ((x.abs() + d.abs()).double() * y.abs().double()).sum() * 2
    assert abs(float(left - right)) <= 2.0 ** -20 * float(scale)


def cache_values(cache, kind):
    if kind == 0:
        return cache.view(torch.bfloat16)
    return (cache[:, :512].view(torch.float8_e4m3fn).float().view(-1, 4, 128),
            cache[:, 512:528].view(torch.float32), cache[:, 528:656].view(torch.bfloat16))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("kind", [W.KV_BF16, W.KV_FP8_E4M3])
@pytest.mark.parametrize("T,H,pad", [(1, 1, 0), (1, 0, 16), (9, 16, 0), (64, 64, 48), (333, 3, 0)])
def test_rope_append(S, layout, kind, T, H, pad):
    row = S.svt.ROW_BYTES[kind] + pad
    pages, page = (T + 40) // 8, 8
    before = torch.randint(0, 256, (pages * page, row), generator=torch.Generator().manual_seed(1), dtype=torch.uint8)
    cache = before.cuda()
    kv = S.KVCache(cache, pages, page, kind, row_stride_bytes=row)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:T].to(torch.int32)
    slots[3::7] = -1
    if T > 8:
        slots[8] = -2 ** 31
    lat, kr = normal(3, T, 512) * 3, normal(4, T, 64)
    lat[0, :128] = 0  # a block of zeros
    lat[-1, 128:256] *= 1e-30
    pos, f = positions(5, T), S.rope_frequencies(64, device="cpu")
    wide = torch.zeros(T, 640, dtype=torch.bfloat16)
    wide[:, :512], wide[:, 512:576] = lat, kr
    wide = wide.cuda()
    q = torch.full((T, H, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    qr = normal(6, T, H, 64)
    ws = S.Workspace()
    S.rope_append(wide[:, :512], wide[:, 512:576], pos.cuda(), slots.cuda(), kv, f.cuda(), layout=layout,
                  q_rope=qr.cuda() if H else None, q_out=q[..., 512:] if H else None, ws=ws)
    assert ws.read_status() == 0
    after = cache.cpu()
    live = slots >= 0
    at = slots[live].long()
    untouched = torch.ones(pages * page, dtype=torch.bool)
    untouched[at] = False
    assert torch.equal(after[untouched], before[untouched])
    n = S.svt.ROW_BYTES[kind]
    assert torch.equal(after[:, n:], before[:, n:])
    ref = R.rotate(kr[:, None], pos, f, layout)[:, 0][live]
    bound = R.rotate_bound(kr[:, None], R.rotate(kr[:, None], pos, f, layout), layout, torch.bfloat16, 1.0, pos, f)[:, 0][live]
    rows = after[at][:, :n].contiguous()
    if kind == W.KV_BF16:
        values = cache_values(rows, kind)
        assert torch.equal(values[:, :512], lat[live])
        R.within(values[:, 512:], ref, bound, "rope")
    else:
        codes, scales, rope = cache_values(rows, kind)
        x = lat[live].float().view(-1, 4, 128)
        amax = x.abs().amax(-1)
        want = torch.where(amax > 0, amax / 448.0, 1.0)
        assert torch.equal(scales, want)
        assert torch.equal(codes, (x / want[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).float())
        # the value held is within half an e4m3 step (2^-4) of the latent, or half the smallest step (2^-10)
        held = codes.double() * scales.double()[..., None]
        assert torch.all((held - x).abs() <= x.abs() * 2.0 ** -4 * 1.001 + want[..., None] * 2.0 ** -10 * 1.001 + 1e-37)
        R.within(rope, ref, bound, "rope")
    if H:
        refq = R.rotate(qr, pos, f, layout)
        R.within(q[..., 512:], refq, R.rotate_bound(qr, refq, layout, torch.bfloat16, 1.0, pos, f), "q")
        assert bool((q[..., :512] == 5).all())


def test_rope_append_reports_what_it_cannot_hold(S):
    f = S.rope_frequencies(64)
    lat, kr = normal(1, 4, 512).cuda(), normal(2, 4, 64).cuda()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    for kind in (W.KV_BF16, W.KV_FP8_E4M3):
        row = S.svt.ROW_BYTES[kind]
        cache = torch.full((8, row), 7, dtype=torch.uint8, device="cuda")
        ws = S.Workspace()
        kv = S.KVCache(cache, 2, 4, kind)
        S.rope_append(lat, kr, pos, torch.tensor([8, 2 ** 31 - 1, -1, 3], dtype=torch.int32).cuda(), kv, f, ws=ws)
        assert ws.read_status() == S.svt.DEV_ERR_INDEX_RANGE
        changed = (cache != 7).any(1).cpu()
        assert changed.tolist() == [False] * 3 + [True] + [False] * 4
        big = lat.clone()
        big[2, 300] = 1e5
        S.rope_append(big, kr, pos, pos, kv, f, ws=ws)
        assert ws.read_status() == (S.svt.DEV_ERR_FP8_RANGE if kind == W.KV_FP8_E4M3 else 0)
        big[2, 300] = float("nan")
        S.rope_append(big, kr, pos, pos, kv, f, ws=ws)
        assert ws.read_status() == (S.svt.DEV_ERR_FP8_RANGE if kind == W.KV_FP8_E4M3 else 0)


def test_rope_append_in_a_graph_and_on_another_stream(S):
    f = S.rope_frequencies(64)
    T, H = 5, 8
    kv = S.KVCache(torch.zeros(16, 1152, dtype=torch.uint8, device="cuda"), 16, 1, W.KV_BF16)
    lat, kr, qr = normal(1, T, 512).cuda(), normal(2, T, 64).cuda(), normal(3, T, H, 64).cuda()
    pos, slots = torch.arange(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    q, ws = torch.zeros(T, H, 64, dtype=torch.bfloat16, device="cuda"), S.Workspace()
    g = torch.cuda.CUDAGraph()
    S.rope_append(lat, kr, pos, slots, kv, f, q_rope=qr, q_out=q, ws=ws)
    with torch.cuda.graph(g):
        S.rope_append(lat, kr, pos, slots, kv, f, q_rope=qr, q_out=q, ws=ws)
    pos += 100
    slots += 6
    g.replay()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        q2 = S.rope(qr, pos, f)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(q, q2)
    ref = R.rotate(kr.cpu()[:, None], pos.cpu(), f.cpu(), "interleaved")[:, 0]
    got = kv.data.view(torch.bfloat16)[6:11, 512:]
    R.within(got, ref, R.rotate_bound(kr.cpu()[:, None], ref[:, None], "interleaved", torch.bfloat16)[:, 0])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_negative_large_and_zero_frequencies(S, layout):
    f = torch.tensor([0.0, -0.75, 1e-12, 3e-320, 41.5, -1e4], dtype=torch.float64)
    check(S, normal(11, 30, 2, 12, dtype=torch.float32), positions(12, 30), f, layout)


def test_rope_broadcast_input_and_refused_overlapping_output(S):
    f = S.rope_frequencies(64, device="cpu")
    x = normal(13, 5, 1, 64)
    wide = x.cuda().expand(5, 7, 64)
    check(S, x.expand(5, 7, 64), positions(14, 5), f, "half", x_dev=wide)
    with pytest.raises(S.SvtError):
        S.rope(wide, positions(14, 5).cuda(), f.cuda(), out=wide)
    with pytest.raises(TypeError):
        S.rope(wide, positions(14, 5), f.cuda())  # positions on the CPU


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_frequencies_that_are_no_frequency_give_nan(S, layout, dtype):
    """NaN, infinities and magnitudes of 2^52 and above: NaN in their own pair, the other pairs as ever."""
    bad = [math.nan, math.inf, -math.inf, 2.0 ** 52, -1e300]
    f = torch.tensor([0.5, *bad, 0.0, -3.25], dtype=torch.float64)
    n, T = len(f), 5
    x, pos = normal(15, T, 2, 2 * n, dtype=dtype), torch.tensor([1, -7, 3, 2 ** 31 - 1, 12], dtype=torch.int32)
    got = S.rope(x.cuda(), pos.cuda(), f.cuda(), layout=layout).cpu()
    ok = torch.ones(n, dtype=torch.bool)
    ok[1: 1 + len(bad)] = False
    cols = torch.cat([ok, ok]) if layout == "half" else ok.repeat_interleave(2)
    assert bool(got[..., ~cols].isnan().all())
    keep = x[..., cols]
    ref = R.rotate(keep, pos, f[ok], layout)
    R.within(got[..., cols], ref, R.rotate_bound(keep, ref, layout, dtype, 1.0, pos, f[ok]))


def test_rope_append_of_a_frequency_that_is_none_gives_nan(S):
    f = S.rope_frequencies(64, device="cpu")
    f[3], f[17] = math.nan, math.inf
    T = 4
    lat, kr, pos = normal(16, T, 512), normal(17, T, 64), torch.arange(1, T + 1, dtype=torch.int32)
    for kind in (W.KV_BF16, W.KV_FP8_E4M3):
        kv = S.KVCache(torch.zeros(T, S.svt.ROW_BYTES[kind], dtype=torch.uint8, device="cuda"), T, 1, kind)
        ws = S.Workspace()
        S.rope_append(lat.cuda(), kr.cuda(), pos.cuda(), (pos - 1).cuda(), kv, f.cuda(), layout="half", ws=ws)
        values = cache_values(kv.data.cpu(), kind)
        rope = values[:, 512:] if kind == W.KV_BF16 else values[2]
        bad = torch.zeros(64, dtype=torch.bool)
        bad[[3, 17, 35, 49]] = True
        assert torch.equal(rope.isnan(), bad.expand(T, 64))


def test_rope_large_frequencies_to_the_documented_error(S):
    """|pos| (|freq| + 1) 2^-64 turns, next to the fp32 roundings: against the angle modulo a turn from exact
    fractions and 50 digits of pi."""
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    f = torch.tensor([2.0 ** 20 + 1 / 3, -(2.0 ** 33) - 0.7, 2.0 ** 45 + 9, 2.0 ** 52 - 1], dtype=torch.float64)
    pos = torch.tensor([1, -3, 1000, 2 ** 31 - 1], dtype=torch.int32)
    x = normal(18, len(pos), 1, 2 * len(f), dtype=torch.float32)
    got = S.rope(x.cuda(), pos.cuda(), f.cuda()).cpu().double()
    for t in range(len(pos)):
        for i in range(len(f)):
            turns = Fraction(int(pos[t])) * Fraction(float(f[i])) / (2 * pi)
            a = float((turns - round(turns)) * 2 * pi)
            u, v = x[t, 0, 2 * i].double(), x[t, 0, 2 * i + 1].double()
            off = 2 * math.pi * abs(int(pos[t])) * (abs(float(f[i])) + 1) * 2.0 ** -64 + 2.0 ** -21
            assert abs(got[t, 0, 2 * i] - (u * math.cos(a) - v * math.sin(a))) <= off * (abs(u) + abs(v))
            assert abs(got[t, 0, 2 * i + 1] - (u * math.sin(a) + v * math.cos(a))) <= off * (abs(u) + abs(v))


def test_rope_an_option_without_a_truth_value_is_refused_as_python_does(S):
    x, pos = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError, match="ambiguous"):
        S.rope(x, pos, S.rope_frequencies(64), inverse=torch.tensor([1, 0]))
    z = torch.zeros(1, 4, device="cuda")
    with pytest.raises(RuntimeError, match="ambiguous"):
        S.distill_topk(z, pos[None], z[:, :1], need_grad=torch.tensor([1, 0]))


def test_rope_out_of_memory_is_torch_s_error(S):
    """An output of 2^46 bytes (nothing is allocated, nor launched)."""
    x = torch.zeros(1, 1, 16384, dtype=torch.bfloat16, device="cuda").expand(131071, 16384, 16384)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        S.rope(x, torch.zeros(131071, dtype=torch.int32, device="cuda"), S.rope_frequencies(64))
