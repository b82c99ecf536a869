"""A beam search's steps, as a server makes them: selection, pages, rows into the cache, attention over the shared prompt."""

import numpy as np
import pytest
import torch

import sparse_mla_attention_top_gb300 as S
from tests import _serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_steps_of_a_search(kind):
    B, W, V, H, page, pages, blocks, steps = 3, 4, 5000, 16, 16, 400, 24, 20
    prompt = [150, 33, 64]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    dtype, row = (S.KV_BF16, 1152) if kind == "bf16" else (S.KV_FP8_E4M3, 656)
    kv = S.KVCache(torch.zeros((pages * page, row), dtype=torch.uint8, device="cuda"), pages, page, dtype)
    freqs = S.rope_frequencies(64)
    ws = S.Workspace()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    empty = torch.empty((0, blocks), dtype=torch.int32, device="cuda")
    # the prompts are admitted and written, then forked into W beams each
    table, lens, slots, _ = S.fork_pages(kv, refs, empty, empty[:, 0], i32([-1] * B), grow=i32(prompt), max_grow=max(prompt),
                                         ws=ws)
    at = slots.flatten()
    pos = torch.arange(max(prompt), dtype=torch.int32, device="cuda").repeat(B)
    S.rope_append(normal(at.numel(), 512), normal(at.numel(), 64), pos, at, kv, freqs, ws=ws)
    table, lens, _, _ = S.fork_pages(kv, refs, table, lens, i32(np.repeat(np.arange(B), W)), ws=ws)
    start, prefix = i32(np.arange(B + 1) * W), i32(prompt)
    scores = torch.full((B, W), -torch.inf, device="cuda")
    scores[:, 0] = 0
    finished = torch.zeros((B, W), dtype=torch.bool, device="cuda")
    head = normal(512 * H, V)
    hidden = normal(B * W, 512 * H)
    # each beam's rows as a list of their values, kept apart
    held = R.cache_rows(kv.data, kind)
    rows = [[held[table[b * W, p // page] * page + p % page] for p in range(prompt[b])] for b in range(B) for _ in range(W)]
    for step in range(steps):
        logits = (hidden.float() @ head.float() * 0.003).view(B, W, V).to(torch.bfloat16)
        value, parents, tokens = S.beam_select(logits, scores, W, finished=finished, end_token=7, ws=ws)
        for b, (v, p, t) in enumerate(R.beam(logits, scores, W, finished, 7)):
            assert parents[b].tolist() == p.tolist() and tokens[b].tolist() == t.tolist()
        finished = finished.gather(1, parents.long()) | (tokens == 7)
        if step == 5:
            finished[0, 1] = True
        scores = value
        whole = (parents + torch.arange(B, dtype=torch.int32, device="cuda")[:, None] * W).flatten().contiguous()
        table, lens, slots, _ = S.fork_pages(kv, refs, table, lens, whole, grow=1, ws=ws)
        assert int(refs.sum()) == int((table >= 0).sum())
        q_pe, q = normal(B * W, H, 64), normal(B * W, H, 576)
        S.rope_append(normal(B * W, 512), normal(B * W, 64), lens - 1, slots[:, 0].contiguous(), kv, freqs, q_rope=q_pe,
                      q_out=q[..., 512:], ws=ws)
        if step == 11:
            table, _, mapping = S.compact_pages(kv, refs, table, ws=ws)
            slots = torch.where(slots >= 0, mapping[(slots // page).long()] * page + slots % page, -1)
            assert int((refs > 0).sum()) == int((mapping >= 0).sum()) == int(mapping.max()) + 1
        out, lse = S.mla_decode_shared_prefix(q, kv, table, lens, start, prefix, 576 ** -0.5, ws=ws)
        held = R.cache_rows(kv.data, kind)
        rows = [rows[p] + [held[int(slots[i, 0])]] for i, p in enumerate(whole.tolist())]
        flat = torch.cat([torch.stack(r) for r in rows])
        ends = np.cumsum([len(r) for r in rows])
        lists = [np.arange(e - len(r), e) for e, r in zip(ends, rows)]
        R.check_attention((out, lse), R.attention(q, flat, lists, 576 ** -0.5, kind))
        hidden = out.flatten(1)
    assert ws.read_status() == 0
    # the search ends: every page is free
    S.fork_pages(kv, refs, table, lens, i32([]), ws=ws)
    assert not refs.any()


def test_items_with_fewer_candidates_than_beams():
    """Items in the middle of the batch that run out of candidates: their rows come back empty, and no other item's row goes on
    in their place."""
    B, W, V, H, page, pages, blocks = 4, 4, 300, 16, 16, 200, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kv = S.KVCache(torch.randn((pages * page, 576), generator=g, device="cuda").to(torch.bfloat16).view(torch.uint8), pages,
                   page, S.KV_BF16)
    refs, ws = torch.zeros(pages, dtype=torch.int32, device="cuda"), S.Workspace()
    empty = torch.empty((0, blocks), dtype=torch.int32, device="cuda")
    prompt = [40, 33, 64, 17]
    table, lens, _, _ = S.fork_pages(kv, refs, empty, empty[:, 0], i32([-1] * B), grow=i32(prompt), max_grow=max(prompt), ws=ws)
    table, lens, _, _ = S.fork_pages(kv, refs, table, lens, i32(np.repeat(np.arange(B), W)), ws=ws)
    logits = torch.randn((B, W, V), generator=g, device="cuda")
    logits[1, :, 2:] = -torch.inf  # two tokens left in one beam of item 1, none in the others
    logits[1, 1:] = -torch.inf
    logits[2] = float("nan")       # no candidate in item 2
    value, parents, tokens = S.beam_select(logits, torch.zeros((B, W), device="cuda"), W, ws=ws)
    assert parents[1].tolist()[2:] == [-1, -1] and parents[1].tolist()[:2] == [0, 0] and (parents[2] == -1).all()
    first = torch.arange(B, dtype=torch.int32, device="cuda")[:, None] * W
    rows = torch.where(parents >= 0, parents + first, -1).flatten()
    old = table.clone()
    table, lens, slots, _ = S.fork_pages(kv, refs, table, lens, rows, grow=1, ws=ws)
    assert ws.read_status() == 0
    live = (parents >= 0).flatten().tolist()
    for i, go_on in enumerate(live):
        assert int(lens[i]) == (prompt[i // W] + 1 if go_on else 1)
        full = prompt[i // W] // page if go_on else 0
        assert torch.equal(table[i, :full], old[i // W * W, :full])
    assert int(refs.sum()) == int((table >= 0).sum())
    held = R.cache_rows(kv.data, "bf16")
    q = torch.randn((B * W, H, 576), generator=g, device="cuda").to(torch.bfloat16)
    got = S.mla_decode_shared_prefix(q, kv, table, lens, i32(np.arange(B + 1) * W), i32(prompt), 576 ** -0.5, ws=ws)
    assert ws.read_status() == 0
    # (an empty row's one position lies below its group's prefix and is read through the group's first row)
    at = lambda i, n: [int(table[i, p // page]) * page + p % page for p in range(n)]  # noqa: E731
    lists = [np.asarray(at(i, int(lens[i])) if go_on else at(i // W * W, 1)) for i, go_on in enumerate(live)]
    R.check_attention(got, R.attention(q, held, lists, 576 ** -0.5, "bf16"))
