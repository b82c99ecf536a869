"""The operators in the order a training step uses them: rotate and append a sequence's rows, select
from the indexer's scores, attend, differentiate, turn the rope gradients back, and train the
indexer on the attention's own weights. Each stage is held against fp64 of the stage's inputs."""

import pytest
import torch

from sparse_mla_attention_top_gb300 import workloads as W
from tests import _layer_ref as R

pytestmark = pytest.mark.gpu


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_training_step(layout):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_mla_attention_top_gb300 as S
    from sparse_mla_attention_top_gb300 import build

    build.build()
    T, H, K, P = 90, 16, 48, 16
    scale = 576 ** -0.5
    pages = -(-T // P)
    f = S.rope_frequencies(64, scaling="by_parts", factor=40.0, original_len=4096)
    bt = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)[None]
    pos = torch.arange(T, dtype=torch.int32)
    slots = (bt[0][pos.long() // P] * P + pos % P).to(torch.int32)
    latent, k_rope, q_in = normal(2, T, 512), normal(3, T, 64), normal(4, T, H, 576)
    kv = S.KVCache(torch.zeros(pages * P, 1152, dtype=torch.uint8, device="cuda"), pages, P, W.KV_BF16)
    ws = S.Workspace()
    q = q_in.cuda()
    S.rope_append(latent.cuda(), k_rope.cuda(), pos.cuda(), slots.cuda(), kv, f, layout=layout,
                  q_rope=q_in.cuda()[..., 512:], q_out=q[..., 512:], ws=ws)
    scores = torch.randn((T, T), generator=torch.Generator().manual_seed(5)).cuda()
    lens = (pos + 1).cuda()
    topk = S.topk_select(scores, K, lens=lens)
    req = torch.zeros(T, dtype=torch.int32, device="cuda")
    seq = torch.tensor([T], dtype=torch.int32, device="cuda")
    lists = dict(block_table=bt.cuda(), seq_lens=seq, req_of_token=req)
    out, lse = S.sparse_mla_decode(q, kv, topk, scale, ws=ws, **lists)
    dout = normal(6, T, H, 512)
    dq, dkv, weights = S.sparse_mla_backward(q, kv, topk, scale, out, lse, dout.cuda(), return_weights=True, ws=ws, **lists)
    loss, dscores = S.distill_topk(scores, topk, weights, lens=lens)
    dq0, dkv0 = dq.clone(), dkv.clone()
    S.rope(dq[..., 512:], pos.cuda(), f, layout=layout, inverse=True, out=dq[..., 512:])
    row_pos = torch.zeros(pages * P, dtype=torch.int32)
    row_pos[slots.long()] = pos
    S.rope(dkv[:, 512:], row_pos.cuda(), f, layout=layout, inverse=True, out=dkv[:, 512:])
    assert ws.read_status() == 0

    cpu = lambda t: t.cpu()  # noqa: E731
    topk_c = topk.cpu().long()
    resolved = torch.where(topk_c >= 0, slots.long()[topk_c.clamp(min=0)], -1)
    cache = kv.data.cpu().view(torch.bfloat16)
    # the rows that attention read are the rotated ones
    want = R.rotate(k_rope[:, None], pos, f.cpu(), layout)
    R.within(cache[slots.long(), 512:], want[:, 0], R.rotate_bound(k_rope[:, None], want, layout, torch.bfloat16)[:, 0])
    for t in (0, K - 1, T - 1):
        o, l = R.attention(q[t].double().cpu(), cache[resolved[t][resolved[t] >= 0]].double(), scale)
        assert float((out[t].double().cpu() - o).abs().max()) <= 2e-2 and float((lse[t].cpu() - l).abs().max()) <= 1e-3
    ref, bound = R.backward(cpu(q), cache, resolved, scale, cpu(out), cpu(lse), dout)
    for a, b, c in zip((dq0, dkv0, weights), ref, bound):
        R.within(a, b, c)
    # each row's weights sum to its heads: the probabilities of the forward, up to lse's 1e-3
    assert float((weights.double().sum(1) - H).abs().max()) <= 1e-3 * H * 1.01
    assert torch.equal(dq[..., :512], dq0[..., :512]) and torch.equal(dkv[:, :512], dkv0[:, :512])
    back = R.rotate(dq0.cpu()[..., 512:], pos, f.cpu(), layout, inverse=True)
    R.within(dq[..., 512:], back, R.rotate_bound(dq0.cpu()[..., 512:], back, layout, torch.bfloat16))
    back = R.rotate(dkv0.cpu()[:, None, 512:], row_pos, f.cpu(), layout, inverse=True)
    R.within(dkv[:, None, 512:], back, R.rotate_bound(dkv0.cpu()[:, None, 512:], back, layout, torch.bfloat16))
    (rl, rg), (bl, bg) = R.distill(cpu(scores), cpu(lens), cpu(topk), cpu(weights), "weights", "candidates", 1.0)
    R.within(loss, rl, bl)
    R.within(dscores, rg, bg + 2.0 ** -24 * rg.abs() + 2.0 ** -126)
    assert float(dscores.sum(1).abs().max()) <= 1e-5  # a softmax's gradient sums to zero
