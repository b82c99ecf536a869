"""Measured cases of the operators around sparse MLA attention in training and serving: rotary
positions, writing rotated rows into the paged latent cache, the attention's backward pass, and
the distillation loss that trains an indexer on a teacher's top entries.

`run` computes each in plain torch operations where `own` is false, and through the package
where it is true. Inputs come from `prepare`, made from the seed alone.
"""

import math

import numpy as np
import torch

own = False

LATENT, ROPE, ROW = 512, 64, 576
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the rope columns of 64 decode queries of 64 heads, rotated into their places in q
        dict(name="rope_decode_t64_h64", op="rope", T=64, H=64, D=64, dim=64, offset=0, layout="interleaved",
             dtype="bf16", inverse=False, into_q=True, scaled=True, far=47104),
        # a prefill's projected query heads (128 plain + 64 rotated columns), out of place
        dict(name="rope_prefill_t8192_h64_d192", op="rope", T=8192, H=64, D=192, dim=64, offset=128, layout="half",
             dtype="bf16", inverse=False, into_q=False, scaled=False, far=8192),
        # the gradient of a rotation in fp32: odd count of tokens, far positions
        dict(name="rope_grad_t1021_h16_f32", op="rope", T=1021, H=16, D=160, dim=96, offset=32, layout="half",
             dtype="f32", inverse=True, into_q=False, scaled=True, far=1000003),
        # one decode step of 128 requests: q's rope columns and the new rows of an e4m3 cache
        dict(name="append_decode_e4m3_t128_h64", op="append", T=128, H=64, layout="interleaved", kv="e4m3",
             page_size=64, far=47104, skip=False),
        # a prefill's rows into a bf16 cache, with the rope columns of its 16-head queries
        dict(name="append_prefill_bf16_t8192_h16", op="append", T=8192, H=16, layout="half", kv="bf16",
             page_size=64, far=32768, skip=False),
        # a padded batch's rows into an e4m3 cache, some of them without a slot, no queries
        dict(name="append_ragged_e4m3_t4093", op="append", T=4093, H=0, layout="interleaved", kv="e4m3",
             page_size=16, far=47104, skip=True),
        # a handful of queries late in a short sequence
        dict(name="backward_t7_h16_k200", op="backward", T=7, H=16, K=200, ctx=333, page_size=16, dlse=True),
        # 16 heads over a long context, an odd count of queries
        dict(name="backward_t333_h16_k2048", op="backward", T=333, H=16, K=2048, ctx=24576, page_size=64, dlse=False),
        # the last 1024 tokens of an 8192-token sequence, 64 heads
        dict(name="backward_t1024_h64_k2048", op="backward", T=1024, H=64, K=2048, ctx=8192, page_size=64,
             dlse=False),
        # 128 heads, the first tokens of a sequence (most lists short of K)
        dict(name="backward_t509_h128_k1024", op="backward", T=509, H=128, K=1024, ctx=1531, page_size=64,
             dlse=False),
        # the indexer's loss over all candidates of a 1024-token step at context 32768
        dict(name="distill_t1024_n32768_f32", op="distill", T=1024, N=32768, K=2048, dtype="f32", scope="candidates",
             kind="weights", ragged=True),
        # the loss over the selected entries alone, scores in bf16, from teacher logits
        dict(name="distill_t67_n8191_bf16_listed", op="distill", T=67, N=8191, K=500, dtype="bf16", scope="listed",
             kind="logits", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "backward", "backward", "distill"])
    if op == "rope":
        T, H = _log(rng, 1, 8192), rng.choice([1, 8, 16, 24, 64])
        dim = rng.choice([32, 64, 96])
        D = dim + rng.choice([0, 0, 32, 128])
        return dict(op="rope", T=T, H=H, D=D, dim=dim, offset=rng.choice([0, D - dim]),
                    layout=rng.choice(["interleaved", "half"]), dtype=rng.choice(["bf16", "f32"]) if T < 2048 else "bf16",
                    inverse=rng.random() < 0.5, into_q=False, scaled=rng.random() < 0.5, far=_log(rng, 256, 1 << 20))
    if op == "append":
        return dict(op="append", T=_log(rng, 1, 8192), H=rng.choice([0, 1, 8, 16]),
                    layout=rng.choice(["interleaved", "half"]), kv=rng.choice(["bf16", "e4m3"]),
                    page_size=rng.choice([1, 16, 64]), far=_log(rng, 256, 1 << 17), skip=rng.random() < 0.5)
    if op == "backward":
        H = rng.choice([1, 5, 8, 16, 16, 32, 64, 128])
        T = _log(rng, 1, min(1024, 32768 // H))
        ctx = T + _log(rng, 64, 16384)
        return dict(op="backward", T=T, H=H, K=_log(rng, 16, 2048 if T * H <= 32768 else 1024), ctx=ctx,
                    page_size=rng.choice([1, 16, 64]), dlse=rng.random() < 0.5)
    T = _log(rng, 1, 1024)
    N = _log(rng, 64, 32768)
    return dict(op="distill", T=T, N=N, K=_log(rng, 1, 2048), dtype=rng.choice(["f32", "bf16"]),
                scope=rng.choice(["candidates", "listed"]), kind=rng.choice(["weights", "logits"]),
                ragged=rng.random() < 0.7)


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _frequencies(dim, scaled):
    """Radians per position of each rotated pair, fp64: base 10000, and where `scaled` the by-parts
    rule for a context 40 times a 4096-token original one (fast pairs keep their frequency, slow
    ones are divided by the factor, those between are blended)."""
    f = 10000.0 ** (-np.arange(0, dim, 2, dtype=np.float64) / dim)
    if scaled:
        def pair_of(turns):
            return dim * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
        lo, hi = max(math.floor(pair_of(32)), 0), min(math.ceil(pair_of(1)), dim - 1)
        ramp = np.clip((np.arange(dim // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        f = f / 40 * ramp + f * (1 - ramp)
    return torch.from_numpy(f).cuda()


def _block_table(g, ctx, page):
    pages = -(-ctx // page)
    return torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None, :], pages


def _prepare_rope(c, g):
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    x = _normal(g, (c["T"], c["H"], c["D"]), dt)
    pos = torch.randint(0, c["far"], (c["T"],), generator=g, device="cuda", dtype=torch.int32)
    # decode: the rotated columns go to their place behind q's latent ones
    out = torch.empty((c["T"], c["H"], ROW), dtype=dt, device="cuda")[..., LATENT:] if c["into_q"] else torch.empty_like(x)
    return dict(x=x, pos=pos, out=out, freqs=_frequencies(c["dim"], c["scaled"]),
                amplitude=0.1 * math.log(40) + 1 if c["scaled"] else 1.0)


def _prepare_append(c, g):
    T, P = c["T"], c["page_size"]
    pages = -(-(T + T // 8 + P) // P)
    row = 1152 if c["kv"] == "bf16" else 656
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:T].to(torch.int32)
    if c["skip"]:
        slots = torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, -1, slots).to(torch.int32)
    s = dict(cache=torch.zeros((pages * P, row), dtype=torch.uint8, device="cuda"), pages=pages, slots=slots,
             latent=_normal(g, (T, LATENT)), k_rope=_normal(g, (T, ROPE)), freqs=_frequencies(ROPE, True),
             pos=torch.randint(0, c["far"], (T,), generator=g, device="cuda", dtype=torch.int32))
    if c["H"]:
        s["q_rope"] = _normal(g, (T, c["H"], ROPE))
        s["q"] = torch.zeros((T, c["H"], ROW), dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_backward(c, g):
    T, H, K, ctx = c["T"], c["H"], c["K"], c["ctx"]
    bt, pages = _block_table(g, ctx, c["page_size"])
    kv = _normal(g, (pages * c["page_size"], ROW))
    q, dout = _normal(g, (T, H, ROW)), _normal(g, (T, H, LATENT))
    # query i sits at position ctx - T + i and selects from its prefix, in ascending order
    topk = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    for a in range(0, T, 256):
        b = min(T, a + 256)
        score = torch.rand((b - a, ctx), generator=g, device="cuda")
        prefix = torch.arange(ctx - T + a + 1, ctx - T + b + 1, device="cuda")[:, None]
        score = torch.where(torch.arange(ctx, device="cuda")[None] < prefix, score, -1.0)
        v, i = score.topk(min(K, ctx), dim=1)
        i = torch.where(v >= 0, i, ctx).sort(dim=1).values
        topk[a:b, :i.shape[1]] = torch.where(i < ctx, i, -1).to(torch.int32)
    scale = ROW ** -0.5
    out = torch.empty((T, H, LATENT), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((T, H), device="cuda")
    for a in range(0, T, 64):
        rows, live = _rows(kv, bt, topk[a:a + 64], c["page_size"])
        sc = torch.matmul(q[a:a + 64].float(), rows.transpose(1, 2)) * scale
        sc = torch.where(live[:, None], sc, -math.inf)
        lse[a:a + 64] = torch.logsumexp(sc, -1)
        out[a:a + 64] = torch.matmul(torch.exp(sc - lse[a:a + 64, :, None]), rows[..., :LATENT]).to(torch.bfloat16)
    s = dict(q=q, kv=kv, pages=pages, page_size=c["page_size"], topk=topk, block_table=bt, out=out, lse=lse,
             dout=dout, dlse=None, scale=scale, seq=torch.tensor([ctx], dtype=torch.int32, device="cuda"),
             req=torch.zeros(T, dtype=torch.int32, device="cuda"))
    if c["dlse"]:
        s["dlse"] = torch.randn((T, H), generator=g, device="cuda")
    return s


def _prepare_distill(c, g):
    T, N, K = c["T"], c["N"], c["K"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    scores = (torch.randn((T, N), generator=g, device="cuda") * 2).to(dt)
    lens = torch.full((T,), N, dtype=torch.int32, device="cuda")
    if c["ragged"]:
        lens = torch.randint(0, N + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    # the student's own selection with noise, as a teacher that mostly agrees: distinct, ascending
    noisy = scores.float() + torch.randn((T, N), generator=g, device="cuda")
    noisy = torch.where(torch.arange(N, device="cuda")[None] < lens[:, None], noisy, -math.inf)
    v, i = noisy.topk(min(K, N), dim=1)
    i, order = torch.where(v > -math.inf, i, N).sort(dim=1)
    v = v.gather(1, order)
    idx = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    idx[:, :i.shape[1]] = torch.where(i < N, i, -1).to(torch.int32)
    teacher = torch.zeros((T, K), device="cuda")
    value = torch.where(i < N, v, 0.0)
    teacher[:, :i.shape[1]] = torch.exp(value) if c["kind"] == "weights" else value
    return dict(scores=scores, lens=lens, idx=idx, teacher=teacher, temperature=1.0 if c["kind"] == "weights" else 2.0,
                row_weight=torch.full((T,), 1.0 / T, device="cuda"))


def prepare(case, seed):
    g = _gen(seed)
    s = {"rope": _prepare_rope, "append": _prepare_append, "backward": _prepare_backward,
         "distill": _prepare_distill}[case["op"]](case, g)
    s["case"] = dict(case)
    return s


# -------------------------------------------------------------------------------- plain forms

def _rotate(x, pos, freqs, layout, inverse, amplitude):
    """Rotation of the pairs of x [T, H, dim] by pos * freqs, in 32 bits; the angles in 64."""
    angle = pos.double()[:, None] * freqs[None]
    cos, sin = (torch.cos(angle) * amplitude).float()[:, None], (torch.sin(angle) * amplitude).float()[:, None]
    if inverse:
        sin = -sin
    x = x.float()
    if layout == "half":
        a, b = x[..., :x.shape[-1] // 2], x[..., x.shape[-1] // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _plain_rope(s, c):
    lo, hi = c["offset"], c["offset"] + c["dim"]
    out = s["out"]
    out[..., :lo] = s["x"][..., :lo]
    out[..., hi:] = s["x"][..., hi:]
    out[..., lo:hi] = _rotate(s["x"][..., lo:hi], s["pos"], s["freqs"], c["layout"], c["inverse"],
                              s["amplitude"]).to(out.dtype)
    return out


def _cache_parts(cache, kind):
    """The cache's values as they are held: bf16 rows, or e4m3 codes, fp32 scales and bf16 rope."""
    if kind == "bf16":
        return cache.view(torch.bfloat16)
    return (cache[:, :LATENT].view(torch.float8_e4m3fn), cache[:, LATENT:LATENT + 16].view(torch.float32),
            cache[:, LATENT + 16:].view(torch.bfloat16))


def _plain_append(s, c):
    T = c["T"]
    rope = _rotate(s["k_rope"][:, None], s["pos"], s["freqs"], c["layout"], False, 1.0)[:, 0].to(torch.bfloat16)
    if c["kv"] == "bf16":
        row = torch.cat([s["latent"], rope], 1).view(torch.uint8)
    else:
        x = s["latent"].float().view(T, 4, 128)
        amax = x.abs().amax(-1)
        scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
        codes = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(T, LATENT)
        row = torch.cat([codes.view(torch.uint8), scale.view(torch.uint8), rope.view(torch.uint8)], 1)
    live = s["slots"] >= 0
    s["cache"][s["slots"][live].long()] = row[live]
    out = [_cache_parts(s["cache"], c["kv"])]
    if c["H"]:
        s["q"][..., LATENT:] = _rotate(s["q_rope"], s["pos"], s["freqs"], c["layout"], False, 1.0).to(torch.bfloat16)
        out.append(s["q"])
    return out


def _rows(kv, bt, topk, page):
    """The listed rows [T, K, 576] in fp32, zero where the entry is dead, and which are live."""
    live = topk >= 0
    pos = topk.clamp(min=0).long()
    slot = bt[0].long()[pos // page] * page + pos % page
    return torch.where(live[..., None], kv[slot].float(), 0.0), live


def _plain_backward(s, c):
    kv, scale = s["kv"], s["scale"]
    rows, live = _rows(kv, s["block_table"], s["topk"], c["page_size"])
    q, do = s["q"].float(), s["dout"].float()
    p = torch.exp(torch.matmul(q, rows.transpose(1, 2)) * scale - s["lse"][..., None])
    p = torch.where(live[:, None], p, 0.0)
    delta = (do * s["out"].float()).sum(-1)
    if s["dlse"] is not None:
        delta = delta - s["dlse"]
    dp = torch.matmul(do, rows[..., :LATENT].transpose(1, 2))
    ds = p * (dp - delta[..., None]) * scale
    dq = torch.matmul(ds, rows).to(torch.bfloat16)
    drows = torch.matmul(ds.transpose(1, 2), q)
    drows[..., :LATENT] += torch.matmul(p.transpose(1, 2), do)
    pos = s["topk"].clamp(min=0).long()
    slot = s["block_table"][0].long()[pos // c["page_size"]] * c["page_size"] + pos % c["page_size"]
    dkv = torch.zeros((kv.shape[0], ROW), device="cuda")
    dkv.index_add_(0, slot.flatten(), drows.flatten(0, 1))  # dead entries add a row of zeros
    return dq, dkv.to(torch.bfloat16), p.sum(1)


def _plain_distill(s, c):
    x, tau = s["scores"].float() / s["temperature"], s["temperature"]
    T, N = x.shape
    live = (s["idx"] >= 0) & (s["idx"] < s["lens"][:, None])
    at = torch.where(live, s["idx"], 0).long()
    w = s["teacher"]
    if c["kind"] == "logits":
        w = torch.where(live, w / tau, -math.inf)
        w = torch.exp(w - w.amax(1, keepdim=True).clamp(min=-3e38))
    w = torch.where(live, w, 0.0)
    p = w / w.sum(1, keepdim=True).clamp(min=1e-38)
    p = torch.where(w.sum(1, keepdim=True) > 0, p, 0.0)
    if c["scope"] == "candidates":
        x = torch.where(torch.arange(N, device="cuda")[None] < s["lens"][:, None], x, -math.inf)
    else:
        inside = torch.zeros((T, N), device="cuda").scatter_add_(1, at, live.float()) > 0
        x = torch.where(inside, x, -math.inf)
    m = x.amax(1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - m)
    z = e.sum(1, keepdim=True).clamp(min=1e-38)
    log_q = (x - m).gather(1, at) - torch.log(z)
    loss = torch.where(p > 0, p * (torch.log(p.clamp(min=1e-38)) - log_q), 0.0).sum(1)
    some = (p > 0).any(1, keepdim=True)
    grad = torch.where(some, e / z, 0.0).scatter_add_(1, at, -p)
    return loss, (grad * s["row_weight"][:, None] / tau).to(s["scores"].dtype)


# ----------------------------------------------------------------------------------- one pass

def _own(s, c):
    import sparse_mla_attention_top_gb300 as S

    if c["op"] == "rope":
        return S.rope(s["x"], s["pos"], s["freqs"], offset=c["offset"], layout=c["layout"], inverse=c["inverse"],
                      amplitude=s["amplitude"], out=s["out"])
    if c["op"] == "append":
        kv = S.KVCache(s["cache"], s["pages"], c["page_size"], S.KV_BF16 if c["kv"] == "bf16" else S.KV_FP8_E4M3)
        if c["H"]:
            S.rope_append(s["latent"], s["k_rope"], s["pos"], s["slots"], kv, s["freqs"], layout=c["layout"],
                          q_rope=s["q_rope"], q_out=s["q"][..., LATENT:])
            return [_cache_parts(s["cache"], c["kv"]), s["q"]]
        S.rope_append(s["latent"], s["k_rope"], s["pos"], s["slots"], kv, s["freqs"], layout=c["layout"])
        return [_cache_parts(s["cache"], c["kv"])]
    if c["op"] == "backward":
        kv = S.KVCache(s["kv"], s["pages"], c["page_size"], S.KV_BF16)
        return S.sparse_mla_backward(s["q"], kv, s["topk"], s["scale"], s["out"], s["lse"], s["dout"], dlse=s["dlse"],
                                     block_table=s["block_table"], seq_lens=s["seq"], req_of_token=s["req"],
                                     return_weights=True)
    return S.distill_topk(s["scores"], s["idx"], s["teacher"], lens=s["lens"], row_weight=s["row_weight"],
                          temperature=s["temperature"], teacher_kind=c["kind"], over=c["scope"])


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"rope": _plain_rope, "append": _plain_append, "backward": _plain_backward,
            "distill": _plain_distill}[c["op"]](state, c)


# ------------------------------------------------------------------------- work, exact values

def work(case):
    c = case
    T = c["T"]
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2.0 * T * c["H"] * c["D"] * size + 4 * T + 4 * c["dim"], "flops": 3.0 * T * c["H"] * c["dim"]}
    if c["op"] == "append":
        live = T * (0.8 if c["skip"] else 1.0)
        row = 1152 if c["kv"] == "bf16" else 656
        return {"bytes": live * (1152 + row) + 8 * T + 4.0 * T * c["H"] * ROPE,
                "flops": 3.0 * T * (c["H"] + 1) * ROPE + live * LATENT}
    if c["op"] == "backward":
        live = float(sum(min(c["K"], c["ctx"] - T + i + 1) for i in range(T)))
        slots = -(-c["ctx"] // c["page_size"]) * c["page_size"]
        rows = T * c["H"]
        return {"bytes": rows * (1152 * 2 + 1024 * 2 + 4) + slots * 1152.0 * 2 + 8.0 * T * c["K"],
                "flops": 2 * c["H"] * live * (3 * ROW + 2 * LATENT)}
    size = 2 if c["dtype"] == "bf16" else 4
    n = c["N"] * (0.5 if c["ragged"] else 1.0)
    read = n if c["scope"] == "candidates" else min(n, c["K"])
    return {"bytes": T * (read * size + c["N"] * size + 8.0 * c["K"]), "flops": T * (6.0 * read + 6 * c["K"])}


def _exact_rotate(x, pos, freqs, layout, inverse, amplitude):
    # each pair as a complex number times amplitude * exp(+-i angle)
    a = pos.double()[:, None, None] * freqs
    turn = torch.polar(torch.full_like(a, amplitude), -a if inverse else a)
    x = x.double()
    n = freqs.numel()
    z = torch.complex(x[..., :n], x[..., n:]) if layout == "half" else torch.view_as_complex(
        x.unflatten(-1, (n, 2)).contiguous())
    z = z * turn
    return torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).flatten(-2)


def _exact_backward(s, c):
    T, K, P = c["T"], c["K"], c["page_size"]
    kv = s["kv"].double()
    dq = torch.zeros((T, c["H"], ROW), dtype=torch.float64, device="cuda")
    dkv = torch.zeros((kv.shape[0], ROW), dtype=torch.float64, device="cuda")
    weights = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    table = s["block_table"][0].long()
    for t in range(T):  # one query at a time, its live entries alone
        where = torch.nonzero(s["topk"][t] >= 0)[:, 0]
        pos = s["topk"][t][where].long()
        slot = table[torch.div(pos, P, rounding_mode="floor")] * P + pos.remainder(P)
        k, q, do = kv[slot], s["q"][t].double(), s["dout"][t].double()
        v = k[:, :LATENT]
        prob = torch.exp(q @ k.T * s["scale"] - s["lse"][t].double()[:, None])
        inner = (do * s["out"][t].double()).sum(1, keepdim=True)
        if s["dlse"] is not None:
            inner = inner - s["dlse"][t].double()[:, None]
        d_score = prob * (do @ v.T - inner) * s["scale"]
        dq[t] = d_score @ k
        d_row = d_score.T @ q
        d_row[:, :LATENT] += prob.T @ do
        dkv.index_add_(0, slot, d_row)
        weights[t, where] = prob.sum(0)
    return dq, dkv, weights


def _exact_distill(s, c):
    T, N = s["scores"].shape
    tau = s["temperature"]
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    grad = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for t in range(T):
        i = s["idx"][t]
        ok = (i >= 0) & (i < lens[t])
        i, w = i[ok].long(), s["teacher"][t][ok].double()
        if not i.numel():
            continue
        p = torch.softmax(w / tau, 0) if c["kind"] == "logits" else w / w.sum()
        x = s["scores"][t].double() / tau
        among = torch.arange(lens[t], device="cuda") if c["scope"] == "candidates" else i
        log_q = torch.log_softmax(x[among], 0)
        lq = log_q[i] if c["scope"] == "candidates" else log_q
        loss[t] = torch.special.xlogy(p, p).sum() - (p * lq).sum()
        grad[t, among] += torch.exp(log_q)
        grad[t].index_add_(0, i, -p)
    return loss, grad * s["row_weight"].double()[:, None] / tau


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rope":
        lo, hi = c["offset"], c["offset"] + c["dim"]
        x = s["x"].double()
        return torch.cat([x[..., :lo], _exact_rotate(x[..., lo:hi], s["pos"], s["freqs"], c["layout"], c["inverse"],
                                                     s["amplitude"]), x[..., hi:]], -1)
    if c["op"] == "append":
        live = torch.nonzero(s["slots"] >= 0)[:, 0]
        slot = s["slots"][live].long()
        n = s["cache"].shape[0]
        rope = torch.zeros((n, ROPE), dtype=torch.float64, device="cuda")
        rope[slot] = _exact_rotate(s["k_rope"][live][:, None], s["pos"][live], s["freqs"], c["layout"], False, 1.0)[:, 0]
        latent = torch.zeros((n, LATENT), dtype=torch.float64, device="cuda")
        x = s["latent"][live].double()
        if c["kv"] == "bf16":
            latent[slot] = x
            out = [torch.cat([latent, rope], 1)]
        else:
            # a block's scale is held in fp32: the value that fp32 nearest to its largest magnitude / 448
            block = x.unflatten(1, (4, 128))
            big = block.abs().amax(2)
            scale = torch.where(big > 0, (big / E4M3_MAX).float().double(), 1.0)
            scales = torch.zeros((n, 4), dtype=torch.float64, device="cuda")
            scales[slot] = scale
            latent[slot] = (block / scale[..., None]).flatten(1)  # the codes before their rounding
            out = [(latent, scales, rope)]
        if c["H"]:
            q = torch.zeros((c["T"], c["H"], ROW), dtype=torch.float64, device="cuda")
            q[..., LATENT:] = _exact_rotate(s["q_rope"], s["pos"], s["freqs"], c["layout"], False, 1.0)
            out.append(q)
        return out
    return _exact_backward(s, c) if c["op"] == "backward" else _exact_distill(s, c)
