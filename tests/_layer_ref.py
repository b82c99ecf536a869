"""fp64 statements of the operators around the attention, on the CPU in plain torch, with bounds on
what fp32 arithmetic and the stated roundings may add. They share no code with the library."""

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def rotate(x, pos, freqs, layout, inverse=False, amplitude=1.0):
    """x [T, H, dim] any type -> fp64, each pair as a complex number."""
    x = x.double()
    n = freqs.numel()
    a = pos.double()[:, None, None] * freqs.double() * (-1 if inverse else 1)
    z = torch.complex(x[..., :n], x[..., n:]) if layout == "half" else torch.complex(x[..., 0::2], x[..., 1::2])
    z = z * amplitude * torch.complex(torch.cos(a), torch.sin(a))
    return torch.cat([z.real, z.imag], -1) if layout == "half" else torch.view_as_real(z).flatten(-2)


def rotate_bound(x, ref, layout, dtype, amplitude=1.0, pos=None, freqs=None):
    """The angle pos * freq in fp64 has rounded here once (2^-53 of it) and in the kernel in 1 / 2 pi, in
    its product with freq and in the 64-bit fraction (each at most 2^-53 of it): with pos and freqs given,
    2^-51 |pos freq| rad, which turns a pair by that much of |a| + |b|; 2^-21 covers it while |pos freq| is
    below 2^29. The reduced angle is rounded to fp32 (at most pi 2^-24), sincospif is within 2 ulp, the cosine,
    the amplitude and the two products and their sum each round once: below 2^-21 of |a| + |b|. Then
    one rounding to dtype."""
    x = x.double().abs()
    n = x.shape[-1] // 2
    if layout == "half":
        s = x[..., :n] + x[..., n:]
        s = torch.cat([s, s], -1)
    else:
        s = (x[..., 0::2] + x[..., 1::2]).repeat_interleave(2, -1)
    slack = 2.0 ** -21 * abs(amplitude) * s
    if pos is not None:
        a = (pos.double().abs()[:, None, None] * freqs.double().abs()) * 2.0 ** -51 * abs(amplitude)
        slack = slack + s * (torch.cat([a, a], -1) if layout == "half" else a.repeat_interleave(2, -1))
    return slack + HALF[dtype] * (ref.abs() + slack) + 1e-38


def attention(q, rows, scale):
    """Forward of one query: q [H, 576], rows [n, 576] fp64 -> out [H, 512], lse [H]."""
    s = q @ rows.T * scale
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - lse[:, None]) @ rows[:, :512], lse


def backward(q, kv, slots, scale, out, lse, dout, dlse=None):
    """q, dout, out, lse, dlse as tensors of any type; kv [n, 576]; slots: [T, K] int64, -1 dead.
    Returns (dq, dkv, weights) in fp64 and a bound for each of them."""
    q, kv, out, dout = q.double(), kv.double(), out.double(), dout.double()
    T, H, _ = q.shape
    K = slots.shape[1]
    dq, bq = torch.zeros_like(q), torch.zeros_like(q)
    dkv, bk = torch.zeros((kv.shape[0], 576), dtype=torch.float64), torch.zeros((kv.shape[0], 576), dtype=torch.float64)
    w, bw = torch.zeros((T, K), dtype=torch.float64), torch.zeros((T, K), dtype=torch.float64)
    half = HALF[torch.bfloat16]
    # a sum of n fp32 terms, in any order and with truncated alignment: n 2^-23 of the sum of magnitudes
    g = 600 * 2.0 ** -23
    many = (128 + T * K) * 2.0 ** -23
    for t in range(T):
        live = torch.nonzero(slots[t] >= 0)[:, 0]
        at = slots[t][live]
        k = kv[at]
        v = k[:, :512]
        rows = torch.isfinite(lse[t])
        p = torch.where(rows[:, None], torch.exp(q[t] @ k.T * scale - lse[t].double()[:, None]), 0.0)
        delta = (dout[t] * out[t]).sum(-1)
        e_delta = g * (dout[t].abs() * out[t].abs()).sum(-1)
        if dlse is not None:
            delta = delta - dlse[t].double()
            e_delta = e_delta + 2.0 ** -23 * dlse[t].double().abs()
        gap = dout[t] @ v.T - delta[:, None]
        ds = p * gap * scale
        # the exponent: S in fp32, its scaling, lse and the subtraction; then the exponential (2^-22)
        e_s = g * (q[t].abs() @ k.abs().T) * abs(scale) + 2.0 ** -22 * (lse[t].double().abs().nan_to_num(0, 0, 0)[:, None] + 1)
        e_p = p * (e_s * 1.01 + 2.0 ** -21)
        e_gap = g * (dout[t].abs() @ v.abs().T) + e_delta[:, None] + 2.0 ** -22 * gap.abs()
        e_ds = abs(scale) * (e_p * gap.abs() + (p + e_p) * e_gap) * 1.01
        r_ds = e_ds + half * (ds.abs() + e_ds)  # with the operand's rounding to bf16
        r_p = e_p + half * (p + e_p)
        dq[t] = ds @ k
        bq[t] = r_ds @ k.abs() + g * (ds.abs() @ k.abs()) * max(1.0, len(at) / 600)
        d_row = ds.T @ q[t]
        b_row = r_ds.T @ q[t].abs() + many * (ds.abs().T @ q[t].abs())
        d_row[:, :512] += p.T @ dout[t]
        b_row[:, :512] += r_p.T @ dout[t].abs() + many * (p.T @ dout[t].abs())
        dkv.index_add_(0, at, d_row)
        bk.index_add_(0, at, b_row)
        w[t, live] = p.sum(0)
        bw[t, live] = e_p.sum(0) + H * 2.0 ** -23 * p.sum(0)
    bq = bq + half * (dq.abs() + bq) + 1e-30
    bk = bk + half * (dkv.abs() + bk) + 1e-30
    return (dq, dkv, w), (bq, bk, bw + 1e-30)


def distill(scores, lens, topk, teacher, kind, scope, temperature, row_weight=None):
    """(loss [T], dscores [T, N]) in fp64 and a bound for each (of the gradient before its rounding)."""
    T, N = scores.shape
    loss, grad = torch.zeros(T, dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64)
    b_loss, b_grad = torch.zeros(T, dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64)
    for t in range(T):
        n = N if lens is None else max(0, min(N, int(lens[t])))
        i = topk[t].long()
        ok = (i >= 0) & (i < n)
        i, w = i[ok], teacher[t][ok].double()
        if kind == "logits" and i.numel() and w.max() > -math.inf:
            w = torch.exp((w - w.max()) / temperature)
        elif kind == "logits":
            w = torch.zeros_like(w)
        x = scores[t].double() / temperature
        among = torch.arange(n) if scope == "candidates" else i
        if not i.numel() or w.sum() == 0 or not (x[among] > -math.inf).any():
            continue
        p = w / w.sum()
        lse = torch.logsumexp(x[among], 0)
        pos = p > 0
        lp, lq = torch.log(p[pos]), x[i][pos] - lse
        loss[t] = (p[pos] * (lp - lq)).sum()
        gw = (1.0 if row_weight is None else float(row_weight[t])) / temperature
        q = torch.exp(x[among] - lse)
        grad[t].index_add_(0, among, q * gw)
        grad[t].index_add_(0, i, -p * gw)
        # exponents: products and differences of magnitude m round to m 2^-22 together; sums of n terms run
        # in at most n / 512 + 64 sequential steps; exponentials 2^-21
        fin = x[among][torch.isfinite(x[among])]
        tv = teacher[t][ok].double()
        m = float(fin.abs().max()) * 2 + 4 + (float(tv[torch.isfinite(tv)].abs().max()) * 2 / temperature
                                             if kind == "logits" else 0.0)
        u = 2.0 ** -21 * m + (len(among) / 512 + len(i) / 512 + 64) * 2.0 ** -24 + 2.0 ** -20
        b_grad[t].index_add_(0, among, q * abs(gw) * u)
        b_grad[t].index_add_(0, i, p * abs(gw) * u)
        b_loss[t] = u * (1 + (p[pos] * (lp.abs() + lq.abs())).sum())
    return (loss, grad), (b_loss + 1e-30, b_grad + 1e-30)


def within(got, ref, bound, what=""):
    got, ref = got.detach().double().cpu(), ref.double()
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: finite in different places"
    off = (got - ref).abs()
    bad = (off > bound) & fine
    if bad.any():
        i = int(torch.where(fine, off / bound, torch.zeros_like(off)).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; at {i}: got "
                             f"{got.flatten()[i]:.9g}, want {ref.flatten()[i]:.9g}, bound {bound.flatten()[i]:.3g}")
