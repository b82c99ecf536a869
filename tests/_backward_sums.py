"""The attention's backward pass row by row: what the stated roundings leave of a row's 2-norm.

A row of dkv is the sum, over the lists that hold it and their heads, of dS q and P dout with P and dS
rounded to bf16; a row of dq the sum of dS K over a list. A rounding to bf16 is off by at most 2^-8 of the
value and, over many values, by 2^-8 / sqrt(3) of it in the mean square (evenly spread over the step), in a
direction of its own. So the mean square of a row's error is 2^-16 / 3 of the sum of its terms' squares, and
as much again of the row itself for the rounding of the output. The tolerance is three times its root, with
2^-13 of the terms for fp32 (sums of a few hundred terms, exponents of about ten). The bound of element by
element sums has to allow all roundings one sign, 2^-8 of the sum of magnitudes, in which one missing
addition of a hundred goes unseen; here it is 0.1 of the row's norm against 0.007."""

import math

import torch

ROUND = 2.0 ** -8 / math.sqrt(3)


def rows(q, kv, slots, scale, out, lse, dout, dlse=None, bf16_operands=False, skip=None):
    """dq [T, H, 576], dkv [n, 576] in fp64 and the tolerance of each row's 2-norm, [T, H] and [n].
    bf16_operands: with P and dS rounded as the kernel does. skip(t, entry) -> columns of dkv that the entry's
    contribution leaves out (a planted mistake)."""
    q, kv, out, dout = q.double(), kv.double(), out.double(), dout.double()
    T, H, _ = q.shape
    n = kv.shape[0]
    held = (lambda x: x.to(torch.bfloat16).double()) if bf16_operands else (lambda x: x)
    dq, sq = torch.zeros_like(q), torch.zeros((T, H), dtype=torch.float64)
    dkv, skv = torch.zeros((n, 576), dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    for t in range(T):
        live = torch.nonzero(slots[t] >= 0)[:, 0]
        at = slots[t][live].long()
        k = kv[at]
        ok = torch.isfinite(lse[t])[:, None]
        p = torch.where(ok, torch.exp(q[t] @ k.T * scale - lse[t].double()[:, None]), 0.0)
        delta = (dout[t] * out[t]).sum(-1) - (0.0 if dlse is None else dlse[t].double())
        ds = p * (dout[t] @ k[:, :512].T - delta[:, None]) * scale
        p, ds = held(p), held(ds)
        dq[t] = ds @ k
        sq[t] = (ds ** 2) @ (k ** 2).sum(-1)
        row = ds.T @ q[t]
        row[:, :512] += p.T @ dout[t]
        if skip is not None:
            for i, entry in enumerate(live.tolist()):
                row[i, skip(t, entry)] = 0
        dkv.index_add_(0, at, row)
        skv.index_add_(0, at, (ds ** 2).T @ (q[t] ** 2).sum(-1) + (p ** 2).T @ (dout[t] ** 2).sum(-1))
    if bf16_operands:
        dq, dkv = held(dq), held(dkv)
    tol = lambda x, s: 3 * ROUND * torch.sqrt(s + (x ** 2).sum(-1)) + 2.0 ** -13 * torch.sqrt(s)  # noqa: E731
    return dq, dkv, tol(dq, sq), tol(dkv, skv)


def off(got, ref, tol):
    """How many rows are off by more than their tolerance, and the largest ratio."""
    err = (got.double().cpu() - ref).norm(dim=-1)
    bad = err > tol + 1e-30
    return int(bad.sum()), float((err / (tol + 1e-30)).max())
