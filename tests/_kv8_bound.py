"""Attention over the paged 8-bit cache in 64 bits, with a bound on the error
that follows the sums as the kernel forms them.

The bound is relative to sum p |v| of each channel, not to the largest value of
a row: outputs of long rows average out to a small part of their values, and a
bound made of the largest value would let all of them be wrong."""
from __future__ import annotations

import torch

from tests import _kv8 as R

D = R.D


def stretch(lens, H, rows, fp32, sms):
    """32-token steps that one team of warps takes of the line of all rows' steps."""
    per = 4 if rows <= 4 else 8 if rows <= 8 or fp32 else 16
    teams = (8 if per == 16 else 12) // R.ceil_div(rows, per)
    total = sum(R.ceil_div(int(x), 32) for x in lens) * H
    return R.ceil_div(max(R.ceil_div(total, sms), 4), teams)


def dense(codes, scale, kind, ids, h, T):
    """The first T tokens of head h in pages ids, and their scales."""
    s = scale[ids, h].double()[:, None].expand(-1, codes.shape[2]).reshape(-1)[:T, None]
    return R.decode(codes[ids, h], kind).reshape(-1, D)[:T] * s, s


def head(qq, kk, vv, sv, m, fp32, S):
    """One kv head: queries qq [G, D] over the seen tokens (m) of kk, vv [T, D].
    Returns (out, tol), fp64.

    A score is 128 products added in 8 groups of 16 (16 where fp32 queries go in
    as two halves), each group adding at most 2^-22 of sum |q k|; the halves
    leave 2^-22 of it; the score's factor and its distance from the reference
    are rounded, 2^-24 each.  An error d of a score moves the output by
    sum p d |v| + |out| sum p d.
    A probability has 2^-22 from exp2 and 2^-22 from its two halves, the weights
    of the merges of teams and of CTAs 2^-22 each, above and below the fraction
    line; a half ends at 2^-25 where the row's largest p times value scale is
    2^4 or more.
    The running sums take 64 products between two flushes, each adding at most
    2^-22; a flush adds 2^-22; the sum of probabilities takes 4 adds a step."""
    kk, vv, sv = kk[m], vv[m], sv[m]
    x = qq @ kk.T / D ** 0.5
    p = torch.softmax(x, -1)
    out = p @ vv
    size = qq.abs() @ kk.abs().T / D ** 0.5
    d = (17 if fp32 else 8) * 2.0 ** -22 * size + 2.0 ** -24 * (4 * x.abs() + (x.amax(-1, keepdim=True) - x) + 8)
    tol = (p * d) @ vv.abs() + (p * d).sum(-1, keepdim=True) * out.abs()
    A = p @ vv.abs()
    tol += ((64 + S / 16 + 8) * 2.0 ** -22 + 32 * 2.0 ** -24) * A + (4 * S + 32) * 2.0 ** -24 * out.abs()
    tol += 2.0 ** -29 * (p * sv.T).amax(-1, keepdim=True) * (vv.abs() / sv.clamp(min=2.0 ** -126)).sum(0)
    return out, tol


def attention(q, k, v, ks, vs, kind, table, lens, n_new, G, page, sms=148):
    """As R.attention (NaN where a row is not written), with the bound above."""
    H, n_q = q.shape[1] // G, q.shape[2]
    fp32 = q.dtype == torch.float32
    S = stretch(lens, H, G * n_q, fp32, sms)
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for b in range(table.shape[0]):
        T, nn = int(lens[b]), int(n_new[b])
        ids = table[b, :R.ceil_div(T, page)].long()
        at = torch.arange(T, device=q.device)
        for h in range(H):
            kk, _ = dense(k, ks, kind, ids, h, T)
            vv, sv = dense(v, vs, kind, ids, h, T)
            for i in range(nn):
                m = at <= T - nn + i
                sl = (b, slice(h * G, (h + 1) * G), i)
                if not bool(m.any()):
                    out[sl] = 0.0
                    continue
                out[sl], tol[sl] = head(q[sl].double(), kk, vv, sv, m, fp32, S)
    return out, tol


def worst(got, ref, tol):
    """The largest error in units of its bound, over the places that are written."""
    w = ~torch.isnan(ref)
    return float(((got.double() - ref).abs()[w] / tol[w].clamp(min=1e-300)).max())
