"""Plain implementations of the paged 8-bit cache's rules, on the host and in
64 bits, for the tests: page tables and slot maps, the write in 8 bits, and
the attention over the pages."""
from __future__ import annotations

import numpy as np
import torch

D = 128
E4M3, I8 = 0, 1
TOP = {E4M3: 448.0, I8: 127.0}


def ceil_div(a, b):
    return -(-a // b)


def extend(lens, n_new, page, pool, taken, table, n_cap):
    """Returns (table, slots, lens_out, taken_out, ran_out); lists of ints."""
    table = [list(r) for r in table]
    slots = [[-1] * n_cap for _ in lens]
    out, ran_out, n_pages = [], False, len(pool)
    for b, (ln, nn) in enumerate(zip(lens, n_new)):
        got = ln
        for p in range(ceil_div(ln, page), ceil_div(ln + nn, page)):
            ran_out |= taken >= n_pages
            table[b][p] = pool[taken] if taken < n_pages else -1
            taken += taken < n_pages
        for j in range(nn):
            pg = table[b][(ln + j) // page]
            if pg >= 0:
                slots[b][j] = pg * page + (ln + j) % page
                got = ln + j + 1
        out.append(got)
    return table, slots, out, taken, ran_out


def trim(lens, keep, page, pool, taken, table):
    pool, back, out = list(pool), [], []
    for b, (ln, kp) in enumerate(zip(lens, keep)):
        kp = min(kp, ln)
        back += table[b][ceil_div(kp, page):ceil_div(ln, page)]
        out.append(kp)
    pool[taken - len(back):taken] = back
    return pool, out, taken - len(back)


def decode(codes: torch.Tensor, kind: int) -> torch.Tensor:
    """uint8 codes -> fp64 values (without the scale)."""
    return codes.view(torch.float8_e4m3fn if kind == E4M3 else torch.int8).double()


def _e4m3(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 number (fp64 in and out), ties to even, largest 448."""
    mag = np.minimum(np.abs(y), 448.0)
    _, e = np.frexp(mag)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.copysign(np.round(mag / step) * step, y)


def round8(y: np.ndarray, kind: int) -> np.ndarray:
    """Code values of y (already divided by the scale)."""
    if kind == E4M3:
        return _e4m3(y)
    return np.where(np.isnan(y), 0.0, np.clip(np.round(y), -127, 127))


def scale_of(a: float, kind: int) -> float:
    """The smallest 2^E, E in [-126, 120], with a <= TOP 2^E."""
    for e in range(-126, 121):
        if a <= TOP[kind] * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 120


def append(val, scale, x, slots, page, kind):
    """val [pages, H, page, D] code values and scale [pages, H], fp64, changed
    in place; x [B, H, n, D]."""
    x = x.astype(np.float64)
    for b, row in enumerate(slots):
        j = 0
        while j < len(row):
            if row[j] < 0 or row[j] >= val.shape[0] * page:
                j += 1
                continue
            pg, o = divmod(row[j], page)
            n = 1
            while j + n < len(row) and o + n < page and row[j + n] == row[j] + n:
                n += 1
            for h in range(val.shape[1]):
                y = x[b, h, j:j + n]
                fin = np.abs(y[np.isfinite(y)])
                s = scale_of(float(fin.max()) if fin.size else 0.0, kind)
                if o > 0 and scale[pg, h] >= s:
                    s = scale[pg, h]
                elif o > 0:
                    val[pg, h, :o] = round8(val[pg, h, :o] * (scale[pg, h] / s), kind)
                val[pg, h, o:o + n] = round8(y / s, kind)
                scale[pg, h] = s
            j += n


def attention(q, k, v, ks, vs, kind, table, lens, n_new, G, page):
    """fp64 attention on q's device; k, v uint8 codes.  Returns (out, tol):
    out is NaN where a row is not written, tol the error that fp32 arithmetic
    may make at each value.

    tol: a score is 128 products added in 8 groups of 16, each group adding at
    most 2^-22 of sum |q k| (a rounded or truncated partial sum and the group's
    own), and 4 more roundings of 2^-24 of the score; p then has twice that
    relative error with respect to its row's sum, plus 2^-21 for exp2, the
    split of p into two halves and the scales; the sums over tokens add
    2^-23 a step of 16 tokens, in numerator and denominator."""
    B, cap = table.shape
    H, n_q = q.shape[1] // G, q.shape[2]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for b in range(B):
        T, nn = int(lens[b]), int(n_new[b])
        ids = table[b, :ceil_div(T, page)].long()
        good = (ids >= 0) & (ids < k.shape[0])
        seen = good.repeat_interleave(page)[:T]
        ids = torch.where(good, ids, 0)
        for h in range(H):
            kk = (decode(k[ids, h], kind) * ks[ids, h].double()[:, None, None]).reshape(-1, D)[:T][seen]
            vv = (decode(v[ids, h], kind) * vs[ids, h].double()[:, None, None]).reshape(-1, D)[:T][seen]
            at = torch.arange(T, device=q.device)[seen]
            for i in range(nn):
                m = at <= T - nn + i
                sl = (b, slice(h * G, (h + 1) * G), i)
                if not bool(m.any()):
                    out[sl] = 0.0
                    continue
                qq = q[sl].double()
                x = qq @ kk[m].T / D ** 0.5
                out[sl] = torch.softmax(x, -1) @ vv[m]
                size = (qq.abs() @ kk[m].abs().T / D ** 0.5).amax()
                d = 8 * 2.0 ** -22 * size + 4 * 2.0 ** -24 * x.abs().amax()
                rel = 2 * d + 2.0 ** -21 + 2 * (int(m.sum()) / 16 + 16) * 2.0 ** -23
                assert float(rel) < 5e-3  # the bound says something
                tol[sl] = rel * vv[m].abs().amax()
    return out, tol
