"""The write into the paged 8-bit cache and the attention over it against the
plain rules in 64 bits (tests/_kv8.py).  Codes and scales are exact; attention
is held to the error that fp32 arithmetic may make (derived there)."""
import random

import numpy as np
import pytest
import torch

from channel_pruned_decode_b200 import (KV8Cache, spark_decode_attn_kv8, spark_device_status, spark_kv8_append,
                                        spark_pages_extend, spark_pages_trim, spark_snapkv_evict,
                                        spark_workspace_bytes, spark_workspace_bytes_kv8, workspace,
                                        SPARK_KV8_E4M3, SPARK_KV8_I8, SPARK_OP_SNAPKV)
from channel_pruned_decode_b200.binding import SPARK_ERR_ARG
from tests import _kv8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
KINDS = [SPARK_KV8_E4M3, SPARK_KV8_I8]
NAN_CODE = {SPARK_KV8_E4M3: 0x7f, SPARK_KV8_I8: 0x80}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _values(gen, shape, dtype=torch.float32, spread=0.5):
    x = torch.randn(shape, generator=gen, device=DEV)
    x *= torch.exp(spread * torch.randn(shape[:-2] + (1,) + shape[-1:], generator=gen, device=DEV))
    return x.to(dtype)


# ------------------------------------------------------------------ append
def _slot_map(rng, B, n_cap, page, new, off):
    """Slots of rows that start inside a page (off > 0) or on one; also the pages used."""
    need = [R.ceil_div(o + n, page) for o, n in zip(off, new)]
    ids = list(range(sum(need) + 3))
    rng.shuffle(ids)
    rows, at = [], 0
    for o, n, c in zip(off, new, need):
        pages = ids[at:at + c]
        at += c
        rows.append([pages[(o + j) // page] * page + (o + j) % page for j in range(n)] + [-1] * (n_cap - n))
    return rows, len(ids)


def _check_append(kc, val0, sc0, x, slots, kind, which):
    val, sc = val0.copy(), sc0.copy()
    R.append(val, sc, x, slots, kc.page, kind)
    got = R.decode(kc.k if which == "k" else kc.v, kind).cpu().numpy()
    got_sc = (kc.k_scale if which == "k" else kc.v_scale).double().cpu().numpy()
    assert np.array_equal(got_sc, sc)
    assert np.array_equal(got, val, equal_nan=True)


def _filled(n_pages, H, page, kind, seed):
    kc = KV8Cache.empty(n_pages, H, page, kind)
    g = _gen(seed)
    for c, s in ((kc.k, kc.k_scale), (kc.v, kc.v_scale)):
        y = (30 * torch.randn(c.shape, generator=g, device=DEV)).clamp(-120, 120)
        c.copy_((y.to(torch.float8_e4m3fn) if kind == SPARK_KV8_E4M3 else y.round().to(torch.int8)).view(torch.uint8))
        s.copy_(torch.exp2(torch.randint(-9, 1, s.shape, generator=g, device=DEV).float()))
    return kc


def _before(kc, kind):
    return [(R.decode(c, kind).cpu().numpy(), s.double().cpu().numpy()) for c, s in ((kc.k, kc.k_scale),
                                                                                     (kc.v, kc.v_scale))]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,B,H,n_cap", [(16, 1, 1, 1), (16, 5, 3, 40), (32, 3, 2, 77), (64, 2, 2, 200),
                                            (128, 3, 1, 300), (16, 9, 2, 1), (128, 4, 2, 3), (64, 1, 8, 64)])
def test_append(kind, dtype, page, B, H, n_cap):
    rng = random.Random(page + n_cap)
    new = [n_cap] + [rng.choice([0, 1, n_cap, rng.randint(0, n_cap)]) for _ in range(B - 1)]
    off = [rng.choice([0, page - 1, rng.randrange(page)]) for _ in range(B)]
    slots, n_pages = _slot_map(rng, B, n_cap, page, new, off)
    kc = _filled(n_pages, H, page, kind, 3)
    (k0, ks0), (v0, vs0) = _before(kc, kind)
    k_new, v_new = (_values(_gen(s), (B, H, n_cap, D), dtype) for s in (1, 2))
    ws = workspace(256)
    spark_kv8_append(k_new, v_new, i32(slots), kc, ws)
    assert spark_device_status(ws) == 0
    _check_append(kc, k0, ks0, k_new.double().cpu().numpy(), slots, kind, "k")
    _check_append(kc, v0, vs0, v_new.double().cpu().numpy(), slots, kind, "v")


@pytest.mark.parametrize("kind", KINDS)
def test_append_token_by_token(kind):
    """One token a call: the page's scale grows as larger values come, and older codes follow it."""
    H, page, n = 2, 16, 35
    kc = _filled(4, H, page, kind, 7)
    (k0, ks0), (v0, vs0) = _before(kc, kind)
    x = _values(_gen(8), (1, H, n, D)) * torch.exp2(torch.arange(n, device=DEV) % 9 - 4.0)[None, None, :, None]
    ws = workspace(256)
    for j in range(n):
        slot = [[(j // page + 1) * page + j % page]]
        y = x[:, :, j].contiguous()
        spark_kv8_append(y, -y, i32(slot), kc, ws)
        R.append(k0, ks0, y.double().cpu().numpy()[:, :, None], slot, page, kind)
        R.append(v0, vs0, -y.double().cpu().numpy()[:, :, None], slot, page, kind)
    assert spark_device_status(ws) == 0
    for c, s, val, sc in ((kc.k, kc.k_scale, k0, ks0), (kc.v, kc.v_scale, v0, vs0)):
        assert np.array_equal(s.double().cpu().numpy(), sc)
        assert np.array_equal(R.decode(c, kind).cpu().numpy(), val)


@pytest.mark.parametrize("kind", KINDS)
def test_append_special_values(kind):
    """Zeros, the type's extremes, subnormals, infinities and NaN; a page of nothing but zeros."""
    H, page = 1, 16
    x = torch.zeros((8, H, 4, D), device=DEV)
    x[0] = 0.0
    x[1, :, 0, :3] = torch.tensor([float("inf"), 1.0, -float("inf")])
    x[2, :, 1, 5] = float("nan")
    x[2, :, 2, 5] = -3.0
    x[3] = torch.finfo(torch.float32).max
    x[4] = 1e-42
    x[5, :, 0, 0] = 448.0
    x[5, :, 1, :6] = torch.tensor([447.9, 16.5, 17.0, 17.5, 2.0 ** -10, 3 * 2.0 ** -10])
    x[6, :, 0, :2] = torch.tensor([127.0, 63.5])
    x[7] = float("nan")
    slots = [[b * page + j for j in range(4)] for b in range(8)]
    kc = _filled(8, H, page, kind, 1)
    (k0, ks0), _ = _before(kc, kind)
    ws = workspace(256)
    spark_kv8_append(x, x, i32(slots), kc, ws)
    _check_append(kc, k0, ks0, x.double().cpu().numpy(), slots, kind, "k")


def test_append_skips_bad_slots():
    kc = _filled(3, 2, 16, SPARK_KV8_E4M3, 1)
    (k0, ks0), (v0, vs0) = _before(kc, SPARK_KV8_E4M3)
    slots = [[48, 49, 2 ** 30, -1, -5, 4, 5, -1], [2 ** 31 - 1, 16, 17, 19, 20, -1, 40, 48]]
    x = _values(_gen(1), (2, 2, 8, D))
    ws = workspace(256)
    spark_kv8_append(x, x, i32(slots), kc, ws)
    assert spark_device_status(ws) == SPARK_ERR_ARG
    # 16, 17 and 19, 20 are one page twice: its codes are not specified, all others are
    val, sc = k0.copy(), ks0.copy()
    R.append(val, sc, x.double().cpu().numpy(), slots, 16, SPARK_KV8_E4M3)
    got = R.decode(kc.k, SPARK_KV8_E4M3).cpu().numpy()
    assert np.array_equal(got[[0, 2]], val[[0, 2]])


def test_append_far_pages():
    """Codes beyond 4 GB of the cache."""
    H, page, n_pages = 8, 128, 40000  # 5.2 GB of keys
    kc = KV8Cache.empty(n_pages, H, page)
    ids = [0, 39999, 32768, 16384]
    x = _values(_gen(1), (4, H, 10, D), torch.bfloat16)
    slots = [[i * page + 118 + j for j in range(10)] for i in ids]
    kc.k_scale[ids] = 2.0 ** -20
    kc.v_scale[ids] = 2.0 ** -20
    for i in ids:
        kc.k[i] = 0
        kc.v[i] = 0
    ws = workspace(256)
    spark_kv8_append(x, x, i32(slots), kc, ws)
    val, sc = np.zeros((4, H, page, D)), np.full((4, H), 2.0 ** -20)
    R.append(val, sc, x.double().cpu().numpy(), [[i * page + s % page for s in r] for i, r in enumerate(slots)], page,
             SPARK_KV8_E4M3)
    assert np.array_equal(R.decode(kc.k[ids], SPARK_KV8_E4M3).cpu().numpy(), val)
    assert np.array_equal(kc.v_scale[ids].double().cpu().numpy(), sc)
    lens = i32([128] * 4)
    q = _values(_gen(2), (4, H, 1, D))
    out, ws = torch.zeros_like(q), workspace(spark_workspace_bytes_kv8(4, H, 1, 1))
    spark_decode_attn_kv8(q, kc, i32([[i] for i in ids]), lens, 1, out, ws)
    ref, tol = R.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, 0, i32([[i] for i in ids]), lens, [1] * 4, 1, page)
    assert bool(((out - ref).abs() <= tol).all())


# --------------------------------------------------------------- attention
def _context(lens, H, page, kind, seed, spread=0.5, cap=None):
    """A cache whose rows hold lens tokens; every code, scale and table entry
    that no token owns is filled with what must not be used."""
    rng = random.Random(seed)
    need = [R.ceil_div(x, page) for x in lens]
    cap = max(1, max(need)) if cap is None else cap
    ids = list(range(sum(need) + 2))
    rng.shuffle(ids)
    kc = KV8Cache.empty(len(ids), H, page, kind)
    for t in (kc.k, kc.v):
        t.fill_(NAN_CODE[kind])
    for s in (kc.k_scale, kc.v_scale):
        s.fill_(float("nan"))
    table, at = torch.full((len(lens), cap), 2 ** 30, dtype=torch.int32, device=DEV), 0
    slots = torch.full((len(lens), max(1, max(lens))), -1, dtype=torch.int32, device=DEV)
    for b, (x, n) in enumerate(zip(lens, need)):
        mine = i32(ids[at:at + n])
        at += n
        table[b, :n] = mine
        t = torch.arange(x, device=DEV)
        slots[b, :x] = mine[t // page] * page + (t % page).int() if x else slots[b, :0]
    g = _gen(seed)
    k, v = (_values(g, (len(lens), H, slots.shape[1], D), spread=spread) for _ in range(2))
    ws = workspace(256)
    spark_kv8_append(k, v, slots, kc, ws)
    assert spark_device_status(ws) == 0
    return kc, table


def _attend(q, kc, table, lens, G, n_new=None, ws=None):
    B, Hq, n_q, _ = q.shape
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device=DEV)
    if ws is None:
        ws = workspace(spark_workspace_bytes_kv8(B, Hq // G, G, n_q))
    spark_decode_attn_kv8(q, kc, table, i32(lens), G, out, ws, n_new=None if n_new is None else i32(n_new))
    return out, ws


def _check_attn(lens, H, G, n_q, page, kind, dtype, seed=0, n_new=None, spread=0.5, cap=None):
    kc, table = _context(lens, H, page, kind, seed, spread, cap)
    q = _values(_gen(seed + 1), (len(lens), H * G, n_q, D), dtype, spread)
    out, ws = _attend(q, kc, table, lens, G, n_new)
    assert spark_device_status(ws) == 0
    nn = [n_q] * len(lens) if n_new is None else n_new
    ref, tol = R.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, kind, table, lens, nn, G, page)
    unseen = torch.isnan(ref)  # rows of queries past n_new: left as they were
    assert torch.equal(torch.isnan(out), unseen)
    err = torch.where(unseen, 0.0, (out.double() - ref).abs())
    assert bool((err <= torch.where(unseen, 1.0, tol)).all()), float((err / tol.clamp(min=1e-30)).max())
    again, _ = _attend(q, kc, table, lens, G, n_new)
    assert torch.equal(torch.nan_to_num(again, 7.0), torch.nan_to_num(out, 7.0))  # the same bits


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attn_lengths(kind, dtype, page):
    """Lengths around pages and tiles, empty rows among them."""
    _check_attn([0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 0], 2, 4, 1, page, kind, dtype)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 32, 33, 48, 64])
def test_attn_groups(kind, G):
    _check_attn([200, 77], 2, G, 1, 16, kind, torch.bfloat16)
    _check_attn([200, 77], 2, G, 1, 64, kind, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,n_q", [(1, 2), (4, 4), (4, 2), (2, 5), (8, 8), (3, 7), (1, 64), (5, 3), (4, 16)])
def test_attn_several_new_tokens(dtype, G, n_q):
    """Each query sees the tokens up to its own; rows shorter than n_q and with fewer queries than n_q."""
    lens = [1, 2, n_q, n_q + 1, 40, 300, 33, 0]
    _check_attn(lens, 2, G, n_q, 16, SPARK_KV8_E4M3, dtype)
    _check_attn(lens, 1, G, n_q, 32, SPARK_KV8_I8, dtype, n_new=[1, 0, n_q, n_q, n_q // 2, 1, n_q, n_q])


@pytest.mark.parametrize("H,lens", [(8, [5000]), (1, [20011]), (8, [3, 9000, 1, 0, 2500, 64, 64, 1111]),
                                    (3, [700] * 40), (2, [1] * 300), (8, [100] * 130)])
def test_attn_long_and_many(H, lens):
    _check_attn(lens, H, 4, 1, 16, SPARK_KV8_E4M3, torch.bfloat16)
    _check_attn(lens, H, 8, 2, 64, SPARK_KV8_I8, torch.float32)


@pytest.mark.parametrize("n_q", [1, 3])
def test_attn_long_rows_without_queries(n_q):
    """Rows that many teams share, some of them without a query: left as they were."""
    lens = [9000, 4000, 20000, 700, 5000]
    _check_attn(lens, 2, 4, n_q, 16, SPARK_KV8_E4M3, torch.bfloat16, n_new=[0, n_q, 0, 0, 1])
    _check_attn(lens, 1, 13, n_q, 32, SPARK_KV8_I8, torch.float32, n_new=[0, n_q, 0, 0, 1])


def test_attn_very_long():
    _check_attn([131072, 65537], 2, 4, 1, 32, SPARK_KV8_E4M3, torch.bfloat16)


@pytest.mark.parametrize("G,n_q,kind", [(2, 1, SPARK_KV8_I8), (8, 1, SPARK_KV8_E4M3), (8, 2, SPARK_KV8_I8),
                                        (16, 2, SPARK_KV8_E4M3)])
def test_attn_long_stretches(G, n_q, kind):
    """More steps to a warp than its running sums stay in registers for."""
    _check_attn([150000, 150001, 7], 8, G, n_q, 128, kind, torch.bfloat16)


def test_attn_many_rows():
    """More rows than a CTA has threads; most of them without tokens."""
    lens = [0] * 3000
    for i, x in ((0, 5), (1, 40), (700, 129), (2047, 1), (2999, 333)):
        lens[i] = x
    _check_attn(lens, 1, 4, 1, 16, SPARK_KV8_E4M3, torch.float32)


@pytest.mark.parametrize("lens", [[0, 0], [5, 0]])
def test_attn_without_any_page(lens):
    """A pool without pages, tables without places: nothing is seen, and rows that claim tokens are flagged."""
    kc = KV8Cache.empty(0, 2, 16)
    q = _values(_gen(5), (2, 8, 1, D))
    out, ws = _attend(q, kc, torch.zeros((2, 0), dtype=torch.int32, device=DEV), lens, 4)
    assert float(out.abs().max()) == 0.0
    assert spark_device_status(ws) == (SPARK_ERR_ARG if any(lens) else 0)
    out, ws = _attend(q, kc, torch.zeros((2, 3), dtype=torch.int32, device=DEV), lens, 4)
    assert float(out.abs().max()) == 0.0
    assert spark_device_status(ws) == (SPARK_ERR_ARG if any(lens) else 0)


def test_attn_rows_that_share_pages():
    """Rows may list the same pages (a common prefix), each with an end of its own."""
    kc, table = _context([200, 200], 2, 16, SPARK_KV8_I8, 4)
    table[1, :6] = table[0, :6]
    lens = [200, 130]
    q = _values(_gen(5), (2, 8, 1, D), torch.bfloat16)
    out, ws = _attend(q, kc, table, lens, 4)
    ref, tol = R.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, SPARK_KV8_I8, table, lens, [1, 1], 4, 16)
    assert bool(((out - ref).abs() <= tol).all())


def test_attn_workspace_serves_calls_of_other_shapes():
    """One workspace, sized for the largest call, through calls of different shapes in any order."""
    shapes = [([3000, 10], 8, 4, 1), ([77] * 30, 2, 8, 2), ([20000], 1, 16, 4), ([1, 2, 3], 4, 1, 1)]
    ws = workspace(max(spark_workspace_bytes_kv8(len(x), H, G, n) for x, H, G, n in shapes))
    rng = random.Random(3)
    ctx = [(_context(x, H, 16, SPARK_KV8_E4M3, i), _values(_gen(i), (len(x), H * G, n, D), torch.bfloat16), x, G)
           for i, (x, H, G, n) in enumerate(shapes)]
    alone = [_attend(q, kc, t, x, G)[0] for (kc, t), q, x, G in ctx]
    for _ in range(20):
        i = rng.randrange(len(ctx))
        (kc, t), q, x, G = ctx[i]
        out, _ = _attend(q, kc, t, x, G, ws=ws)
        assert torch.equal(torch.nan_to_num(out, 7.0), torch.nan_to_num(alone[i], 7.0))
    assert spark_device_status(ws) == 0


def test_attn_peaked_scores():
    """Scores of some hundreds: the softmax is one token, or nearly."""
    _check_attn([300, 1000], 2, 4, 1, 16, SPARK_KV8_E4M3, torch.float32, spread=1.5)


@pytest.mark.parametrize("kind", KINDS)
def test_attn_pages_of_very_different_size(kind):
    """Value scales from 2^-20 to 2^20 and a page of zeros in one row."""
    page, lens = 16, [16 * 12 + 5]
    kc, table = _context(lens, 2, page, kind, 4)
    for i, p in enumerate(table[0].tolist()):
        kc.v_scale[p] *= 2.0 ** (20 - 4 * (i * 5 % 11)) if i != 3 else 0.0
    q = _values(_gen(5), (1, 8, 1, D))
    out, ws = _attend(q, kc, table, lens, 4)
    ref, tol = R.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, kind, table, lens, [1], 4, page)
    assert bool(((out - ref).abs() <= tol).all())


@pytest.mark.parametrize("kind", KINDS)
def test_attn_scales_that_are_no_powers_of_two(kind):
    """A cache that another program filled."""
    lens, page = [100, 35], 32
    kc, table = _context(lens, 2, page, kind, 4)
    kc.k_scale.mul_(1.37)
    kc.v_scale.mul_(0.81)
    q = _values(_gen(5), (2, 8, 1, D), torch.bfloat16)
    out, ws = _attend(q, kc, table, lens, 4)
    ref, tol = R.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, kind, table, lens, [1, 1], 4, page)
    assert bool(((out - ref).abs() <= tol).all())


@pytest.mark.parametrize("scale", [1e-30, 1e30, 0.0])
def test_attn_query_magnitudes(scale):
    """Queries far from 1 (keys as far the other way) and queries of zeros."""
    lens, page = [90], 16
    kc, table = _context(lens, 2, page, SPARK_KV8_E4M3, 4)
    q = _values(_gen(5), (1, 8, 1, D)) * scale
    if scale:
        kc.k_scale.div_(scale)
    out, ws = _attend(q, kc, table, lens, 4)
    ref, tol = R.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, 0, table, lens, [1], 4, page)
    assert bool(((out - ref).abs() <= tol + 1e-6).all())


def test_attn_nan_reaches_only_those_who_see_it():
    """A NaN key or value in a seen place makes its head's output NaN, no other's."""
    lens, page = [40, 40], 16
    kc, table = _context(lens, 2, page, SPARK_KV8_E4M3, 4)
    q = _values(_gen(5), (2, 8, 1, D))
    clean, _ = _attend(q, kc, table, lens, 4)
    kc.k[table[0, 1], 1, 3, 7] = 0x7f
    kc.v[table[1, 0], 0, 2, 9] = 0x7f
    out, _ = _attend(q, kc, table, lens, 4)
    assert bool(out[0, 4:].isnan().all()) and torch.equal(out[0, :4], clean[0, :4])
    assert bool(out[1, :4, :, 9].isnan().all()) and torch.equal(out[1, 4:], clean[1, 4:])
    assert torch.equal(out[1, :4, :, :9], clean[1, :4, :, :9])
    assert torch.equal(out[1, :4, :, 10:], clean[1, :4, :, 10:])


@pytest.mark.parametrize("G,n_q", [(2, 2), (4, 4), (3, 20), (8, 8)])
def test_attn_nan_in_a_place_that_some_queries_do_not_see(G, n_q):
    lens, page = [100 + n_q], 16
    kc, table = _context(lens, 2, page, SPARK_KV8_E4M3, 4)
    q = _values(_gen(5), (1, 2 * G, n_q, D), torch.bfloat16)
    clean, _ = _attend(q, kc, table, lens, G)
    first = {}  # channel -> first query that sees the NaN
    for i, ch in ((0, 3), (1, 64), (n_q - 1, 127)):
        t = lens[0] - n_q + i
        kc.v[table[0, t // page], 0, t % page, ch] = 0xff if i else 0x7f
        first[ch] = i
    t = lens[0] - n_q + n_q // 2
    kc.k[table[0, t // page], 1, t % page, 5] = 0x7f
    out, _ = _attend(q, kc, table, lens, G)
    for i in range(n_q):
        nan = [ch for ch, f in first.items() if f <= i]
        rest = [ch for ch in range(D) if ch not in nan]
        assert bool(out[0, :G, i][:, nan].isnan().all())
        assert torch.equal(out[0, :G, i][:, rest], clean[0, :G, i][:, rest])
        if i < n_q // 2:
            assert torch.equal(out[0, G:, i], clean[0, G:, i])
        else:
            assert bool(out[0, G:, i].isnan().all())


def test_attn_flags_bad_lengths_and_pages():
    kc, table = _context([112, 100], 2, 16, SPARK_KV8_E4M3, 4)
    q = _values(_gen(5), (2, 8, 2, D))
    n_pages = kc.n_pages
    for lens, nn, edit in (([113, 20], [2, 2], None), ([-1, 20], [2, 2], None), ([50, 20], [3, 2], None),
                           ([50, 20], [-1, 2], None), ([50, 20], [2, 2], (0, 1, n_pages)),
                           ([50, 20], [2, 2], (0, 1, -1)), ([50, 20], [2, 2], (1, 0, 2 ** 31 - 1))):
        t = table.clone()
        if edit:
            t[edit[0], edit[1]] = edit[2]
        out, ws = _attend(q, kc, t, lens, 4, nn)
        assert spark_device_status(ws, clear=True) == SPARK_ERR_ARG, (lens, nn, edit)
        cl = [min(max(x, 0), 7 * 16) for x in lens]
        cn = [min(max(x, 0), 2) for x in nn]
        ref, tol = R.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, 0, t, cl, cn, 4, 16)
        unseen = torch.isnan(ref)
        assert torch.equal(torch.isnan(out), unseen)
        assert bool((torch.where(unseen, 0.0, (out - ref).abs()) <= torch.where(unseen, 1.0, tol)).all())


def test_attn_row_without_any_good_page():
    kc, table = _context([40, 40], 1, 16, SPARK_KV8_E4M3, 4)
    table[0] = -1
    q = _values(_gen(5), (2, 4, 1, D))
    out, ws = _attend(q, kc, table, [40, 40], 4)
    assert spark_device_status(ws) == SPARK_ERR_ARG
    assert float(out[0].abs().max()) == 0.0 and bool(out[1].abs().max() > 0)


# ------------------------------------------------------------ used together
class _Serve:
    """A serving loop's state, and the plain rules beside it."""

    def __init__(self, B, H, G, page, kind, n_pages, cap, n_cap, dtype):
        self.B, self.H, self.G, self.page, self.kind, self.n_cap, self.dtype = B, H, G, page, kind, n_cap, dtype
        self.lens, self.taken, self.ws = i32([0] * B), i32([0]), workspace(256)
        self.table = torch.full((B, cap), -1, dtype=torch.int32, device=DEV)
        self.pool = i32(random.Random(1).sample(range(n_pages), n_pages))
        self.slots = torch.zeros((B, n_cap), dtype=torch.int32, device=DEV)
        self.kc = KV8Cache.empty(n_pages, H, page, kind)
        self.out = torch.zeros((B, H * G, n_cap, D), device=DEV)
        self.wsa = workspace(spark_workspace_bytes_kv8(B, H, G, n_cap))

    def step(self, n_new, k, v, q, stream=None):
        spark_pages_extend(self.lens, n_new, self.page, self.pool, self.taken, self.table, self.slots, self.lens,
                           self.taken, self.ws, stream)
        spark_kv8_append(k, v, self.slots, self.kc, self.ws, stream)
        spark_decode_attn_kv8(q, self.kc, self.table, self.lens, self.G, self.out, self.wsa, n_new=n_new,
                              stream=stream)

    def trim(self, keep, stream=None):
        spark_pages_trim(self.lens, keep, self.page, self.pool, self.taken, self.table, self.lens, self.taken,
                         self.ws, stream)

    def status(self):
        return spark_device_status(self.ws), spark_device_status(self.wsa)


def _inputs(seed, B, H, G, n, dtype):
    g = _gen(seed)
    return [_values(g, (B, h, n, D), dtype) for h in (H, H, H * G)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 64])
def test_serving_steps(kind, page):
    """Verify steps of up to 4 tokens, of which some are taken back; requests
    end and others start in their pages.  The attention of every step is
    compared with a dense history that the test keeps itself."""
    B, H, G, n = 4, 2, 4, 4
    s = _Serve(B, H, G, page, kind, 40, 8, n, torch.bfloat16)
    rng = random.Random(page)
    hist = [[] for _ in range(B)]  # (k, v) of each row's tokens, as given
    for it in range(25):
        k, v, q = _inputs(100 + it, B, H, G, n, torch.bfloat16)
        nn = [rng.randint(0, n) for _ in range(B)]
        s.step(i32(nn), k, v, q)
        for b in range(B):
            hist[b] += [(k[b, :, j], v[b, :, j]) for j in range(nn[b])]
        assert s.lens.tolist() == [len(h) for h in hist]
        ref, tol = R.attention(q, s.kc.k, s.kc.v, s.kc.k_scale, s.kc.v_scale, kind, s.table, s.lens.tolist(), nn, G,
                               page)
        unseen = torch.isnan(ref)
        assert bool((torch.where(unseen, 0.0, (s.out - ref).abs()) <= torch.where(unseen, 1.0, tol)).all())
        # the cache holds what went in: within a step of its scale (two
        # roundings where a page's scale grew, and at most half a step more)
        for b in range(B):
            for t in range(0, len(hist[b]), 5):
                pg = int(s.table[b, t // page])
                sc = s.kc.k_scale[pg].double()[:, None]
                got = R.decode(s.kc.k[pg, :, t % page], kind) * sc
                want = hist[b][t][0].double()
                # e4m3: half a step is 2^-4 of the value, or 2^-10 of the scale below 2^-6
                room = sc * 2 if kind == SPARK_KV8_I8 else (want.abs() * 2.0 ** -3).clamp(min=2.0 ** -8 * sc)
                assert bool(((got - want).abs() <= room).all())
        keep = [max(0, x - rng.randint(0, 2)) if rng.random() < 0.8 else 0 for x in s.lens.tolist()]
        s.trim(i32(keep))
        hist = [h[:x] for h, x in zip(hist, keep)]
        assert s.status() == (0, 0)
    held = [p for row, x in zip(s.table.tolist(), s.lens.tolist()) for p in row[:R.ceil_div(x, page)]]
    assert sorted(held + s.pool.tolist()[s.taken.item():]) == list(range(40))


def test_step_replayed_from_a_graph():
    """One captured step, replayed: the lengths advance on the GPU and the
    outputs are those of the same calls made one by one, bit for bit."""
    B, H, G, steps = 3, 2, 4, 40
    eager, graphed = (_Serve(B, H, G, 16, SPARK_KV8_E4M3, 30, 4, 1, torch.bfloat16) for _ in range(2))
    one = i32([1, 1, 0])
    inputs = [_inputs(200 + i, B, H, G, 1, torch.bfloat16) for i in range(steps)]
    k, v, q = (x.clone() for x in inputs[0])
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            graphed.step(one, k, v, q)
    torch.cuda.synchronize()
    for i in range(steps):
        for a, x in zip((k, v, q), inputs[i]):
            a.copy_(x)
        eager.step(one, *inputs[i])
        g.replay()
        assert torch.equal(eager.out, graphed.out)
    assert eager.lens.tolist() == graphed.lens.tolist() == [steps, steps, 0]
    assert torch.equal(eager.slots, graphed.slots)
    assert eager.status() == graphed.status() == (0, 0)
    del g


@pytest.mark.parametrize("B,H,G,n", [(3, 2, 4, 1), (8, 8, 4, 3), (1, 8, 4, 4)])
def test_steps_behind_one_another(B, H, G, n):
    """Steps without anything between them (each kernel is set up while the one
    ahead of it ends) give what the same steps give when each call is waited for."""
    rng = random.Random(B)
    steps = 40
    ins = [_inputs(400 + i, B, H, G, n, torch.bfloat16) for i in range(steps)]
    nn = [i32([rng.randint(0, n) for _ in range(B)]) for _ in range(steps)]
    keep = [i32([rng.choice([10 ** 6, 10 ** 6, rng.randint(0, 60)]) for _ in range(B)]) for _ in range(steps)]
    fast, slow = (_Serve(B, H, G, 16, SPARK_KV8_E4M3, 400, 40, n, torch.bfloat16) for _ in range(2))
    torch.cuda.synchronize()
    for i in range(steps):
        fast.step(nn[i], *ins[i])
        fast.trim(keep[i])
    torch.cuda.synchronize()
    for i in range(steps):
        k, v, q = ins[i]
        spark_pages_extend(slow.lens, nn[i], 16, slow.pool, slow.taken, slow.table, slow.slots, slow.lens, slow.taken,
                           slow.ws)
        torch.cuda.synchronize()
        spark_kv8_append(k, v, slow.slots, slow.kc, slow.ws)
        torch.cuda.synchronize()
        spark_decode_attn_kv8(q, slow.kc, slow.table, slow.lens, G, slow.out, slow.wsa, n_new=nn[i])
        torch.cuda.synchronize()
        slow.trim(keep[i])
        torch.cuda.synchronize()
    for name in ("out", "lens", "taken", "pool", "slots"):
        assert torch.equal(getattr(fast, name), getattr(slow, name)), name
    assert fast.status() == slow.status() == (0, 0)


def test_two_streams_with_workspaces_of_their_own():
    """Two serving loops on two streams at once do not disturb each other."""
    shape = (5, 4, 4, 16, SPARK_KV8_I8, 100, 8, 4, torch.bfloat16)
    alone, side = _Serve(*shape), [_Serve(*shape) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    nn = i32([4, 3, 0, 1, 4])
    ins = [_inputs(300 + i, 5, 4, 4, 4, torch.bfloat16) for i in range(10)]
    torch.cuda.synchronize()
    for x in ins:
        for s, st in zip(side, streams):
            s.step(nn, *x, stream=st)
    for x in ins:
        alone.step(nn, *x)
    torch.cuda.synchronize()
    for s in side:
        assert torch.equal(s.out, alone.out) and torch.equal(s.kc.k_scale[s.table.clamp(min=0)[0, 0]],
                                                             alone.kc.k_scale[alone.table.clamp(min=0)[0, 0]])
        assert s.status() == (0, 0)


def test_evicted_prompt_goes_into_the_pages():
    """What spark_snapkv_evict keeps ([B][Hkv][keep][D]) is written as it
    comes, and decoded."""
    B, H, G, S, W, keep = 2, 2, 4, 700, 16, 100
    g = _gen(9)
    k, v = (_values(g, (B, H, S, D), torch.bfloat16) for _ in range(2))
    q_obs = _values(g, (B, H * G, W, D), torch.bfloat16)
    ko, vo = (torch.empty((B, H, keep, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    idx = torch.empty((B, H, keep), dtype=torch.int32, device=DEV)
    ws = workspace(spark_workspace_bytes(SPARK_OP_SNAPKV, B, H, G, S, D, 0, 0))
    spark_snapkv_evict(k, v, q_obs, G, W, keep, 7, ko, vo, idx, ws)
    s = _Serve(B, H, G, 32, SPARK_KV8_I8, 10, 5, 1, torch.bfloat16)
    slots = torch.zeros((B, keep), dtype=torch.int32, device=DEV)
    spark_pages_extend(s.lens, i32([keep] * B), 32, s.pool, s.taken, s.table, slots, s.lens, s.taken, s.ws)
    spark_kv8_append(ko, vo, slots, s.kc, s.ws)
    kn, vn, q = _inputs(10, B, H, G, 1, torch.bfloat16)
    s.step(i32([1, 1]), kn, vn, q)
    assert s.status() == (0, 0) and s.lens.tolist() == [keep + 1] * B
    # the dense attention over the values as they were, to int8's error: a
    # score's is at most scale/2 * sum |q| / sqrt(D), a value's scale/2
    kd, vd = torch.cat([ko, kn], 2).double(), torch.cat([vo, vn], 2).double()
    for b in range(B):
        for h in range(H):
            sk, sv = (float(x[s.table[b, :4].long(), h].max()) for x in (s.kc.k_scale, s.kc.v_scale))
            qq = q[b, h * G:(h + 1) * G, 0].double()
            ref = torch.softmax(qq @ kd[b, h].T / D ** 0.5, -1) @ vd[b, h]
            dx = sk / 2 * qq.abs().sum(-1, keepdim=True) / D ** 0.5
            room = (torch.exp(2 * dx) - 1) * vd[b, h].abs().max() + sv / 2 + 1e-4
            assert bool(((s.out[b, h * G:(h + 1) * G, 0] - ref).abs() <= room).all())
