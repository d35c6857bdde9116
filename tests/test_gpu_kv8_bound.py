"""Attention over the paged 8-bit cache held to the bound of
tests/_kv8_bound.py, which is relative to sum p |v| of each channel."""
import math
import random

import pytest
import torch

from channel_pruned_decode_b200 import (KV8Cache, spark_decode_attn_kv8, spark_device_status, spark_kv8_append,
                                        spark_workspace_bytes_kv8, workspace, SPARK_KV8_E4M3, SPARK_KV8_I8)
from tests import _kv8 as R
from tests import _kv8_bound as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
KINDS = [SPARK_KV8_E4M3, SPARK_KV8_I8]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _values(gen, shape, spread=0.5):
    x = torch.randn(shape, generator=gen, device=DEV)
    return x * torch.exp(spread * torch.randn(shape[:-2] + (1, D), generator=gen, device=DEV))


def _cache(lens, H, page, kind, seed, mean=0.0):
    """Rows of lens tokens in shuffled pages; values with the given mean."""
    need = [R.ceil_div(x, page) for x in lens]
    ids = list(range(sum(need)))
    random.Random(seed).shuffle(ids)
    kc = KV8Cache.empty(len(ids), H, page, kind)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    ws, g, at = workspace(256), _gen(seed), 0
    for b, (x, n) in enumerate(zip(lens, need)):
        table[b, :n] = i32(ids[at:at + n])
        at += n
        t = torch.arange(x, device=DEV)
        slots = (table[b, t // page].long() * page + t % page).int()[None].contiguous()
        k, v = (_values(g, (1, H, x, D)) for _ in range(2))
        spark_kv8_append(k, v + mean, slots, kc, ws)
    assert spark_device_status(ws) == 0
    return kc, table


def _worst(q, kc, table, lens, G, n_new=None, status=0):
    B, Hq, n_q, _ = q.shape
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device=DEV)
    ws = workspace(spark_workspace_bytes_kv8(B, Hq // G, G, n_q))
    spark_decode_attn_kv8(q, kc, table, i32(lens), G, out, ws, n_new=None if n_new is None else i32(n_new))
    assert spark_device_status(ws) == status
    nn = [n_q] * B if n_new is None else n_new
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ref, tol = A.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, kc.type, table, lens, nn, G, kc.page, sms)
    assert torch.equal(torch.isnan(out), torch.isnan(ref))
    return A.worst(out, ref, tol)


@pytest.mark.parametrize("mean", [0.0, 1.0])
@pytest.mark.parametrize("lens,H,G,n_q,page,kind,dtype", [
    ([131072, 65537], 2, 4, 1, 32, SPARK_KV8_E4M3, torch.bfloat16),
    ([131072], 8, 4, 1, 16, SPARK_KV8_I8, torch.float32),
    ([150000, 150001, 7], 8, 2, 1, 128, SPARK_KV8_I8, torch.bfloat16),
    ([150000, 150001, 7], 8, 8, 1, 128, SPARK_KV8_E4M3, torch.bfloat16),
    ([150000, 150001, 7], 8, 8, 2, 128, SPARK_KV8_I8, torch.bfloat16),
    ([150000, 150001, 7], 8, 16, 2, 128, SPARK_KV8_E4M3, torch.bfloat16),
    ([20011, 20012], 8, 8, 8, 64, SPARK_KV8_E4M3, torch.float32),
    ([20011, 30000], 4, 13, 4, 32, SPARK_KV8_I8, torch.bfloat16)])
def test_long_rows(lens, H, G, n_q, page, kind, dtype, mean):
    kc, table = _cache(lens, H, page, kind, 3, mean)
    q = _values(_gen(4), (len(lens), H * G, n_q, D)).to(dtype)
    assert _worst(q, kc, table, lens, G) <= 1


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G,n_q,page", [(1, 1, 16), (4, 1, 32), (8, 1, 64), (4, 4, 16), (16, 2, 128), (8, 8, 16)])
def test_short_rows(kind, dtype, G, n_q, page):
    lens = [n_q, 15 + n_q, 100, 515, 2049]
    kc, table = _cache(lens, 2, page, kind, 5)
    q = _values(_gen(6), (len(lens), 2 * G, n_q, D)).to(dtype)
    assert _worst(q, kc, table, lens, G) <= 1


def _pages_of_size(T, page, kind, dtype, G, n_q, bits):
    """One row in which page i's scores lie bits[i][0] powers of two from zero
    and its values bits[i][1] from 1.  Returns the cache, its table and q."""
    g = _gen(7)
    k, v, q = _values(g, (1, 2, T, D)), _values(g, (1, 2, T, D)), _values(g, (1, 2 * G, n_q, D)).to(dtype)
    at = torch.arange(T, device=DEV) // page
    score, size = (torch.tensor([b[i] for b in bits], device=DEV, dtype=torch.float32)[at] for i in (0, 1))
    q[..., 0] = 4.0
    k[..., 0] = score * (0.6931471805599453 * D ** 0.5 / 4.0)
    v *= torch.exp2(size)[:, None]
    kc = KV8Cache.empty(len(bits), 2, page, kind)
    table = i32([random.Random(T).sample(range(len(bits)), len(bits))])
    t = torch.arange(T, device=DEV)
    ws = workspace(256)
    spark_kv8_append(k, v, (table[0, t // page].long() * page + t % page).int()[None].contiguous(), kc, ws)
    assert spark_device_status(ws) == 0
    return kc, table, q


def _worst_of_copies(q, kc, table, T, G, copies):
    """One row `copies` times over the same pages: the teams of warps then take
    stretches of many steps, which begin and end anywhere in the row."""
    n_q = q.shape[2]
    out = torch.full((copies,) + q.shape[1:], float("nan"), dtype=torch.float32, device=DEV)
    ws = workspace(spark_workspace_bytes_kv8(copies, q.shape[1] // G, G, n_q))
    spark_decode_attn_kv8(q.expand(copies, -1, -1, -1).contiguous(), kc, table.expand(copies, -1).contiguous(),
                          i32([T] * copies), G, out, ws)
    assert spark_device_status(ws) == 0
    ref, tol = A.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, kc.type, table, [T], [n_q], G, kc.page)
    return max(A.worst(out[i:i + 1], ref, tol) for i in range(copies))


FORMS = [(4, 1, torch.bfloat16), (4, 1, torch.float32), (8, 1, torch.bfloat16), (4, 4, torch.bfloat16),
         (4, 4, torch.float32)]


@pytest.mark.parametrize("copies", [1, 301])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n_q,dtype", FORMS)
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("where", [0, 5, 12])
@pytest.mark.parametrize("R_", [12, 20, 28, 60])
def test_a_page_of_large_values_without_weight(copies, kind, G, n_q, dtype, page, where, R_):
    """Its value scale is 2^R times the others', its weight 2^-(R + 20)."""
    bits = [(0, 0)] * 13
    bits[where] = (-(R_ + 20), R_)
    T = 13 * page - 3
    kc, table, q = _pages_of_size(T, page, kind, dtype, G, n_q, bits)
    assert _worst_of_copies(q, kc, table, T, G, copies) <= 1


@pytest.mark.parametrize("copies", [1, 301])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n_q,dtype", FORMS)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("step", [(3, -3), (-3, 3), (3, 2), (-2, -3), (0.25, 0), (5, -1)])
def test_scores_and_values_that_climb_or_fall(copies, kind, G, n_q, dtype, page, step):
    """Each page's scores and values lie some powers of two above or below those of the page before."""
    bits = [(i * step[0] - 12 * step[0], i * step[1] - 12 * step[1]) for i in range(25)]
    T = 25 * page - 5
    kc, table, q = _pages_of_size(T, page, kind, dtype, G, n_q, bits)
    assert _worst_of_copies(q, kc, table, T, G, copies) <= 1


@pytest.mark.parametrize("copies", [1, 301])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n_q,dtype", FORMS)
@pytest.mark.parametrize("size", [-116, -100, 100])
def test_values_far_from_one(copies, kind, G, n_q, dtype, size):
    T, page = 500, 32
    kc, table, q = _pages_of_size(T, page, kind, dtype, G, n_q, [(0, size)] * 16)
    assert _worst_of_copies(q, kc, table, T, G, copies) <= 1


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n_q,dtype", FORMS)
@pytest.mark.parametrize("top", [3, 250, 399])
@pytest.mark.parametrize("a", [10, 24, 26, 27, 28, 31, 40, 100])
def test_scores_far_beyond_the_steps_of_fp32(kind, G, n_q, dtype, top, a):
    """Scores of 2^a / sqrt(128) times 0 .. 8: the softmax is the one token with
    8, whatever its page's value scale and where the scores' reference stood."""
    T, page, H = 400, 16, 2
    g = _gen(9)
    k, v = torch.zeros((1, H, T, D), device=DEV), _values(g, (1, H, T, D))
    k[..., 0] = torch.randint(0, 8, (1, H, T), generator=g, device=DEV).float()
    k[..., top, 0] = 8.0
    v *= torch.exp2(torch.randint(-20, 21, (T // page,), generator=g, device=DEV).float()).repeat_interleave(page)[:, None]
    q = torch.zeros((1, H * G, n_q, D), device=DEV)
    q[..., 0] = 2.0 ** a
    kc = KV8Cache.empty(T // page, H, page, kind)
    table, ws = torch.arange(T // page, dtype=torch.int32, device=DEV)[None], workspace(256)
    spark_kv8_append(k, v, torch.arange(T, dtype=torch.int32, device=DEV)[None], kc, ws)
    copies = 301
    out = torch.full((copies, H * G, n_q, D), float("nan"), dtype=torch.float32, device=DEV)
    wsa = workspace(spark_workspace_bytes_kv8(copies, H, G, n_q))
    spark_decode_attn_kv8(q.to(dtype).expand(copies, -1, -1, -1).contiguous(), kc,
                          table.expand(copies, -1).contiguous(), i32([T] * copies), G, out, wsa)
    assert spark_device_status(wsa) == 0
    for h in range(H):
        want = R.decode(kc.v[top // page, h, top % page], kind) * kc.v_scale[top // page, h].double()
        sees = torch.tensor([top <= T - n_q + i for i in range(n_q)], device=DEV)
        got = out[:, h * G:(h + 1) * G][:, :, sees].double()
        # p is 1, its halves keep 22 bits, and a merge and the division round once
        # each; the other tokens weigh at most exp(-2^a / sqrt(128)) each
        room = 2.0 ** -20 * want.abs() + T * float(v.abs().max()) * 2 * math.exp(-min(700.0, 2.0 ** a / D ** 0.5))
        assert bool(((got - want).abs() <= room).all())


@pytest.mark.parametrize("copies", [1, 301])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,n_q,dtype", FORMS)
@pytest.mark.parametrize("where", [0, 5, 12])
def test_value_scales_at_both_ends_of_their_range(copies, kind, G, n_q, dtype, where):
    """A page whose value scale is 2^200 times the others' and whose weight is 2^-240."""
    bits = [(0, -100)] * 13
    bits[where] = (-240, 100)
    T, page = 13 * 16 - 3, 16
    kc, table, q = _pages_of_size(T, page, kind, dtype, G, n_q, bits)
    assert _worst_of_copies(q, kc, table, T, G, copies) <= 1
