"""Steps in which the page pool runs out, or new tokens are clamped: how many
tokens each row got, and the attention of those that it got."""
import random

import pytest
import torch

from channel_pruned_decode_b200 import (spark_decode_attn_kv8, spark_device_status, spark_kv8_append,
                                        spark_pages_extend, KV8Cache, spark_workspace_bytes_kv8, workspace)
from channel_pruned_decode_b200.binding import SPARK_ERR_ARG, SPARK_ERR_PAGES
from tests import _kv8 as R
from tests import _kv8_bound as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("free", [0, 1, 7, 100])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_cap", [50, 5000])
def test_tokens_served(free, in_place, n_cap):
    rng = random.Random(free)
    lens, new, page = [0, 15, 16, 40, 3, 0] + [7] * 300, [50, 1, 33, 0, 14, 9] + [12] * 300, 16
    need = [R.ceil_div(x, page) for x in lens]
    ids = rng.sample(range(sum(need) + free), sum(need) + free)
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [-9] * (8 - n))
        at += n
    want = R.extend(lens, new, page, ids, at, table, n_cap)
    L, T, tk, S = i32(lens), i32(table), i32([at]), torch.full((len(lens),), -7, dtype=torch.int32, device=DEV)
    slots = torch.zeros((len(lens), n_cap), dtype=torch.int32, device=DEV)
    lo, to = (L, tk) if in_place else (torch.full_like(L, -1), torch.full_like(tk, -1))
    ws = workspace(256)
    spark_pages_extend(L, i32(new), page, i32(ids), tk, T, slots, lo, to, ws, n_served=S)
    assert spark_device_status(ws, clear=True) == (SPARK_ERR_PAGES if want[4] else 0)
    assert (T.tolist(), slots.tolist(), lo.tolist(), to.tolist()) == (want[0], want[1], want[2], [want[3]])
    assert S.tolist() == [a - b for a, b in zip(want[2], lens)]


@pytest.mark.parametrize("lens,new,served", [([-5, 3], [1, 1], [1, 1]), ([0, 3], [-1, 1], [0, 1]),
                                             ([0, 3], [9, 1], [4, 1]), ([40, 3], [1, 1], [0, 1]),
                                             ([31, 3], [4, 1], [1, 1])])
def test_tokens_served_of_clamped_rows(lens, new, served):
    L, lo, to, S, ws = i32(lens), i32([0, 0]), i32([0]), i32([-7, -7]), workspace(256)
    slots = torch.zeros((2, 4), dtype=torch.int32, device=DEV)
    spark_pages_extend(L, i32(new), 16, i32(list(range(16))), i32([4]), i32([[0, 1], [2, 3]]), slots, lo, to, ws,
                       n_served=S)
    assert spark_device_status(ws) == SPARK_ERR_ARG
    assert S.tolist() == served


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("n", [1, 5])
def test_attention_when_the_pool_runs_out(captured, n):
    """Rows of which all, some or none of the new tokens found a page: each
    query that has a token sees its own and those before it, the others' rows
    stay as they were.  The same step again, eager and replayed."""
    B, H, G, page, cap = 5, 2, 4, 16, 8
    g = torch.Generator(device=DEV).manual_seed(n)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.float32)  # noqa: E731
    n_pages = 12
    kc = KV8Cache.empty(n_pages, H, page)
    L, tk, S, T = i32([0] * B), i32([0]), i32([0] * B), torch.full((B, cap), -1, dtype=torch.int32, device=DEV)
    pool, ws = i32(random.Random(3).sample(range(n_pages), n_pages)), workspace(256)
    wsa = workspace(spark_workspace_bytes_kv8(B, H, G, n))
    # prompts that leave no place (16, 32), one (31, 15) and some (13), and one page in the pool
    held = [16, 31, 32, 15, 13]
    first = torch.zeros((B, 40), dtype=torch.int32, device=DEV)
    pk, pv = rand(B, H, 40, D), rand(B, H, 40, D)
    spark_pages_extend(L, i32(held), page, pool, tk, T, first, L, tk, ws)
    spark_kv8_append(pk, pv, first, kc, ws)
    assert spark_device_status(ws) == 0 and tk.item() == 7
    tk.fill_(n_pages - 1)
    new = i32([n] * B)
    slots, out = torch.zeros((B, n), dtype=torch.int32, device=DEV), torch.zeros((B, H * G, n, D), device=DEV)
    k, v, q = rand(B, H, n, D), rand(B, H, n, D), rand(B, H * G, n, D)

    def step():
        spark_pages_extend(L, new, page, pool, tk, T, slots, L, tk, ws, n_served=S)
        spark_kv8_append(k, v, slots, kc, ws)
        spark_decode_attn_kv8(q, kc, T, L, G, out, wsa, n_new=S)

    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
        torch.cuda.synchronize()
    lens, left = list(held), 1
    some = False
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay() if captured else step()
        served = []
        for b, x in enumerate(lens):
            want = R.ceil_div(x + n, page) - R.ceil_div(x, page)
            got = min(want, left)
            left -= got
            served.append(min(n, (R.ceil_div(x, page) + got) * page - x))
        some |= any(0 < s < n for s in served)
        lens = [x + s for x, s in zip(lens, served)]
        assert (S.tolist(), L.tolist()) == (served, lens) and 0 in served and n in served
        ref, tol = A.attention(q, kc.k, kc.v, kc.k_scale, kc.v_scale, 0, T, lens, served, G, page)
        assert torch.equal(torch.isnan(out), torch.isnan(ref))
        assert A.worst(out, ref, tol) <= 1
    assert some == (n > 1)
    assert spark_device_status(ws) == SPARK_ERR_PAGES and spark_device_status(wsa) == 0
    del graph
