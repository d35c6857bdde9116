"""Page tables and slot maps built on the GPU against the plain rules: whole
numbers, equal in every place."""
import random

import pytest
import torch

from channel_pruned_decode_b200 import (spark_device_status, spark_pages_extend, spark_pages_trim, workspace)
from channel_pruned_decode_b200.binding import SPARK_ERR_ARG, SPARK_ERR_PAGES
from tests import _kv8 as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _state(rng, lens, page, cap, free):
    """Tables that hold the rows' pages (-9 behind them) and a pool with `free` pages left."""
    need = [R.ceil_div(x, page) for x in lens]
    ids = list(range(sum(need) + free))
    rng.shuffle(ids)
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [-9] * (cap - n))
        at += n
    return table, ids, at


@pytest.mark.parametrize("B,page,n_cap,longest", [(1, 16, 1, 40), (7, 32, 5, 300), (300, 16, 1, 2000),
                                                  (33, 64, 129, 1000), (5, 16, 5000, 100), (2, 128, 2048, 0),
                                                  (513, 16, 4, 37), (1, 16, 0, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(B, page, n_cap, longest, in_place):
    rng = random.Random(B * 131 + n_cap)
    lens = [rng.randint(0, longest) for _ in range(B)]
    new = [rng.choice([0, n_cap, rng.randint(0, n_cap)]) for _ in range(B)]
    cap = max(1, max(R.ceil_div(a + n, page) for a, n in zip(lens, new))) + 2
    table, pool, taken = _state(rng, lens, page, cap, sum(R.ceil_div(n, page) + 1 for n in new))
    want = R.extend(lens, new, page, pool, taken, table, n_cap)
    L, T, tk = i32(lens), i32(table), i32([taken])
    slots = torch.full((B, n_cap), -77, dtype=torch.int32, device=DEV)
    lo, to = (L, tk) if in_place else (torch.full_like(L, -1), torch.full_like(tk, -1))
    ws = workspace(256)
    spark_pages_extend(L, i32(new), page, i32(pool), tk, T, slots, lo, to, ws)
    assert spark_device_status(ws) == 0
    assert T.tolist() == want[0]
    assert slots.tolist() == want[1]
    assert lo.tolist() == want[2]
    assert to.tolist() == [want[3]]
    assert int(ws.count_nonzero()) == 0  # the ticket is back at zero


@pytest.mark.parametrize("free", [0, 1, 7])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_when_the_pool_runs_out(free, in_place):
    rng = random.Random(free)
    lens, new, page = [0, 15, 16, 40, 3], [50, 1, 33, 0, 14], 16
    table, pool, taken = _state(rng, lens, page, 8, free)
    want = R.extend(lens, new, page, pool, taken, table, 50)
    assert want[4]
    L, T, tk = i32(lens), i32(table), i32([taken])
    slots = torch.zeros((5, 50), dtype=torch.int32, device=DEV)
    lo, to = (L, tk) if in_place else (torch.full_like(L, -1), torch.full_like(tk, -1))
    ws = workspace(256)
    spark_pages_extend(L, i32(new), page, i32(pool), tk, T, slots, lo, to, ws)
    assert spark_device_status(ws, clear=True) == SPARK_ERR_PAGES
    assert (T.tolist(), slots.tolist(), lo.tolist(), to.tolist()) == (want[0], want[1], want[2], [want[3]])


@pytest.mark.parametrize("lens,new,taken,want_lens", [
    ([-5, 3], [1, 1], 4, [1, 4]),          # a negative length counts as 0
    ([0, 3], [-1, 1], 4, [0, 4]),
    ([0, 3], [9, 1], 4, [4, 4]),           # more new tokens than n_cap
    ([40, 3], [1, 1], 4, [32, 4]),         # longer than the table
    ([31, 3], [4, 1], 4, [32, 4]),
    ([3, 3], [1, 1], -3, [4, 4]),
])
def test_extend_clamps_and_flags_bad_lengths(lens, new, taken, want_lens):
    page, cap, n_cap = 16, 2, 4
    table = [[0, 1], [2, 3]]
    pool = list(range(16))
    slots = torch.zeros((2, n_cap), dtype=torch.int32, device=DEV)
    L, T = i32(lens), i32(table)
    lo, to, ws = torch.zeros_like(L), i32([0]), workspace(256)
    spark_pages_extend(L, i32(new), page, i32(pool), i32([taken]), T, slots, lo, to, ws)
    assert spark_device_status(ws) == SPARK_ERR_ARG
    assert lo.tolist() == want_lens
    s = slots.tolist()
    assert all(-1 <= x < 16 * page for r in s for x in r)


def test_extend_refuses_bad_page_numbers():
    """A page number outside the pool, in the table or among the free pages, gives no slot."""
    slots = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    T, lo, to, ws = i32([[99, -1], [1, -1]]), i32([0, 0]), i32([0]), workspace(256)
    spark_pages_extend(i32([3, 16]), i32([2, 2]), 16, i32([0, 1, -4, 3]), i32([2]), T, slots, lo, to, ws)
    assert spark_device_status(ws) == SPARK_ERR_ARG
    assert slots.tolist() == [[-1, -1], [-1, -1]]
    assert T.tolist() == [[99, -1], [1, -1]]


@pytest.mark.parametrize("B,page,longest,mode", [(1, 16, 40, "all"), (9, 32, 300, "some"), (300, 16, 2000, "drafts"),
                                                 (64, 128, 9000, "some"), (5, 16, 0, "all"), (40, 16, 500, "none")])
@pytest.mark.parametrize("in_place", [False, True])
def test_trim(B, page, longest, mode, in_place):
    rng = random.Random(B + longest)
    lens = [rng.randint(0, longest) for _ in range(B)]
    keep = {"all": [0] * B, "none": [x + rng.randint(0, 3) for x in lens],
            "some": [rng.choice([0, x, x // 2]) for x in lens],
            "drafts": [max(0, x - rng.randint(0, 4)) for x in lens]}[mode]
    cap = max(1, R.ceil_div(longest, page))
    table, pool, taken = _state(rng, lens, page, cap, 11)
    want = R.trim(lens, keep, page, pool, taken, table)
    L, T, tk, Pl = i32(lens), i32(table), i32([taken]), i32(pool)
    lo, to = (L, tk) if in_place else (torch.full_like(L, -1), torch.full_like(tk, -1))
    ws = workspace(256)
    spark_pages_trim(L, i32(keep), page, Pl, tk, T, lo, to, ws)
    assert spark_device_status(ws) == 0
    assert (Pl.tolist(), lo.tolist(), to.tolist()) == (want[0], want[1], [want[2]])
    assert T.tolist() == table
    assert int(ws.count_nonzero()) == 0


def test_trim_flags_bad_input():
    for lens, keep, taken, table in (([-1], [0], 2, [[0, 1]]), ([20], [-2], 2, [[0, 1]]), ([99], [0], 2, [[0, 1]]),
                                     ([20], [0], 2, [[0, 50]]), ([20], [0], 1, [[0, 1]]), ([20], [0], 9, [[0, 1]])):
        Pl, lo, to, ws = i32([5, 5, 5, 5]), i32([0]), i32([0]), workspace(256)
        spark_pages_trim(i32(lens), i32(keep), 16, Pl, i32([taken]), i32(table), lo, to, ws)
        assert spark_device_status(ws) == SPARK_ERR_ARG
        assert all(-1 <= x <= 5 for x in Pl.tolist()) and 0 <= to.item() <= 4


def test_pages_come_back_in_the_order_they_are_taken():
    """Extend and trim by turns: no page is lost or handed out twice."""
    rng = random.Random(5)
    B, page, cap, n_pages = 12, 16, 16, 150
    L, tk = i32([0] * B), i32([0])
    T, Pl = i32([[-1] * cap for _ in range(B)]), i32(rng.sample(range(n_pages), n_pages))
    slots, ws = torch.zeros((B, 40), dtype=torch.int32, device=DEV), workspace(256)
    for _ in range(30):
        room = [cap * page - x for x in L.tolist()]
        spark_pages_extend(L, i32([min(r, rng.randint(0, 40)) for r in room]), page, Pl, tk, T, slots, L, tk, ws)
        spark_device_status(ws, clear=True)  # it may run out
        spark_pages_trim(L, i32([rng.choice([x, x, max(0, x - 5), 0]) for x in L.tolist()]), page, Pl, tk, T, L, tk,
                         ws)
        assert spark_device_status(ws) == 0
        held = [p for row, x in zip(T.tolist(), L.tolist()) for p in row[:R.ceil_div(x, page)]]
        assert sorted(held + Pl.tolist()[tk.item():]) == list(range(n_pages))


def test_largest_batch():
    """65536 rows, the most a call takes: extended in place, then cut back to what they were."""
    B, page, cap = 1 << 16, 16, 4
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 40, (B,), generator=g)
    new = torch.randint(0, 3, (B,), generator=g)
    have, want = (lens + page - 1) // page, (lens + new + page - 1) // page
    ids = torch.randperm(int(want.sum()), generator=g)
    held, places = int(have.sum()), torch.arange(cap)[None]
    table = torch.full((B, cap), -9)
    table[places < have[:, None]] = ids[:held]
    full = table.clone()
    full[(places >= have[:, None]) & (places < want[:, None])] = ids[held:]
    at = lens[:, None] + torch.arange(2)[None]
    slots = torch.gather(full, 1, (at // page).clamp(max=cap - 1)) * page + at % page
    slots[torch.arange(2)[None] >= new[:, None]] = -1
    put = lambda t: t.to(torch.int32).to(DEV)
    L, N, T, P, K = put(lens), put(new), put(table), put(ids), put(lens)
    tk, S, ws = i32([held]), put(torch.full((B, 2), -77)), workspace(256)
    spark_pages_extend(L, N, page, P, tk, T, S, L, tk, ws)
    assert torch.equal(L, put(lens + new)) and torch.equal(T, put(full)) and torch.equal(S, put(slots))
    assert int(tk) == ids.numel() and spark_device_status(ws) == 0
    spark_pages_trim(L, K, page, P, tk, T, L, tk, ws)
    assert torch.equal(L, K) and torch.equal(P, put(ids)) and int(tk) == held and spark_device_status(ws) == 0
