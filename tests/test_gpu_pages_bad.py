"""Page numbers outside the pool that spark_pages_extend meets: each one is
reported by itself, and its tokens get no slot."""
import pytest
import torch

from channel_pruned_decode_b200 import spark_device_status, spark_pages_extend, workspace
from channel_pruned_decode_b200.binding import SPARK_ERR_ARG

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_cap", [1, 2, 4, 40, 5000])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 8, 2 ** 31 - 1])
def test_a_page_that_the_row_already_holds(bad, n_cap, in_place):
    """Only the second row's last page is bad, and its new tokens start inside it."""
    L, T, tk = i32([3, 19, 16]), i32([[0, -9], [1, bad], [3, -9]]), i32([4])
    slots = torch.full((3, n_cap), -77, dtype=torch.int32, device=DEV)
    lo, to = (L, tk) if in_place else (torch.zeros_like(L), torch.zeros_like(tk))
    ws = workspace(256)
    spark_pages_extend(L, i32([1, min(n_cap, 3), 0]), 16, i32(list(range(8))), tk, T, slots, lo, to, ws)
    assert spark_device_status(ws) == SPARK_ERR_ARG
    assert slots[0].tolist() == [3] + [-1] * (n_cap - 1)
    assert slots[1].tolist() == slots[2].tolist() == [-1] * n_cap
    assert T.tolist() == [[0, -9], [1, bad], [3, -9]]


@pytest.mark.parametrize("n_cap", [1, 2, 4, 40, 5000])
@pytest.mark.parametrize("bad", [-1, 8])
def test_a_free_page(bad, n_cap):
    slots = torch.full((2, n_cap), -77, dtype=torch.int32, device=DEV)
    T, lo, to, ws = i32([[0, -9], [1, -9]]), i32([0, 0]), i32([0]), workspace(256)
    spark_pages_extend(i32([3, 16]), i32([1, 1]), 16, i32([0, 1, bad, 3, 4, 5, 6, 7]), i32([2]), T, slots, lo, to, ws)
    assert spark_device_status(ws) == SPARK_ERR_ARG
    assert slots.tolist() == [[3] + [-1] * (n_cap - 1), [-1] * n_cap]
    assert T.tolist() == [[0, -9], [1, -1]]


def test_a_page_that_no_new_token_touches_is_not_read():
    slots, lo, to, ws = i32([[-77], [-77]]), i32([0, 0]), i32([0]), workspace(256)
    T = i32([[99, 2, -9], [99, -9, -9]])
    spark_pages_extend(i32([20, 5]), i32([1, 0]), 16, i32(list(range(8))), i32([3]), T, slots, lo, to, ws)
    assert spark_device_status(ws) == 0 and slots.tolist() == [[36], [-1]]
