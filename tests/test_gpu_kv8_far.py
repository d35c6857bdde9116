"""Attention over rows at the end of the 32-bit ranges that the call accepts:
tables that list a few pages over and over.  Keys are zeros, so that every
token weighs the same and the output is the mean of the values."""
import pytest
import torch

from channel_pruned_decode_b200 import (KV8Cache, spark_decode_attn_kv8, spark_device_status,
                                        spark_workspace_bytes_kv8, workspace, SPARK_KV8_I8)
from channel_pruned_decode_b200.binding import SPARK_ERR_ARG
from tests import _kv8_bound as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128


@pytest.mark.parametrize("page,cap,cycle,H,n_q,lens,status", [
    # 2^31 - 16 tokens in one row: its steps are counted up to a sum past 2^31
    (16, (1 << 27) - 1, 7, 1, 1, (1 << 31) - 16, 0),
    (16, (1 << 27) - 1, 7, 1, 3, (1 << 31) - 1, SPARK_ERR_ARG),  # longer than the table: cut to it, and flagged
    # 2^31 - 128 steps of all heads: the line ends less than one step a CTA below 2^31
    (128, (1 << 24) - 1, 15, 32, 1, (1 << 31) - 128, 0),
])
def test_mean_of_a_row_that_repeats_its_pages(page, cap, cycle, H, n_q, lens, status):
    g = torch.Generator(device=DEV).manual_seed(cycle)
    kc = KV8Cache.empty(cycle, H, page, SPARK_KV8_I8)
    kc.k.zero_()
    kc.v.copy_(torch.randint(1, 128, kc.v.shape, generator=g, device=DEV).to(torch.uint8))
    kc.k_scale.fill_(1.0)
    kc.v_scale.fill_(2.0 ** -6)
    table = torch.arange(cap, dtype=torch.int32, device=DEV).remainder_(cycle)[None]
    q = torch.randn((1, H, n_q, D), generator=g, device=DEV).bfloat16()
    out = torch.full(q.shape, float("nan"), dtype=torch.float32, device=DEV)
    ws = workspace(spark_workspace_bytes_kv8(1, H, 1, n_q))
    spark_decode_attn_kv8(q, kc, table, torch.tensor([lens], dtype=torch.int32, device=DEV), 1, out, ws)
    assert spark_device_status(ws) == status
    T = min(lens, cap * page)
    v = kc.v.double() * 2.0 ** -6                     # [cycle, H, page, D]
    total = v.sum((0, 2)) * (cap // cycle)            # [H, D]
    S = A.stretch([T], H, n_q, False, torch.cuda.get_device_properties(0).multi_processor_count)
    for i in range(n_q):
        behind = n_q - 1 - i  # the row's last tokens, which this query does not see
        want = (total - v[cycle - 1, :, page - behind:].sum(1)) / (T - behind)
        # every p is 1: their sum (up to 2^23) is exact, and so are scores and halves
        tol = ((64 + S / 16 + 8) * 2.0 ** -22 + 32 * 2.0 ** -24) * want
        assert bool(((out[0, :, i] - want).abs() <= tol).all())
