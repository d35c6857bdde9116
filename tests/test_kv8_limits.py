"""Counts near the end of 32 bits that spark_kv8_append refuses on the host."""
import ctypes

import pytest

from channel_pruned_decode_b200 import binding as B


@pytest.fixture(scope="module")
def L():
    from channel_pruned_decode_b200 import build
    build.build()
    return B.lib()


@pytest.mark.parametrize("n_cap", [(1 << 30) + 1, (1 << 31) - 120, (1 << 31) - 1])
@pytest.mark.parametrize("page", [16, 128])
def test_append_more_tokens_than_a_row_can_index(L, n_cap, page):
    """The pieces of a row are counted by a sum past n_cap."""
    kc = B.spark_kv8cache(n_pages=8, Hkv=1, page=page, D=128, type=0, k=16, v=16, k_scale=16, v_scale=16)
    assert L.spark_kv8_append(16, 16, 1, n_cap, B.SPARK_BF16, 16, ctypes.byref(kc), 256, 256, None) == B.SPARK_ERR_UNSUPPORTED
