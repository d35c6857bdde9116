"""Refusals of spark_pages_extend_served and of n_served in the binding: no
call here launches anything."""
import pytest
import torch

from channel_pruned_decode_b200 import binding as B


@pytest.fixture(scope="module")
def L():
    from channel_pruned_decode_b200 import build
    build.build()
    return B.lib()


def test_refusals(L):
    def f(lens=16, nn=32, b=2, page=16, pool=48, n=8, tk=64, t=80, cap=4, ncap=4, s=96, lo=112, to=128, sv=144,
          ws=256, wsb=256):
        return L.spark_pages_extend_served(lens, nn, b, page, pool, n, tk, t, cap, ncap, s, lo, to, sv, ws, wsb, None)
    for kw in (dict(sv=None), dict(sv=146), dict(sv=16), dict(sv=20), dict(sv=32), dict(sv=28), dict(sv=112),
               dict(sv=116), dict(lens=None), dict(nn=None), dict(lo=None), dict(lo=20), dict(s=None), dict(ncap=-1)):
        assert f(**kw) == B.SPARK_ERR_ARG, kw
    assert f(page=20) == f(cap=1 << 27) == f(b=(1 << 16) + 1) == B.SPARK_ERR_UNSUPPORTED
    assert f(ws=None) == f(ws=8) == f(wsb=128) == B.SPARK_ERR_WORKSPACE
    assert f(lens=None, sv=None, b=0) == B.SPARK_OK


def test_binding_checks_n_served():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    args = (i32(3), i32(3), 16, i32(9), i32(1), i32(3, 4), i32(3, 5), i32(3), i32(1), torch.zeros(256, dtype=torch.uint8))
    for bad in (i32(4), i32(3).long(), i32(6)[::2]):
        with pytest.raises(ValueError, match="n_served"):
            B.spark_pages_extend(*args, n_served=bad)
    with pytest.raises(ValueError, match="current CUDA device"):
        B.spark_pages_extend(*args, n_served=i32(3))
