"""Host side of the paged 8-bit cache: sizes, refusals (every call here fails
validation, launches nothing and touches no device) and the test
implementation's own pins."""
import ctypes

import numpy as np
import pytest
import torch

from channel_pruned_decode_b200 import binding as B
from tests import _kv8 as R


@pytest.fixture(scope="module")
def L():
    from channel_pruned_decode_b200 import build
    build.build()
    return B.lib()


def _kc(**kw):
    d = dict(n_pages=8, Hkv=2, page=16, D=128, type=0, k=16, v=16, k_scale=16, v_scale=16)
    d.update(kw)
    return B.spark_kv8cache(**d)


def test_sizes(L):
    total, sz = B.spark_kv8_sizes(10, 8, 32)
    assert sz == [10 * 8 * 32 * 128] * 2 + [10 * 8 * 4] * 2
    assert total == 2 * 10 * 8 * 32 * 128 + 2 * 512
    assert B.spark_kv8_sizes(10, 8, 24)[0] == 0            # page
    assert B.spark_kv8_sizes(10, 8, 32, 64)[0] == 0        # D
    assert B.spark_kv8_sizes(-1, 8, 32)[0] == 0
    assert B.spark_kv8_sizes(1 << 20, 64, 32)[0] == 0      # 2^31 rows
    assert B.spark_kv8_sizes((1 << 20) - 1, 64, 32)[0] > 0


def test_workspace_bytes(L):
    f = B.spark_workspace_bytes_kv8
    assert f(4, 8, 4, 1) >= 256
    assert f(4, 8, 0, 1) == 0 and f(4, 8, 4, 0) == 0 and f(-1, 8, 4, 1) == 0
    assert f(4, 8, 8, 8) > 0 and f(4, 8, 13, 5) == 0       # 64 rows per kv head at most


@pytest.mark.parametrize("kw,want", [
    (dict(D=64), B.SPARK_ERR_UNSUPPORTED),
    (dict(page=24), B.SPARK_ERR_UNSUPPORTED),
    (dict(page=256), B.SPARK_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 30), B.SPARK_ERR_UNSUPPORTED),
    (dict(n_pages=-1), B.SPARK_ERR_ARG),
    (dict(Hkv=-1), B.SPARK_ERR_ARG),
    (dict(type=2), B.SPARK_ERR_ARG),
    (dict(k=None), B.SPARK_ERR_ARG),
    (dict(v=24), B.SPARK_ERR_ARG),
    (dict(k_scale=None), B.SPARK_ERR_ARG),
    (dict(v_scale=8), B.SPARK_ERR_ARG),
])
def test_bad_cache(L, kw, want):
    kc = _kc(**kw)
    assert L.spark_kv8_append(16, 16, 1, 4, B.SPARK_BF16, 16, ctypes.byref(kc), 256, 256, None) == want
    assert L.spark_decode_attn_kv8(16, B.SPARK_BF16, ctypes.byref(kc), 16, 4, 16, None, 1, 4, 1, 16, 256, 1 << 30,
                                   None) == want
    assert L.spark_kv8_append(16, 16, 1, 4, B.SPARK_BF16, 16, None, 256, 256, None) == B.SPARK_ERR_ARG


def test_append_rejects_bad_args(L):
    def f(k=16, v=16, b=1, n=4, dt=B.SPARK_BF16, s=16, ws=256, wsb=256):
        return L.spark_kv8_append(k, v, b, n, dt, s, ctypes.byref(_kc()), ws, wsb, None)
    assert f(k=None) == f(v=8) == f(s=None) == f(s=18) == B.SPARK_ERR_ARG
    assert f(b=-1) == f(n=-1) == f(dt=3) == B.SPARK_ERR_ARG
    assert f(b=1 << 20, n=1 << 12) == B.SPARK_ERR_UNSUPPORTED
    assert f(ws=None) == f(ws=8) == f(wsb=255) == B.SPARK_ERR_WORKSPACE
    assert f(k=None, b=0) == f(k=None, n=0) == B.SPARK_OK


def test_attn_rejects_bad_args(L):
    def f(q=16, dt=B.SPARK_BF16, t=16, cap=4, lens=16, nn=None, b=1, G=4, n=1, out=16, ws=256, wsb=1 << 30):
        return L.spark_decode_attn_kv8(q, dt, ctypes.byref(_kc()), t, cap, lens, nn, b, G, n, out, ws, wsb, None)
    assert f(q=None) == f(q=8) == f(out=None) == f(out=24) == f(lens=None) == f(lens=2) == B.SPARK_ERR_ARG
    assert f(t=None) == f(t=2) == f(nn=2) == f(cap=-1) == f(b=-1) == f(G=0) == f(n=0) == f(dt=7) == B.SPARK_ERR_ARG
    assert f(G=13, n=5) == f(G=65) == f(n=65) == B.SPARK_ERR_UNSUPPORTED
    assert f(cap=1 << 28) == f(b=1 << 25) == B.SPARK_ERR_UNSUPPORTED
    assert f(ws=None) == f(ws=8) == f(wsb=0) == B.SPARK_ERR_WORKSPACE
    assert f(q=None, b=0) == B.SPARK_OK


def test_pages_reject_bad_args(L):
    def ext(lens=16, nn=32, b=2, page=16, pool=48, n=8, tk=64, t=80, cap=4, ncap=4, s=96, lo=112, to=128, ws=256,
            wsb=256):
        return L.spark_pages_extend(lens, nn, b, page, pool, n, tk, t, cap, ncap, s, lo, to, ws, wsb, None)

    def trim(lens=16, nn=32, b=2, page=16, pool=48, n=8, tk=64, t=80, cap=4, lo=112, to=128, ws=256, wsb=256):
        return L.spark_pages_trim(lens, nn, b, page, pool, n, tk, t, cap, lo, to, ws, wsb, None)
    for f in (ext, trim):
        for kw in (dict(lens=None), dict(nn=None), dict(pool=None), dict(tk=None), dict(t=None), dict(lo=None),
                   dict(to=None), dict(lens=18), dict(pool=50), dict(b=-1), dict(n=-1), dict(cap=-1),
                   dict(lo=20), dict(lo=12),        # overlaps lens without being it
                   dict(lo=32), dict(lo=36)):       # overlaps n_new / keep
            assert f(**kw) == B.SPARK_ERR_ARG, kw
        assert f(page=20) == f(cap=1 << 27) == f(b=1 << 16, cap=1 << 15) == B.SPARK_ERR_UNSUPPORTED
        assert f(ws=None) == f(ws=8) == f(wsb=128) == B.SPARK_ERR_WORKSPACE
        assert f(lens=None, b=0) == B.SPARK_OK
    assert ext(ncap=-1) == ext(s=None) == ext(s=20) == B.SPARK_ERR_ARG


def test_binding_refuses_wrong_tensors():
    """The library sees bare pointers: shapes, types, layout and device are checked before the call."""
    kc = B.KV8Cache.empty(4, 2, 16, device="cpu")
    with pytest.raises(ValueError, match="uint8"):
        B.KV8Cache(4, 2, 16, 128, 0, kc.k.view(torch.int8), kc.v, kc.k_scale, kc.v_scale)
    with pytest.raises(ValueError, match="shape"):
        B.KV8Cache(4, 2, 32, 128, 0, kc.k, kc.v, kc.k_scale, kc.v_scale)
    with pytest.raises(ValueError, match="contiguous"):
        B.KV8Cache(4, 2, 16, 128, 0, kc.k.transpose(0, 1).contiguous().transpose(0, 1), kc.v, kc.k_scale, kc.v_scale)
    ws = torch.zeros(256, dtype=torch.uint8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x, slots = torch.zeros((3, 2, 5, 128)), i32(3, 5)
    with pytest.raises(ValueError, match="current CUDA device"):
        B.spark_kv8_append(x, x, slots, kc, ws)
    with pytest.raises(ValueError, match="contiguous"):
        B.spark_kv8_append(x.transpose(1, 2).contiguous().transpose(1, 2), x, slots, kc, ws)
    with pytest.raises(ValueError, match="v_new"):
        B.spark_kv8_append(x, x.bfloat16(), slots, kc, ws)
    with pytest.raises(ValueError, match="slots"):
        B.spark_kv8_append(x, x, slots.long(), kc, ws)
    with pytest.raises(ValueError, match="k_new"):
        B.spark_kv8_append(x[:, :1], x, slots, kc, ws)
    q, out = torch.zeros((3, 8, 1, 128)), torch.zeros((3, 8, 1, 128))
    with pytest.raises(ValueError, match="current CUDA device"):
        B.spark_decode_attn_kv8(q, kc, i32(3, 4), i32(3), 4, out, ws)
    with pytest.raises(ValueError, match="lens"):
        B.spark_decode_attn_kv8(q, kc, i32(3, 4), i32(4), 4, out, ws)
    with pytest.raises(ValueError, match="out"):
        B.spark_decode_attn_kv8(q, kc, i32(3, 4), i32(3), 4, out.bfloat16(), ws)
    with pytest.raises(ValueError, match="q:"):
        B.spark_decode_attn_kv8(q, kc, i32(3, 4), i32(3), 2, out, ws)
    with pytest.raises(ValueError, match="n_new"):
        B.spark_decode_attn_kv8(q, kc, i32(3, 4), i32(3), 4, out, ws, n_new=i32(3).long())
    with pytest.raises(ValueError, match="current CUDA device"):
        B.spark_pages_extend(i32(3), i32(3), 16, i32(9), i32(1), i32(3, 4), i32(3, 5), i32(3), i32(1), ws)
    with pytest.raises(ValueError, match="ws"):
        B.spark_pages_extend(i32(3), i32(3), 16, i32(9), i32(1), i32(3, 4), i32(3, 5), i32(3), i32(1),
                             torch.zeros((64, 8), dtype=torch.uint8).t())
    with pytest.raises(ValueError, match="ws"):
        B.spark_kv8_append(x, x, slots, kc, torch.zeros((64, 8), dtype=torch.uint8).t())
    with pytest.raises(ValueError, match="taken"):
        B.spark_pages_extend(i32(3), i32(3), 16, i32(9), i32(2), i32(3, 4), i32(3, 5), i32(3), i32(1), ws)
    with pytest.raises(ValueError, match="table"):
        B.spark_pages_trim(i32(3), i32(3), 16, i32(9), i32(1), i32(2, 4), i32(3), i32(1), ws)


def test_oracle_rounding_pins():
    """The tests' own 8-bit rounding against torch's conversion and hand values."""
    y = np.concatenate([np.linspace(-448, 448, 20001), np.exp2(np.linspace(-12, 8.8, 4001)), [0.0, 2.0 ** -10]])
    want = torch.tensor(y, dtype=torch.float64).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.round8(y.astype(np.float32).astype(np.float64), R.E4M3), want)
    assert R.round8(np.array([0.5, 1.5, -2.5, 300.0, np.nan]), R.I8).tolist() == [0, 2, -2, 127, 0]
    assert R.scale_of(448.0, R.E4M3) == 1.0 and R.scale_of(448.0001, R.E4M3) == 2.0
    assert R.scale_of(127.0, R.I8) == 1.0 and R.scale_of(63.5, R.I8) == 0.5
    assert R.scale_of(0.0, R.E4M3) == 2.0 ** -126


def test_oracle_page_pins():
    table, slots, lens, taken, out = R.extend([0, 15, 16], [3, 2, 0], 16, [5, 9, 2, 7], 1,
                                              [[-9, -9], [4, -9], [3, -9]], 4)
    assert table == [[9, -9], [4, 2], [3, -9]] and lens == [3, 17, 16] and taken == 3 and not out
    assert slots == [[144, 145, 146, -1], [79, 32, -1, -1], [-1] * 4]
    _, slots, lens, taken, out = R.extend([15], [20], 16, [5], 0, [[4, -9, -9]], 20)
    assert out and taken == 1 and lens == [32] and slots[0][17:] == [-1] * 3
    pool, lens, taken = R.trim([17, 40], [16, 0], 16, [0, 1, 2, 3, 4, 5], 5, [[8, 9, -1], [10, 11, 12]])
    assert pool == [0, 9, 10, 11, 12, 5] and lens == [16, 0] and taken == 1


def _extend(L, b=1, page=16, n_pages=8, cap=4, n=4):
    return L.spark_pages_extend(16, 32, b, page, 16, n_pages, 16, 16, cap, n, 16, 48, 64, 256, 256, None)


def _trim(L, b=1, page=16, n_pages=8, cap=4):
    return L.spark_pages_trim(16, 32, b, page, 16, n_pages, 16, 16, cap, 48, 64, 256, 256, None)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pool_beyond_32_bit_slots(L, page):
    """A slot is page number * page + place in 32 bits."""
    n = (1 << 31) // page
    assert _extend(L, page=page, n_pages=n) == _trim(L, page=page, n_pages=n) == B.SPARK_ERR_UNSUPPORTED


def test_more_new_tokens_than_a_row_can_index(L):
    assert _extend(L, n=(1 << 30) + 1) == _extend(L, n=(1 << 31) - 1) == B.SPARK_ERR_UNSUPPORTED


def test_more_rows_than_the_sums_are_made_for(L):
    """Each CTA sums the rows before its own, so work grows with the square."""
    b = (1 << 16) + 1
    assert _extend(L, b=b) == _trim(L, b=b) == _trim(L, b=(1 << 31) - 1, cap=0) == B.SPARK_ERR_UNSUPPORTED
