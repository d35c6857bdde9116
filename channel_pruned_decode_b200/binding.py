"""Thin ctypes binding of libspark.so (include/spark.h).

Argument marshalling only: every step of pruning and decode runs in the CUDA
kernels of libspark.so.  The paged cache's calls, of which a decode step makes
several a layer, are marshalled by csrc/calls.cpp.  torch tensors supply device
memory and streams.
There is no CPU fallback: loading fails loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspark.so")

SPARK_OK = 0
SPARK_ERR_ARG = 1
SPARK_ERR_UNSUPPORTED = 2
SPARK_ERR_CUDA = 3
SPARK_ERR_TIMEOUT = 4
SPARK_ERR_WORKSPACE = 5
SPARK_ERR_PAGES = 6
SPARK_F32 = 0
SPARK_BF16 = 1
SPARK_F_DEGENERATE = 0
SPARK_F_GAUSSIAN = 1
SPARK_F_EXPONENTIAL = 2
SPARK_OP_PRUNE = 0
SPARK_OP_DECODE = 1
SPARK_OP_SNAPKV = 2
SPARK_OP_THINK = 3
SPARK_OP_TOPP = 4
SPARK_KV8_E4M3 = 0
SPARK_KV8_I8 = 1

EXPORTS = ("spark_lambda_to_T", "spark_cache_sizes", "spark_cache_bytes", "spark_workspace_bytes",
           "spark_prune", "spark_prune_noalloc", "spark_prune_grouped", "spark_group_budget", "spark_prune_values", "spark_prune_think", "spark_prune_topp", "spark_decode_attn",
           "spark_decode_attn_topp", "spark_topp_offsets_bytes", "spark_topp_vals_used",
           "spark_decode_attn_kv", "spark_workspace_bytes_kv", "spark_selftest_wait_timeout", "spark_tail_append", "spark_device_status",
           "spark_status_str", "spark_snapkv_evict", "spark_snapkv_evict_rows", "spark_pyramid_keep",
           "spark_kv8_sizes", "spark_pages_extend", "spark_pages_extend_served", "spark_pages_trim", "spark_kv8_append",
           "spark_decode_attn_kv8", "spark_workspace_bytes_kv8")


class SparkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


class spark_kcache(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hkv", ctypes.c_int), ("S", ctypes.c_int), ("D", ctypes.c_int),
                ("T", ctypes.c_int), ("dtype", ctypes.c_int), ("mask", ctypes.c_void_p),
                ("vals", ctypes.c_void_p), ("qn", ctypes.c_void_p), ("stats", ctypes.c_void_p),
                ("goff", ctypes.c_void_p), ("lens", ctypes.c_void_p)]


class spark_kv8cache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int), ("Hkv", ctypes.c_int), ("page", ctypes.c_int), ("D", ctypes.c_int),
                ("type", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


_lib = None


def lib():
    """Load libspark.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"SparK CUDA library not found at {_LIB_PATH}; build it with "
                               "`python -m channel_pruned_decode_b200.build` (no CPU fallback exists)")
        L = ctypes.CDLL(_LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.spark_lambda_to_T.argtypes = [ctypes.c_float, I]
        L.spark_lambda_to_T.restype = I
        L.spark_cache_sizes.argtypes = [I, I, I, I, I, I, ctypes.POINTER(Z)]
        L.spark_cache_sizes.restype = Z
        L.spark_cache_bytes.argtypes = [I, I, I, I, I, I]
        L.spark_cache_bytes.restype = Z
        L.spark_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
        L.spark_workspace_bytes.restype = Z
        L.spark_prune.argtypes = [P, P, I, I, ctypes.POINTER(spark_kcache), P, Z, P]
        L.spark_prune.restype = I
        L.spark_prune_noalloc.argtypes = [P, P, I, I, ctypes.POINTER(spark_kcache), P]
        L.spark_prune_noalloc.restype = I
        L.spark_prune_grouped.argtypes = [P, P, I, I, I, ctypes.POINTER(I), ctypes.POINTER(spark_kcache), P, Z, P]
        L.spark_prune_grouped.restype = I
        L.spark_group_budget.argtypes = [I, I, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(I)]
        L.spark_group_budget.restype = I
        L.spark_prune_values.argtypes = [P, ctypes.POINTER(spark_kcache), P, Z, P]
        L.spark_prune_values.restype = I
        L.spark_prune_think.argtypes = [P, P, I, I, ctypes.POINTER(spark_kcache), P, Z, P]
        L.spark_prune_think.restype = I
        L.spark_prune_topp.argtypes = [P, P, I, I, ctypes.c_float, ctypes.POINTER(spark_kcache), P, Z, P]
        L.spark_prune_topp.restype = I
        L.spark_decode_attn_topp.argtypes = [P, ctypes.POINTER(spark_kcache), P, P, P, I, I, I, I,
                                             ctypes.c_ulonglong, P, P, Z, P]
        L.spark_decode_attn_topp.restype = I
        L.spark_topp_offsets_bytes.argtypes = [I, I, I]
        L.spark_topp_offsets_bytes.restype = Z
        L.spark_topp_vals_used.argtypes = [ctypes.POINTER(spark_kcache), ctypes.POINTER(Z), P]
        L.spark_topp_vals_used.restype = I
        L.spark_selftest_wait_timeout.argtypes = [P, I, P]
        L.spark_selftest_wait_timeout.restype = I
        L.spark_decode_attn_kv.argtypes = [P, ctypes.POINTER(spark_kcache), ctypes.POINTER(spark_kcache), P, P, I,
                                           I, I, P, P, Z, P]
        L.spark_decode_attn_kv.restype = I
        L.spark_workspace_bytes_kv.argtypes = [I, I, I, I, I, I, I, I]
        L.spark_workspace_bytes_kv.restype = Z
        L.spark_decode_attn.argtypes = [P, ctypes.POINTER(spark_kcache), P, P, P, I, I, I, I,
                                        ctypes.c_ulonglong, P, P, Z, P]
        L.spark_decode_attn.restype = I
        L.spark_snapkv_evict.argtypes = [P, P, P, I, I, I, I, I, I, I, I, I, P, P, P, P, Z, P]
        L.spark_snapkv_evict.restype = I
        L.spark_snapkv_evict_rows.argtypes = [P, P, P, I, I, I, I, I, I, P, I, I, I, P, P, P, P, Z, P]
        L.spark_snapkv_evict_rows.restype = I
        L.spark_pyramid_keep.argtypes = [I, I, ctypes.c_float, I, I, ctypes.POINTER(I)]
        L.spark_pyramid_keep.restype = I
        L.spark_tail_append.argtypes = [P, P, P, P, I, I, I, I, I, I, P]
        L.spark_tail_append.restype = I
        KV8 = ctypes.POINTER(spark_kv8cache)
        L.spark_kv8_sizes.argtypes = [I, I, I, I, ctypes.POINTER(Z)]
        L.spark_kv8_sizes.restype = Z
        L.spark_pages_extend.argtypes = [P, P, I, I, P, I, P, P, I, I, P, P, P, P, Z, P]
        L.spark_pages_extend.restype = I
        L.spark_pages_extend_served.argtypes = [P, P, I, I, P, I, P, P, I, I, P, P, P, P, P, Z, P]
        L.spark_pages_extend_served.restype = I
        L.spark_pages_trim.argtypes = [P, P, I, I, P, I, P, P, I, P, P, P, Z, P]
        L.spark_pages_trim.restype = I
        L.spark_kv8_append.argtypes = [P, P, I, I, I, P, KV8, P, Z, P]
        L.spark_kv8_append.restype = I
        L.spark_decode_attn_kv8.argtypes = [P, I, KV8, P, I, P, P, I, I, I, P, P, Z, P]
        L.spark_decode_attn_kv8.restype = I
        L.spark_workspace_bytes_kv8.argtypes = [I, I, I, I]
        L.spark_workspace_bytes_kv8.restype = Z
        L.spark_device_status.argtypes = [P, ctypes.POINTER(I), I, P]
        L.spark_device_status.restype = I
        L.spark_status_str.argtypes = [I]
        L.spark_status_str.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().spark_status_str(status).decode()


def _check(rc: int, where: str):
    if rc != SPARK_OK:
        raise SparkError(rc, where)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return SPARK_BF16
    if t == torch.float32:
        return SPARK_F32
    raise ValueError(f"unsupported dtype {t}")


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ------------------------------------------------------------------ sizes
def spark_lambda_to_T(lam: float, D: int = 128) -> int:
    return int(lib().spark_lambda_to_T(ctypes.c_float(lam), D))


def spark_cache_sizes(B, Hkv, S, D, T, dtype) -> tuple[int, list[int]]:
    sizes = (ctypes.c_size_t * 4)()
    total = lib().spark_cache_sizes(B, Hkv, S, D, T, dtype, sizes)
    return int(total), [int(x) for x in sizes]


def spark_cache_bytes(B, Hkv, S, D, T, dtype) -> int:
    return int(lib().spark_cache_bytes(B, Hkv, S, D, T, dtype))


def spark_workspace_bytes(op, B, Hkv, G, S, D, T, n_tail) -> int:
    return int(lib().spark_workspace_bytes(op, B, Hkv, G, S, D, T, n_tail))


# ------------------------------------------------------------------ cache
@dataclass
class KCache:
    """Device tensors of the packed key cache (layout of include/spark.h)."""
    B: int
    Hkv: int
    S: int
    D: int
    T: int
    dtype: torch.dtype
    mask: torch.Tensor    # uint32 bits stored as int32 [B, Hkv, S, 4]
    vals: torch.Tensor    # [B, Hkv, S32 * T] interleaved by 32-token groups
    qn: torch.Tensor      # fp32 [B, Hkv, D]
    stats: torch.Tensor   # fp64 [B, Hkv, 4]
    goff: torch.Tensor = None  # SparK-p only: int32 [B * Hkv * S32 / 32 + 1] first value row per group
    lens: torch.Tensor = None  # optional int32 [B] prompt tokens per row (S is then the row stride)

    @staticmethod
    def empty(B, Hkv, S, D, T, dtype, device="cuda") -> "KCache":
        S32 = (S + 31) // 32 * 32
        return KCache(B, Hkv, S, D, T, dtype,
                      torch.empty((B, Hkv, S, 4), dtype=torch.int32, device=device),
                      torch.empty((B, Hkv, S32 * T), dtype=dtype, device=device),
                      torch.empty((B, Hkv, D), dtype=torch.float32, device=device),
                      torch.empty((B, Hkv, 4), dtype=torch.float64, device=device))

    @staticmethod
    def empty_topp(B, Hkv, S, D, Tcap, dtype, device="cuda") -> "KCache":
        """A SparK-p cache: masks, a value stream with room for Tcap slots per
        token (the most spark_prune_topp can write) and the group offsets."""
        kc = KCache.empty(B, Hkv, S, D, Tcap, dtype, device)
        kc.vals = kc.vals.reshape(-1)
        kc.goff = torch.empty((B * Hkv * ((S + 31) // 32) + 1,), dtype=torch.int32, device=device)
        return kc

    def struct(self) -> spark_kcache:
        return spark_kcache(self.B, self.Hkv, self.S, self.D, self.T, _dtype_code(self.dtype),
                            _ptr(self.mask), _ptr(self.vals), _ptr(self.qn), _ptr(self.stats),
                            _ptr(self.goff) if self.goff is not None else None,
                            _ptr(self.lens) if self.lens is not None else None)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.mask, self.vals, self.qn, self.stats))


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Zero-initialised workspace (the status word must start at zero)."""
    n = (max(nbytes, 256) + 255) // 256 * 256
    return torch.zeros(n, dtype=torch.uint8, device=device)


# ------------------------------------------------------------- entry points
def spark_prune(k: torch.Tensor, q_obs: torch.Tensor, G: int, W: int, kc: KCache,
                ws: torch.Tensor, stream=None) -> None:
    s = kc.struct()
    rc = lib().spark_prune(_ptr(k), _ptr(q_obs), G, W, ctypes.byref(s), _ptr(ws),
                           ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "spark_prune")


def spark_prune_noalloc(k: torch.Tensor, q_obs: torch.Tensor, G: int, W: int, kc: KCache,
                        stream=None) -> None:
    """spark_prune for callers that cannot allocate a workspace: the library's
    fixed 4 MiB per-device scratch array stands in for it (see spark.h)."""
    s = kc.struct()
    rc = lib().spark_prune_noalloc(_ptr(k), _ptr(q_obs), G, W, ctypes.byref(s), _stream(stream))
    _check(rc, "spark_prune_noalloc")


def spark_prune_grouped(k: torch.Tensor, q_obs: torch.Tensor, G: int, W: int, group_T, kc: KCache,
                        ws: torch.Tensor, stream=None) -> None:
    """SparK-g: per-group kept-channel budgets group_T (host list, one entry
    per group, sum == kc.T); groups by window-query norm rank (see spark.h)."""
    tg = (ctypes.c_int * len(group_T))(*[int(x) for x in group_T])
    s = kc.struct()
    rc = lib().spark_prune_grouped(_ptr(k), _ptr(q_obs), G, W, len(group_T), tg, ctypes.byref(s), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "spark_prune_grouped")


def spark_prune_think(k: torch.Tensor, q_obs: torch.Tensor, G: int, W: int, kc: KCache, ws: torch.Tensor,
                      stream=None) -> None:
    """ThinK structured pruning (comparator): one channel mask per head (see spark.h)."""
    s = kc.struct()
    rc = lib().spark_prune_think(_ptr(k), _ptr(q_obs), G, W, ctypes.byref(s), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "spark_prune_think")


def spark_prune_topp(k: torch.Tensor, q_obs: torch.Tensor, G: int, W: int, p: float, kc: KCache,
                     ws: torch.Tensor, stream=None) -> None:
    """SparK-p: per token the fewest greedy-order channels whose saliency mass
    reaches p of the total, at most kc.T of them (see spark.h)."""
    s = kc.struct()
    rc = lib().spark_prune_topp(_ptr(k), _ptr(q_obs), G, W, ctypes.c_float(p), ctypes.byref(s), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "spark_prune_topp")


def spark_topp_offsets_bytes(B: int, Hkv: int, S: int) -> int:
    return int(lib().spark_topp_offsets_bytes(B, Hkv, S))


def spark_topp_vals_used(kc: KCache, stream=None) -> int:
    """Bytes of kc.vals the last spark_prune_topp used (synchronises the stream)."""
    s = kc.struct()
    n = ctypes.c_size_t(0)
    _check(lib().spark_topp_vals_used(ctypes.byref(s), ctypes.byref(n), _stream(stream)), "spark_topp_vals_used")
    return int(n.value)


def spark_decode_attn_topp(q: torch.Tensor, kc: KCache, v: torch.Tensor, k_tail, v_tail, tail_cap: int,
                           n_tail: int, G: int, out: torch.Tensor, ws: torch.Tensor,
                           recovery: int = SPARK_F_DEGENERATE, seed: int = 0, stream=None) -> None:
    """spark_decode_attn over a SparK-p cache (masks with at most kc.T bits)."""
    s = kc.struct()
    rc = lib().spark_decode_attn_topp(_ptr(q), ctypes.byref(s), _ptr(v), _ptr(k_tail), _ptr(v_tail), tail_cap,
                                      n_tail, G, recovery, seed, _ptr(out), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "spark_decode_attn_topp")


def spark_selftest_wait_timeout(ws: torch.Tensor, limit_us: int, stream=None) -> None:
    """Make one bounded device wait run out on purpose (status word test)."""
    _check(lib().spark_selftest_wait_timeout(_ptr(ws), limit_us, _stream(stream)), "spark_selftest_wait_timeout")


def spark_prune_values(v: torch.Tensor, vc: KCache, ws: torch.Tensor, stream=None) -> None:
    """Value-channel pruning: top-vc.T channels of |v| per token (see spark.h)."""
    s = vc.struct()
    rc = lib().spark_prune_values(_ptr(v), ctypes.byref(s), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream))
    _check(rc, "spark_prune_values")


def spark_decode_attn_kv(q: torch.Tensor, kc: KCache, vc: KCache, k_tail, v_tail, tail_cap: int, n_tail: int,
                         G: int, out: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    sk, sv = kc.struct(), vc.struct()
    rc = lib().spark_decode_attn_kv(_ptr(q), ctypes.byref(sk), ctypes.byref(sv), _ptr(k_tail), _ptr(v_tail),
                                    tail_cap, n_tail, G, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream))
    _check(rc, "spark_decode_attn_kv")


def spark_workspace_bytes_kv(B: int, Hkv: int, G: int, S: int, D: int, T: int, Tv: int, n_tail: int) -> int:
    return int(lib().spark_workspace_bytes_kv(B, Hkv, G, S, D, T, Tv, n_tail))


def spark_group_budget(D: int, rates) -> list:
    """Per-group kept-channel budgets of SparK-g (the C library's
    spark_group_budget): round((1 - rate) * group size), half away from zero,
    for len(rates) equal-rank groups of D channels."""
    g = len(rates)
    arr = (ctypes.c_float * max(g, 1))(*[float(r) for r in rates])
    out = (ctypes.c_int * max(g, 1))()
    _check(lib().spark_group_budget(D, g, arr, out), "spark_group_budget")
    return [int(out[q]) for q in range(g)]


def spark_decode_attn(q: torch.Tensor, kc: KCache, v: torch.Tensor, k_tail, v_tail, tail_cap: int,
                      n_tail: int, G: int, out: torch.Tensor, ws: torch.Tensor,
                      recovery: int = SPARK_F_DEGENERATE, seed: int = 0, stream=None) -> None:
    s = kc.struct()
    rc = lib().spark_decode_attn(_ptr(q), ctypes.byref(s), _ptr(v), _ptr(k_tail), _ptr(v_tail), tail_cap,
                                 n_tail, G, recovery, seed, _ptr(out), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "spark_decode_attn")


def spark_snapkv_evict(k: torch.Tensor, v: torch.Tensor, q_obs: torch.Tensor, G: int, W: int, keep: int,
                       pool: int, k_out: torch.Tensor, v_out: torch.Tensor, idx_out: torch.Tensor,
                       ws: torch.Tensor, stream=None) -> None:
    """SnapKV-style eviction: k, v [B, Hkv, S, D] -> k_out, v_out [B, Hkv, keep, D],
    idx_out int32 [B, Hkv, keep]."""
    B, H, S, D = k.shape
    rc = lib().spark_snapkv_evict(_ptr(k), _ptr(v), _ptr(q_obs), B, H, S, D, G, W, keep, pool,
                                  _dtype_code(k.dtype), _ptr(k_out), _ptr(v_out), _ptr(idx_out), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "spark_snapkv_evict")


def spark_snapkv_evict_rows(k: torch.Tensor, v: torch.Tensor, q_obs: torch.Tensor, G: int, W: int,
                            keep_rows: torch.Tensor, keep_cap: int, pool: int, k_out: torch.Tensor,
                            v_out: torch.Tensor, idx_out: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """SnapKV-style eviction with one budget per row (keep_rows: int32 [B] on
    the device); outputs with row stride keep_cap (see spark.h)."""
    B, Hkv, S, D = k.shape
    rc = lib().spark_snapkv_evict_rows(_ptr(k), _ptr(v), _ptr(q_obs), B, Hkv, S, D, G, W, _ptr(keep_rows),
                                       keep_cap, pool, _dtype_code(k.dtype), _ptr(k_out), _ptr(v_out),
                                       _ptr(idx_out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "spark_snapkv_evict_rows")


def spark_pyramid_keep(L: int, M: int, beta: float, W: int, S: int) -> list:
    """PyramidKV-style layer budgets around the mean M (the library's linear
    reading, see spark.h)."""
    out = (ctypes.c_int * max(L, 1))()
    _check(lib().spark_pyramid_keep(L, M, ctypes.c_float(beta), W, S, out), "spark_pyramid_keep")
    return [int(out[i]) for i in range(L)]


def spark_tail_append(k_new, v_new, k_tail, v_tail, B, Hkv, D, tail_cap, slot, stream=None) -> None:
    rc = lib().spark_tail_append(_ptr(k_new), _ptr(v_new), _ptr(k_tail), _ptr(v_tail), B, Hkv, D,
                                 tail_cap, slot, _dtype_code(k_new.dtype), _stream(stream))
    _check(rc, "spark_tail_append")


# ------------------------------------------------------ paged 8-bit cache
@dataclass(frozen=True)
class KV8Cache:
    """Device tensors of the paged 8-bit cache (layout of include/spark.h).
    Frozen: the descriptor that the calls pass is made once, here."""
    n_pages: int
    Hkv: int
    page: int             # tokens per page: 16, 32, 64 or 128
    D: int
    type: int             # SPARK_KV8_E4M3 or SPARK_KV8_I8
    k: torch.Tensor       # uint8 [n_pages, Hkv, page, D]
    v: torch.Tensor       # uint8 [n_pages, Hkv, page, D]
    k_scale: torch.Tensor  # fp32 [n_pages, Hkv]
    v_scale: torch.Tensor  # fp32 [n_pages, Hkv]

    def __post_init__(self):
        codes, scales = (self.n_pages, self.Hkv, self.page, self.D), (self.n_pages, self.Hkv)
        for name, t, shape, dt in (("k", self.k, codes, torch.uint8), ("v", self.v, codes, torch.uint8),
                                   ("k_scale", self.k_scale, scales, torch.float32),
                                   ("v_scale", self.v_scale, scales, torch.float32)):
            _need(t, name, dt, shape, self.k.device)
        desc = spark_kv8cache(self.n_pages, self.Hkv, self.page, self.D, self.type, _ptr(self.k), _ptr(self.v),
                              _ptr(self.k_scale), _ptr(self.v_scale))
        object.__setattr__(self, "_struct", desc)
        object.__setattr__(self, "address", ctypes.addressof(desc))
        object.__setattr__(self, "index", self.k.get_device())

    @staticmethod
    def empty(n_pages, Hkv, page, type=SPARK_KV8_E4M3, D=128, device="cuda") -> "KV8Cache":
        codes = [torch.empty((n_pages, Hkv, page, D), dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.empty((n_pages, Hkv), dtype=torch.float32, device=device) for _ in range(2)]
        return KV8Cache(n_pages, Hkv, page, D, type, *codes, *scales)

    def struct(self) -> spark_kv8cache:
        return self._struct

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scale, self.v_scale))


def _need(t: torch.Tensor, name: str, dtype, shape, device) -> None:
    """The library sees bare pointers: a tensor of another type, shape, layout
    or device than the call needs is refused.  (csrc/calls.cpp tests the calls'
    tensors; where one does not fit, this says which and why.)"""
    if t.dtype != dtype:
        raise ValueError(f"{name}: {dtype} needed, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} needed, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the call's other tensors are on {device}")


def _refuse(where: str, ws: torch.Tensor, device, *tensors) -> None:
    """A call whose tensors do not fit: say which (name, tensor, dtype, shape)."""
    for name, t, dtype, shape in tensors:
        _need(t, name, dtype, shape, device)
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws: must be contiguous and on {device}")
    raise ValueError(f"{where}: tensors must be on the current CUDA device, whole numbers must fit 32 bits")


_calls = None


def _native():
    """The compiled half of the calls below (raises if it has not been built)."""
    global _calls
    if _calls is None:
        lib()
        try:
            from . import _calls as m
        except ImportError as e:
            raise RuntimeError("the compiled binding (_calls.so) is missing or does not fit this Python; build it with "
                               "`python -m channel_pruned_decode_b200.build`") from e
        from .build import calls_tag
        if m.built_for != calls_tag():
            raise RuntimeError(f"the compiled binding (_calls.so) was built for {m.built_for}, this is {calls_tag()}; "
                               "build it again with `python -m channel_pruned_decode_b200.build`")
        _calls = m
    return _calls


def _raw(stream):
    """A stream as the compiled calls take it: None for the current one."""
    return stream if stream is None else _stream(stream)


def spark_kv8_sizes(n_pages: int, Hkv: int, page: int, D: int = 128) -> tuple[int, list[int]]:
    sizes = (ctypes.c_size_t * 4)()
    total = lib().spark_kv8_sizes(n_pages, Hkv, page, D, sizes)
    return int(total), [int(x) for x in sizes]


def spark_pages_extend(lens: torch.Tensor, n_new: torch.Tensor, page: int, pool: torch.Tensor, taken: torch.Tensor,
                       table: torch.Tensor, slots: torch.Tensor, lens_out: torch.Tensor, taken_out: torch.Tensor,
                       ws: torch.Tensor, stream=None, n_served: torch.Tensor = None) -> None:
    """Pages for each row's n_new tokens (table [B, cap] and taken_out) and
    their slots [B, n_cap]; lens_out / taken_out may be lens / taken.
    n_served [B], an array of its own, gets the number of tokens that each row
    got (fewer than n_new where the pool ran out): what the step's attention
    takes as n_new (spark_pages_extend_served of include/spark.h)."""
    rc = _native().pages_extend(lens, n_new, page, pool, taken, table, slots, lens_out, taken_out, ws, _raw(stream),
                                n_served)
    if rc < 0:
        i32, B = torch.int32, lens.shape[0]
        _refuse("spark_pages_extend", ws, lens.device, ("lens", lens, i32, (B,)), ("n_new", n_new, i32, (B,)),
                ("pool", pool, i32, (pool.numel(),)), ("taken", taken, i32, (1,)),
                ("table", table, i32, (B, table.shape[-1])), ("slots", slots, i32, (B, slots.shape[-1])),
                ("lens_out", lens_out, i32, (B,)), ("taken_out", taken_out, i32, (1,)),
                *([] if n_served is None else [("n_served", n_served, i32, (B,))]))
    if rc:
        _check(rc, "spark_pages_extend")


def spark_pages_trim(lens: torch.Tensor, keep: torch.Tensor, page: int, pool: torch.Tensor, taken: torch.Tensor,
                     table: torch.Tensor, lens_out: torch.Tensor, taken_out: torch.Tensor, ws: torch.Tensor,
                     stream=None) -> None:
    """Cut each row to its first keep tokens and give the pages behind them
    back to the pool; lens_out / taken_out may be lens / taken."""
    rc = _native().pages_trim(lens, keep, page, pool, taken, table, lens_out, taken_out, ws, _raw(stream))
    if rc < 0:
        i32, B = torch.int32, lens.shape[0]
        _refuse("spark_pages_trim", ws, lens.device, ("lens", lens, i32, (B,)), ("keep", keep, i32, (B,)),
                ("pool", pool, i32, (pool.numel(),)), ("taken", taken, i32, (1,)),
                ("table", table, i32, (B, table.shape[-1])), ("lens_out", lens_out, i32, (B,)),
                ("taken_out", taken_out, i32, (1,)))
    if rc:
        _check(rc, "spark_pages_trim")


def spark_kv8_append(k_new: torch.Tensor, v_new: torch.Tensor, slots: torch.Tensor, kc: KV8Cache, ws: torch.Tensor,
                     stream=None) -> None:
    """Write k_new, v_new [B, Hkv, n_cap, D] into the slots [B, n_cap] in 8
    bits ([B, Hkv, D] with n_cap = 1)."""
    rc = _native().kv8_append(k_new, v_new, slots, kc.address, kc.index, ws, _raw(stream))
    if rc < 0:
        B, n_cap = slots.shape
        _dtype_code(k_new.dtype)
        shape = (B, kc.Hkv, kc.D) if n_cap == 1 and k_new.dim() == 3 else (B, kc.Hkv, n_cap, kc.D)
        _refuse("spark_kv8_append", ws, kc.k.device, ("k_new", k_new, k_new.dtype, shape),
                ("v_new", v_new, k_new.dtype, shape), ("slots", slots, torch.int32, (B, n_cap)))
    if rc:
        _check(rc, "spark_kv8_append")


def spark_decode_attn_kv8(q: torch.Tensor, kc: KV8Cache, table: torch.Tensor, lens: torch.Tensor, G: int,
                          out: torch.Tensor, ws: torch.Tensor, n_new: torch.Tensor = None, stream=None) -> None:
    """Attention of q [B, Hkv*G, n_q, D] (or [B, Hkv*G, D]), each row's newest
    tokens, over its pages; out fp32, shaped like q."""
    rc = _native().decode_attn_kv8(q, kc.address, kc.index, table, lens, G, out, ws, n_new, _raw(stream))
    if rc < 0:
        i32, (B, cap) = torch.int32, table.shape
        _dtype_code(q.dtype)
        shape = (B, kc.Hkv * G, q.shape[2], kc.D) if q.dim() == 4 else (B, kc.Hkv * G, kc.D)
        _refuse("spark_decode_attn_kv8", ws, kc.k.device, ("q", q, q.dtype, shape), ("out", out, torch.float32, shape),
                ("table", table, i32, (B, cap)), ("lens", lens, i32, (B,)),
                *([] if n_new is None else [("n_new", n_new, i32, (B,))]))
    if rc:
        _check(rc, "spark_decode_attn_kv8")


def spark_workspace_bytes_kv8(B: int, Hkv: int, G: int, n_q: int = 1) -> int:
    return int(lib().spark_workspace_bytes_kv8(B, Hkv, G, n_q))


def spark_device_status(ws: torch.Tensor, clear: bool = False, stream=None) -> int:
    st = ctypes.c_int(0)
    rc = lib().spark_device_status(_ptr(ws), ctypes.byref(st), int(clear), _stream(stream))
    _check(rc, "spark_device_status")
    return st.value
