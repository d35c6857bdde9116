"""Cases of the paged 8-bit cache's operators: page tables and slot maps built
on the GPU (spark_pages_extend, spark_pages_trim), the write into the cache
(spark_kv8_append) and the attention that reads it (spark_decode_attn_kv8).

A cache is a pool of pages; a page holds `page` tokens of every kv head, each
value in 8 bits (e4m3 or int8), with one power-of-two scale per (page, kv
head) for keys and one for values.  The plain forms below compute the same
results with elementary torch operations.
"""
import random

import torch

own = False

D = 128
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of a serving batch: every request gets one token, some a new page
        dict(name="extend step", op="extend", B=64, page=16, n=1, lo=1, hi=16384),
        # a batch of prompts arrives: empty requests of ragged length get all their pages
        dict(name="extend prompts", op="extend", B=256, page=16, n=8192, lo=0, hi=0),
        # draft tokens that the model rejected are taken back after a verify step
        dict(name="trim drafts", op="trim", B=64, page=16, n=4, lo=1, hi=16384),
        # a quarter of a large batch has ended and gives its pages back
        dict(name="trim ended", op="trim", B=512, page=32, n=0, lo=1024, hi=32768),
        # the new token of each request of a decode batch
        dict(name="append step", op="append", B=32, Hkv=8, page=16, n=1, kv="e4m3", dtype="bf16"),
        # what an eviction kept of each prompt: 2048 tokens of 32 requests
        dict(name="append prompts", op="append", B=32, Hkv=8, page=32, n=2048, kv="e4m3", dtype="bf16"),
        # odd chunks of a few long prompts, in fp32
        dict(name="append chunks", op="append", B=5, Hkv=4, page=64, n=1777, kv="i8", dtype="f32"),
        # the smallest decode: two kv heads of one short request, fp32
        dict(name="attn small", op="attn", B=1, Hkv=2, G=4, n=1, page=16, lo=512, hi=512, kv="i8", dtype="f32"),
        # decode of the requests that an eviction cut to 2048 tokens
        dict(name="attn batch", op="attn", B=32, Hkv=8, G=4, n=1, page=16, lo=2048, hi=2304, kv="e4m3", dtype="bf16"),
        # one request with a long context
        dict(name="attn long", op="attn", B=1, Hkv=8, G=4, n=1, page=32, lo=131072, hi=131072, kv="e4m3", dtype="bf16"),
        # a verify step: four tokens of each request at once
        dict(name="attn verify", op="attn", B=8, Hkv=8, G=4, n=4, page=16, lo=16384, hi=16384, kv="e4m3", dtype="bf16"),
        # a large batch whose lengths differ widely, larger groups of query heads
        dict(name="attn ragged", op="attn", B=48, Hkv=8, G=8, n=1, page=64, lo=17, hi=32768, kv="i8", dtype="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["extend", "trim", "append", "append", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "extend":
        B = _between(rng, 1, 512)
        n = _between(rng, 1, 8192 * 256 // max(B, 256))
        return dict(op=op, B=B, page=page, n=n, lo=0, hi=_between(rng, 1, 16384))
    if op == "trim":
        return dict(op=op, B=_between(rng, 1, 512), page=page, n=rng.choice([0, 4, 8, 16]), lo=0,
                    hi=_between(rng, 16, 32768))
    kv, dtype = rng.choice(["e4m3", "i8"]), rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        B = _between(rng, 1, 256)
        n = _between(rng, 1, max(1, 32 * 2048 * (4 if dtype == "bf16" else 2) // (B * Hkv)))
        return dict(op=op, B=B, Hkv=Hkv, page=page, n=min(n, 16384), kv=kv, dtype=dtype)
    Hkv, G, n = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 1, 1, 2, 3, 4])
    B = _between(rng, 1, 128)
    hi = _between(rng, 33, min(131072, max(64, 2 * 8 * 131072 // (B * Hkv))))
    return dict(op=op, B=B, Hkv=Hkv, G=G, n=n, page=page, lo=_between(rng, 1, hi), hi=hi, kv=kv, dtype=dtype)


# ------------------------------------------------------------------ inputs
def _host(case):
    """Lengths come from the case alone, so that its work is known; values and
    the order of the pages come from the seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _spread(rng, B, lo, hi):
    """B lengths spread evenly over [lo, hi], in random order."""
    v = [lo + (hi - lo) * (2 * i + 1) // (2 * B) if B > 1 else hi for i in range(B)]
    rng.shuffle(v)
    return v


def _lengths(case):
    """(tokens held, new tokens) of each request."""
    rng, B, n = _host(case), case["B"], case["n"]
    op = case["op"]
    if op == "attn":
        held = _spread(rng, B, case["lo"], case["hi"])
        # a verify step's requests bring different numbers of tokens
        return held, [min(x, n if n == 1 else rng.randint(1, n)) for x in held]
    if op == "append":
        # a step of one token lands anywhere in a page; longer ones are ragged
        new = [1] * B if n == 1 else [n if B == 1 or i % 4 else rng.randint(1, n) for i in range(B)]
        return [rng.randrange(case["page"]) for _ in range(B)], new
    held = _spread(rng, B, case["lo"], case["hi"])
    if op == "extend":
        return held, [1] * B if n == 1 else [rng.randint(n // 4, n) for _ in range(B)]
    if n:  # drafts: up to n tokens of each request are taken back
        return held, [max(0, x - rng.randint(0, n)) for x in held]
    return held, [0 if i % 4 == 0 else x for i, x in enumerate(held)]


def _pages(n, page):
    return -(-n // page)


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _codes(x, kv):
    """8-bit codes (as bytes) and power-of-two scales of x [pages, Hkv, page, D]."""
    a = x.abs().amax(dim=(2, 3))
    top = 448.0 if kv == "e4m3" else 127.0
    scale = torch.exp2(torch.ceil(torch.log2(a / top)))
    y = x / scale[:, :, None, None]
    if kv == "e4m3":
        return y.clamp_(-top, top).to(torch.float8_e4m3fn).view(torch.uint8), scale
    return y.round_().clamp_(-top, top).to(torch.int8).view(torch.uint8), scale


def _cache(case, n_pages, gen, dev):
    """A cache of n_pages pages that hold keys or values with per-channel
    magnitudes, and one spare page after them where the plain form puts what
    a padded place would write."""
    H, P = case["Hkv"], case["page"]
    out = []
    for _ in range(2):
        c = torch.empty((n_pages + 1, H, P, D), dtype=torch.uint8, device=dev)
        s = torch.empty((n_pages + 1, H), dtype=torch.float32, device=dev)
        by_channel = torch.exp(0.3 * torch.randn((H, 1, D), generator=gen, device=dev))
        step = max(1, (1 << 27) // (H * P * D))
        for i in range(0, n_pages + 1, step):
            j = min(n_pages + 1, i + step)
            x = torch.randn((j - i, H, P, D), generator=gen, device=dev).mul_(by_channel)
            c[i:j], s[i:j] = _codes(x, case["kv"])
        out += [c, s]
    return out


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, B, P = case["op"], case["B"], case["page"]
    held, other = _lengths(case)
    s = {"op": op, "case": dict(case), "lens": _ints(held, dev), "other": _ints(other, dev)}
    if op in ("extend", "trim"):
        have = [_pages(x, P) for x in held]
        most = max([_pages(x + y, P) for x, y in zip(held, other)] if op == "extend" else have) if B else 0
        cap = max(1, most)
        total = sum(_pages(x + y, P) for x, y in zip(held, other)) if op == "extend" else sum(have)
        ids = torch.randperm(total + 64, generator=gen, device=dev).to(torch.int32)
        first = torch.tensor([0] + have[:-1], device=dev).cumsum(0)
        at = torch.arange(cap, device=dev)
        mine = at[None] < torch.tensor(have, device=dev)[:, None]
        table = torch.where(mine, ids[(first[:, None] + at[None]).clamp(max=ids.numel() - 1)], -1).to(torch.int32)
        s.update(pool=ids, taken=_ints([sum(have)], dev), table=table.contiguous(),
                 lens_out=torch.zeros_like(s["lens"]), taken_out=_ints([0], dev))
        if op == "extend":
            s["slots"] = torch.zeros((B, case["n"]), dtype=torch.int32, device=dev)
        return s
    H, n = case["Hkv"], case["n"]
    s["page"], s["kv"] = P, case["kv"]
    if op == "append":
        need = [_pages(x + y, P) for x, y in zip(held, other)]
        n_pages, cap = sum(need) + 8, max(need)
    else:
        need = [_pages(x, P) for x in held]
        n_pages, cap = sum(need) + 8, max(1, max(need))
    s["n_pages"] = n_pages
    ids = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    first = torch.tensor([0] + need[:-1], device=dev).cumsum(0)
    at = torch.arange(cap, device=dev)
    mine = at[None] < torch.tensor(need, device=dev)[:, None]
    table = torch.where(mine, ids[(first[:, None] + at[None]).clamp(max=n_pages - 1)], 0).to(torch.int32).contiguous()
    s["k"], s["ks"], s["v"], s["vs"] = _cache(case, n_pages, gen, dev)
    if op == "append":
        j = torch.arange(n, device=dev)
        pos = s["lens"][:, None].long() + j[None]
        page_of = torch.gather(table.long(), 1, (pos // P).clamp(max=cap - 1))
        s["slots"] = torch.where(j[None] < s["other"][:, None], page_of * P + pos % P, -1).to(torch.int32).contiguous()
        for name in ("k_new", "v_new"):
            x = torch.randn((B, H, n, D), generator=gen, device=dev)
            x *= torch.exp(0.3 * torch.randn((H, 1, D), generator=gen, device=dev))
            s[name] = x.to(TYPES[case["dtype"]])
        return s
    s["table"] = table
    s["G"], s["n"] = case["G"], n
    s["q"] = torch.randn((B, H * case["G"], n, D), generator=gen, device=dev).to(TYPES[case["dtype"]])
    s["out"] = torch.zeros((B, H * case["G"], n, D), dtype=torch.float32, device=dev)
    return s


# -------------------------------------------------------------- plain forms
def _plain_extend(s):
    P, table, slots = s["case"]["page"], s["table"], s["slots"]
    lens, new = s["lens"].long(), s["other"].long()
    have, want = (lens + P - 1) // P, (lens + new + P - 1) // P
    add = want - have
    base = s["taken"].long() + add.cumsum(0) - add
    at = torch.arange(table.shape[1], device=table.device)
    fresh = (at[None] >= have[:, None]) & (at[None] < want[:, None])
    src = (base[:, None] + at[None] - have[:, None]).clamp(0, s["pool"].numel() - 1)
    table.copy_(torch.where(fresh, s["pool"][src], table))
    j = torch.arange(slots.shape[1], device=table.device)
    pos = lens[:, None] + j[None]
    page_of = torch.gather(table, 1, (pos // P).clamp(max=table.shape[1] - 1)).long()
    slots.copy_(torch.where(j[None] < new[:, None], page_of * P + pos % P, -1))
    s["lens_out"].copy_(lens + new)
    s["taken_out"].copy_(s["taken"] + add.sum())
    return {"table": table, "slots": slots, "lens": s["lens_out"], "taken": s["taken_out"]}


def _plain_trim(s):
    P, table, pool = s["case"]["page"], s["table"], s["pool"]
    lens = s["lens"].long()
    keep = torch.minimum(lens, s["other"].long())
    have, left = (lens + P - 1) // P, (keep + P - 1) // P
    give = have - left
    base = s["taken"].long() - give.sum() + give.cumsum(0) - give
    at = torch.arange(table.shape[1], device=table.device)
    back = (at[None] >= left[:, None]) & (at[None] < have[:, None])
    # places that give nothing back write pool entry n - 1 with its own value
    n = pool.numel()
    dst = torch.where(back, base[:, None] + at[None] - left[:, None], n - 1)
    pool.scatter_(0, dst.reshape(-1), torch.where(back, table, pool[n - 1]).reshape(-1))
    s["lens_out"].copy_(keep)
    s["taken_out"].copy_(s["taken"] - give.sum())
    return {"pool": pool, "lens": s["lens_out"], "taken": s["taken_out"]}


def _values(code, kv):
    return code.view(torch.float8_e4m3fn if kv == "e4m3" else torch.int8).to(torch.float32)


def _round8(y, kv):
    if kv == "e4m3":
        return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return y.round().clamp(-127.0, 127.0).to(torch.int8).view(torch.uint8)


def _plain_write(x, codes, scale, slots, P, kv):
    B, H, n, _ = x.shape
    spare = codes.shape[0] - 1
    x = x.float()
    j = torch.arange(n, device=x.device)
    valid = slots >= 0
    slot = slots.long().clamp(min=0)
    off0 = slot[:, 0] % P
    nth = (off0[:, None] + j[None]) // P  # which of its row's pages a token is in
    n_pages = (n + P - 2) // P + 1
    a = torch.where(valid[:, None], x.abs().amax(-1), 0.0)
    top = torch.zeros((B, H, n_pages), device=x.device).scatter_reduce_(2, nth[:, None].expand(B, H, n), a, "amax")
    # a = m 2^e with m in [0.5, 1): the scale's exponent is the least with a <= 2^E 448 (or 127)
    m, e = torch.frexp(top)
    e = (e - 9 + (m > 0.875).int()) if kv == "e4m3" else (e - 7 + (m > 127 / 128).int())
    e = torch.where(top > 0, e, -126).clamp(-126, 120)
    new = torch.ldexp(torch.ones_like(top), e)
    page = torch.where(valid, slot // P, spare)
    # the tokens that the first page already holds keep their values on the larger scale
    p0 = page[:, 0]
    inside = valid[:, 0] & (off0 > 0)
    old = scale[p0]
    new[:, :, 0] = torch.where(inside[:, None], torch.maximum(new[:, :, 0], old), new[:, :, 0])
    before = codes[p0]
    ratio = (old / new[:, :, 0])[:, :, None, None]
    again = _round8(_values(before, kv) * ratio, kv)
    held = (inside[:, None] & (torch.arange(P, device=x.device)[None] < off0[:, None]))[:, None, :, None]
    codes[p0] = torch.where(held, again, before)
    per_token = torch.gather(new, 2, nth[:, None].expand(B, H, n))
    code = _round8(x / per_token[..., None], kv)
    off = slot % P
    h = torch.arange(H, device=x.device)
    codes[page[:, None, :], h[None, :, None], off[:, None, :]] = code
    scale[page[:, None, :], h[None, :, None]] = per_token
    return codes[:-1].view(torch.float8_e4m3fn if kv == "e4m3" else torch.int8), scale[:-1]


def _plain_append(s):
    k, ks = _plain_write(s["k_new"], s["k"], s["ks"], s["slots"], s["page"], s["kv"])
    v, vs = _plain_write(s["v_new"], s["v"], s["vs"], s["slots"], s["page"], s["kv"])
    return {"k": k, "k_scale": ks, "v": v, "v_scale": vs}


def _plain_attn(s):
    G, n, P = s["G"], s["n"], s["page"]
    table = s["table"].long()
    B, cap = table.shape
    q = s["q"].float()
    H = q.shape[1] // G

    def dense(codes, scale):
        x = _values(codes[table], s["kv"]) * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, cap * P, D)

    x = q.reshape(B, H, G * n, D) @ dense(s["k"], s["ks"]).transpose(2, 3) * D ** -0.5
    lens, new = s["lens"].long(), s["other"].long()
    i = torch.arange(n, device=q.device)
    pos = (lens - new)[:, None] + i[None]  # where each query stands
    t = torch.arange(cap * P, device=q.device)
    seen = (t[None, None] <= pos[..., None]) & (t[None, None] < lens[:, None, None])  # [B, n, T]
    seen = seen[:, None, None].expand(B, H, G, n, cap * P).reshape(B, H, G * n, cap * P)
    x = torch.where(seen, x, -torch.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(m), m, 0.0))
    l = p.sum(-1, keepdim=True)
    o = torch.where(l > 0, (p @ dense(s["v"], s["vs"])) / l, 0.0).reshape(B, H * G, n, D)
    s["out"].copy_(torch.where((i[None] < new[:, None])[:, None, :, None], o, s["out"]))
    return s["out"]


# ------------------------------------------------------- the framework's own
def _own_handle(s):
    """What a program keeps beside its buffers: the cache's descriptor and a workspace."""
    import channel_pruned_decode_b200 as sp
    dev = s["lens"].device
    h = {"sp": sp, "ws": sp.workspace(256, device=dev)}
    if s["op"] in ("append", "attn"):
        c, n = s["case"], s["n_pages"]
        kind = sp.SPARK_KV8_E4M3 if s["kv"] == "e4m3" else sp.SPARK_KV8_I8
        h["cache"] = sp.KV8Cache(n, c["Hkv"], s["page"], D, kind, s["k"][:n], s["v"][:n], s["ks"][:n], s["vs"][:n])
        as_type = torch.float8_e4m3fn if s["kv"] == "e4m3" else torch.int8
        h["k"], h["v"] = s["k"][:n].view(as_type), s["v"][:n].view(as_type)
        if s["op"] == "attn":
            h["ws"] = sp.workspace(sp.spark_workspace_bytes_kv8(c["B"], c["Hkv"], s["G"], s["n"]), device=dev)
    s["handle"] = h
    return h


def _own_run(s):
    h = s.get("handle") or _own_handle(s)
    sp, op = h["sp"], s["op"]
    if op == "extend":
        sp.spark_pages_extend(s["lens"], s["other"], s["case"]["page"], s["pool"], s["taken"], s["table"], s["slots"],
                              s["lens_out"], s["taken_out"], h["ws"])
        return {"table": s["table"], "slots": s["slots"], "lens": s["lens_out"], "taken": s["taken_out"]}
    if op == "trim":
        sp.spark_pages_trim(s["lens"], s["other"], s["case"]["page"], s["pool"], s["taken"], s["table"],
                            s["lens_out"], s["taken_out"], h["ws"])
        return {"pool": s["pool"], "lens": s["lens_out"], "taken": s["taken_out"]}
    c = h["cache"]
    if op == "append":
        sp.spark_kv8_append(s["k_new"], s["v_new"], s["slots"], c, h["ws"])
        return {"k": h["k"], "k_scale": c.k_scale, "v": h["v"], "v_scale": c.v_scale}
    sp.spark_decode_attn_kv8(s["q"], c, s["table"], s["lens"], s["G"], s["out"], h["ws"], n_new=s["other"])
    return s["out"]


_PLAIN = {"extend": _plain_extend, "trim": _plain_trim, "append": _plain_append, "attn": _plain_attn}


def run(state):
    return _own_run(state) if own else _PLAIN[state["op"]](state)


# --------------------------------------------------------------------- work
def work(case):
    held, other = _lengths(case)
    B, P, op = case["B"], case["page"], case["op"]
    if op == "extend":
        add = sum(_pages(x + y, P) - _pages(x, P) for x, y in zip(held, other))
        # lengths in and out, the pages from the pool to the table, the slot map
        return {"bytes": 12 * B + 8 * add + 4 * B * case["n"], "flops": 0}
    if op == "trim":
        give = sum(_pages(x, P) - _pages(min(x, y), P) for x, y in zip(held, other))
        return {"bytes": 12 * B + 8 * give, "flops": 0}
    H = case["Hkv"]
    es = TYPES[case["dtype"]].itemsize
    if op == "append":
        N = sum(other)
        pages = sum(_pages(x + y, P) - x // P for x, y in zip(held, other))
        # new keys and values in, their codes and the touched pages' scales out, the slot map
        return {"bytes": 2 * N * H * D * (es + 1) + 8 * pages * H + 4 * B * case["n"], "flops": 0}
    T, rows = sum(held), sum(other) * case["G"]
    pages = sum(_pages(x, P) for x in held)
    return {"bytes": 2 * T * H * D + 8 * pages * H + 4 * pages + H * rows * D * (es + 4),
            "flops": 4 * H * D * case["G"] * sum(x * y for x, y in zip(held, other))}


# -------------------------------------------------------------------- exact
def _e4m3_exact(y):
    """The nearest e4m3 number to each y (fp64), ties to the even one."""
    mag = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * torch.round(mag / step) * step


def _exact_write(s, x, codes, scale):
    """Row by row and page by page, in fp64."""
    kv, P = s["kv"], s["page"]
    top = 448.0 if kv == "e4m3" else 127.0
    near = _e4m3_exact if kv == "e4m3" else torch.round
    val = (codes.view(torch.float8_e4m3fn) if kv == "e4m3" else codes.view(torch.int8)).double()
    scale = scale.double()
    slots = s["slots"].tolist()
    for b, row in enumerate(slots):
        j = 0
        while j < len(row) and row[j] >= 0:
            pg, off = divmod(row[j], P)
            cnt = 1
            while j + cnt < len(row) and row[j + cnt] == row[j] + cnt and off + cnt < P:
                cnt += 1
            y = x[b, :, j:j + cnt].double()
            a = y.abs().amax((1, 2))
            want = torch.exp2(torch.round(torch.log2((a / top).clamp(min=2.0 ** -126))))
            want = torch.where(want * top < a, 2 * want, want)  # the least power of two that reaches a
            want = torch.where((want / 2 * top >= a) & (want > 2.0 ** -126), want / 2, want)
            if off:
                want = torch.maximum(want, scale[pg])
                val[pg, :, :off] = near(val[pg, :, :off] * (scale[pg] / want)[:, None, None])
            val[pg, :, off:off + cnt] = near(y / want[:, None, None])
            scale[pg] = want
            j += cnt
    val, scale = val[:-1], scale[:-1]
    return (val if kv == "e4m3" else val.to(torch.int8)), scale


def _exact_attn(s):
    G, n, P = s["G"], s["n"], s["page"]
    out = s["out"].double()
    B, H = s["table"].shape[0], s["q"].shape[1] // G
    of = torch.float8_e4m3fn if s["kv"] == "e4m3" else torch.int8
    for b, (T, new) in enumerate(zip(s["lens"].tolist(), s["other"].tolist())):
        ids = s["table"][b, : -(-T // P)].long()
        for h in range(H):
            k = (s["k"][ids, h].view(of).double() * s["ks"][ids, h].double()[:, None, None]).reshape(-1, D)[:T]
            v = (s["v"][ids, h].view(of).double() * s["vs"][ids, h].double()[:, None, None]).reshape(-1, D)[:T]
            for i in range(new):
                last = T - new + i + 1
                if last <= 0:
                    out[b, h * G:(h + 1) * G, i] = 0.0
                    continue
                x = s["q"][b, h * G:(h + 1) * G, i].double() @ k[:last].T / D ** 0.5
                out[b, h * G:(h + 1) * G, i] = torch.softmax(x, -1) @ v[:last]
    return out


def exact(case, seed):
    if case["op"] in ("extend", "trim"):
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    k, ks = _exact_write(s, s["k_new"], s["k"], s["ks"])
    v, vs = _exact_write(s, s["v_new"], s["v"], s["vs"])
    return {"k": k, "k_scale": ks, "v": v, "v_scale": vs}
