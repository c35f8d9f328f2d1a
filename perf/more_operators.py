"""Timed cases of serving from a 4-bit cache: page tables built from request lengths, the
writer that norms, rotates and stores a token's projections, and attention over 4-bit pages.

Each case is one call a serving loop makes: `pages` once per step, `store` and `attend` once
per layer.  `run` computes it in plain torch (`own` false) or through the library (`own`
true) on the same state; `exact` gives the definition in 64 bits.  No run changes what the
next one reads (a page step is computed from the state before it), so a state can be run
again.  A 4-bit cache holds, per page and KV head, 64 rows of 64 bytes (two E2M1 codes a byte,
the even element low) and 64 x 8 E4M3 scales, one for each 16 elements of a row.
"""
import math

import numpy as np
import torch

own = False

PAGE, D, BLOCK = 64, 128, 16
CODES = PAGE * D // 2                       # bytes of codes of one page and KV head
UNIT = CODES + PAGE * D // BLOCK            # with the scales behind them
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
MAX_POS = 32768


# ----------------------------------------------------------------------------- cases
def listed():
    """op: pages | store | attend."""
    return [
        # one session takes its next token: launch latency
        _case("pages one session", "pages", B=1, L=900, spread=0.0, new=1, tight=0),
        # a continuous batch between two decode steps: some sessions end, some begin
        _case("pages decode batch", "pages", B=128, L=8192, spread=0.5, new=1, tight=0),
        # a large pool with chunks of prompts coming in
        _case("pages prefill chunks", "pages", B=1000, L=16000, spread=0.6, new=256, tight=0),
        # one token of one session into an 8-bit cache
        _case("store one token", "store", kv="e4m3", N=1, hq=64, hkv=8, norm="before",
              pairs="half", rot=128, hadamard=False),
        # a decode batch, another order of norm and rotation, transformed for low bits
        _case("store decode batch", "store", kv="e4m3", N=128, hq=64, hkv=8, norm="after",
              pairs="half", rot=128, hadamard=True),
        # chunks of prompts into a 4-bit cache: odd count, part of the head rotated
        _case("store chunk 4-bit", "store", kv="e2m1", N=8191, hq=40, hkv=8, norm="before",
              pairs="interleaved", rot=64, hadamard=True),
        # a long prompt into a bf16 cache
        _case("store prompt", "store", kv="bf16", N=32768, hq=64, hkv=8, norm="before",
              pairs="half", rot=128, hadamard=False),
        # one chat session generating its next token
        _case("attend one session", "attend", B=1, L=900, spread=0.0, hq=64, hkv=8, q_len=1,
              window=0, sinks=0),
        # an ordinary batch of mid-length sessions
        _case("attend batch", "attend", B=32, L=8192, spread=0.5, hq=64, hkv=8, q_len=1,
              window=0, sinks=0),
        # many long sessions verifying one draft token
        _case("attend large", "attend", B=64, L=20000, spread=0.4, hq=64, hkv=8, q_len=2,
              window=0, sinks=0),
        # several draft tokens, another head layout: 20 query rows a KV head
        _case("attend drafts", "attend", B=13, L=20011, spread=0.7, hq=40, hkv=8, q_len=4,
              window=0, sinks=0),
        # a large batch that sees a window and the first tokens
        _case("attend window", "attend", B=128, L=16000, spread=0.6, hq=64, hkv=8, q_len=1,
              window=4096, sinks=16),
    ]


def draw(rng):
    """Another case of the same ranges; no costlier than the largest listed one of its operator."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["pages", "store", "attend"])
    spread = rng.choice([0.0, rng.uniform(0.2, 0.6)])
    if op == "pages":
        B = log_int(1, 1000)
        return _case("", op, B=B, L=log_int(8, min(100000, 16000 * 1000 // B)), spread=spread,
                     new=rng.choice([1, 1, 2, 4, log_int(1, 256)]), tight=rng.choice([0, 0, 1]))
    hq, hkv = rng.choice([(64, 8), (32, 8), (16, 16), (8, 1), (40, 8), (48, 4), (12, 3)])
    if op == "store":
        return _case("", op, kv=rng.choice(["bf16", "e4m3", "e2m1"]),
                     N=log_int(1, 32768 * 80 // max(80, hq + 2 * hkv)), hq=hq, hkv=hkv,
                     norm=rng.choice(["before", "after", "none"]),
                     pairs=rng.choice(["half", "interleaved"]), rot=rng.choice([128, 128, 64, 32]),
                     hadamard=rng.choice([False, True]))
    q_len = rng.choice([1, 1, 1, 2, 3, 5])
    while hq // hkv * q_len > 64:
        q_len -= 1
    B = log_int(1, 64)
    window = rng.choice([0, 0, log_int(1, 8192)])
    most = 64 * 20000 * 8 // max(8 * B, hkv * B, hq * q_len * B // 16)
    return _case("", op, B=B, L=log_int(8, min(100000, most)), spread=spread * 0.7, hq=hq, hkv=hkv,
                 q_len=q_len, window=window,
                 sinks=rng.choice([0, 4, rng.randint(5, 200)]) if window else 0)


def _case(name, op, spread=None, **more):
    c = dict(name=name, op=op, **more)
    if spread is not None:
        c["spread"] = round(spread, 3)
    return c if name else {k: v for k, v in c.items() if k != "name"}


def _lens(c, least):
    """The lengths of a case: L each, or lognormal about L, at most three times L."""
    g = np.random.default_rng([c["B"], c["L"]])
    x = c["L"] * np.exp(c["spread"] * g.standard_normal(c["B"]) - c["spread"] ** 2 / 2)
    return np.clip(np.round(x), least, 3 * c["L"]).astype(np.int64)


def _step(c):
    """(pages held, new length, new tokens) of each request of a page step: of twenty in the
    batch one has just ended and one just begins, the others take their next tokens."""
    before = _lens(c, 1)
    i = np.arange(c["B"])
    ends, begins = i % 20 == 7, i % 20 == 13
    held = np.where(begins, 0, (before + PAGE - 1) // PAGE)
    new = np.where(ends, 0, np.maximum(1, c["new"] - i % 7))
    return held, np.where(ends, 0, np.where(begins, 0, before) + new), new


def _spare(c):
    """Free pages before the step: enough for it, or (tight) for about half of it."""
    held, lens, _ = _step(c)
    grow = np.maximum((lens + PAGE - 1) // PAGE - held, 0).sum()
    back = np.maximum(held - (lens + PAGE - 1) // PAGE, 0).sum()
    return int(max(0, grow // 2 - back) if c["tight"] else grow + 64)


def _row_bytes(kv):
    return {"bf16": 2 * D, "e4m3": D, "e2m1": D // 2 + D // BLOCK}[kv]


def work(c):
    """Each input once and each output once: page ids and slots; projections and rows; visible
    keys and values, queries and outputs, and two products of 2 rows d flops."""
    if c["op"] == "pages":
        held, lens, new = _step(c)
        need = (lens + PAGE - 1) // PAGE
        moved = np.abs(need - held).sum()      # page ids that change owner: read, written
        return {"bytes": int(24 * c["B"] + 4 * np.minimum(held, need).sum() + 4 * need.sum()
                             + 8 * moved + 12 * new.sum()), "flops": 0}
    if c["op"] == "store":
        rows = c["hq"] + 2 * c["hkv"]
        return {"bytes": c["N"] * (rows * 2 * D + c["hq"] * 2 * D
                                   + 2 * c["hkv"] * _row_bytes(c["kv"]) + 4 * c["rot"] + 12),
                "flops": c["N"] * (c["hq"] + c["hkv"]) * D * (8 + 7 * c["hadamard"])}
    lens = _lens(c, c["q_len"])
    if c["window"]:
        low = np.maximum(lens - c["q_len"] + 1 - c["window"], 0)
        lens = lens - low + np.minimum(c["sinks"], low)
    n = int(lens.sum())
    return {"bytes": n * c["hkv"] * 2 * _row_bytes("e2m1") + c["B"] * c["q_len"] * c["hq"] * (4 * D + 4),
            "flops": n * c["hq"] * c["q_len"] * 4 * D}


# ----------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()


def _indptr(n):
    o = np.zeros(len(n) + 1, np.int64)
    np.cumsum(n, out=o[1:])
    return _i32(o)


def prepare(c, seed):
    return {"pages": _prepare_pages, "store": _prepare_store, "attend": _prepare_attend}[c["op"]](
        c, _generator(seed))


def _prepare_pages(c, g):
    held, lens, new = _step(c)
    B, spare = c["B"], _spare(c)
    rows, most = B + 5, int(max(held.max(), (lens.max() + PAGE - 1) // PAGE)) + 3
    pages = int(held.sum()) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    row = torch.randperm(rows, generator=g, device="cuda")[:B]   # sessions in any order
    h = torch.from_numpy(held).cuda()
    table = torch.full((rows, most), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(most, device="cuda")
    mine = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    mine[at < h[:, None]] = perm[:int(held.sum())]
    table[row] = mine
    held_by_row = torch.zeros(rows, dtype=torch.int32, device="cuda")
    held_by_row[row] = h.to(torch.int32)
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:spare] = perm[int(held.sum()):]
    need = (lens + PAGE - 1) // PAGE
    tokens = int(new.sum()) + 9                # a captured step leaves room behind its last token
    return {"case": c, "lens": _i32(lens), "new": _i32(new), "rows": row.to(torch.int32),
            "table": table, "held": held_by_row, "held_out": held_by_row.clone(), "free": free,
            "count": _i32([spare]), "count_out": _i32([0]), "indptr": _i32(np.zeros(B + 1)),
            "indices": torch.zeros(int(np.maximum(need, held).sum()) + 1, dtype=torch.int32,
                                   device="cuda"),
            "slots": torch.zeros(tokens, dtype=torch.int64, device="cuda"),
            "positions": torch.zeros(tokens, dtype=torch.int32, device="cuda"),
            "status": _i32([0])}


def _prepare_store(c, g):
    N, hq, hkv, kv, rot = c["N"], c["hq"], c["hkv"], c["kv"], c["rot"]
    x = torch.randn((N, hq + 2 * hkv, D), generator=g, device="cuda")
    # a few channels of a projection are much larger than the others
    x *= torch.exp(0.5 * torch.randn((hq + 2 * hkv, D), generator=g, device="cuda"))
    x = x.to(torch.bfloat16)
    P = (N + PAGE - 1) // PAGE + 1
    place = torch.arange(N, device="cuda")
    page = torch.randperm(P, generator=g, device="cuda")
    slots = page[place // PAGE] * PAGE + place % PAGE
    slots[N - N // 50:] = -1                   # rows of a captured batch that hold no token
    start = torch.randint(0, MAX_POS, ((N + 999) // 1000,), generator=g, device="cuda")
    positions = (start[place // 1000] + place) % MAX_POS
    angle = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    s = {"case": c, "q": x[:, :hq], "k": x[:, hq:hq + hkv], "v": x[:, hq + hkv:],
         "slots": slots, "positions": positions.to(torch.int32),
         "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float(),
         "q_out": torch.zeros((N, hq, D), dtype=torch.bfloat16, device="cuda"),
         "status": _i32([0])}
    for name in ("q_norm", "k_norm"):
        w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        s[name] = w if c["norm"] != "none" else None
    dtype, shape = {"bf16": (torch.bfloat16, (P, hkv, PAGE, D)),
                    "e4m3": (torch.uint8, (P, hkv, PAGE, D)),
                    "e2m1": (torch.uint8, (P, hkv, UNIT))}[kv]
    for name in ("k", "v"):
        s[name + "_pool"] = torch.zeros(shape, dtype=dtype, device="cuda")
        unit = (0.5 + torch.rand(hkv, generator=g, device="cuda")) / 64
        s[name + "_scale"] = None if kv == "bf16" else unit
    return s


def _quantise(y):
    """(codes 0..15, scales) of y [..][d] in units of the head's scale."""
    blocks = y.unflatten(-1, (-1, BLOCK))
    scale = (blocks.abs().amax(-1) / 6.0).clamp_(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    z = torch.where(s > 0, blocks / s, torch.zeros_like(blocks))
    a = z.abs()
    code = (a > 0.25).to(torch.uint8)          # to the nearest of E2M1, ties to the even code
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(z).to(torch.uint8) * 8
    return code.flatten(-2), scale


def _pack(pool, rows, code, scale):
    """Codes [n][Hkv][d] and scales into pool places rows = (page, slot)."""
    page, slot = rows
    pool[..., :CODES].unflatten(-1, (PAGE, D // 2))[page, :, slot] = (
        code[..., 0::2] | (code[..., 1::2] << 4))
    pool[..., CODES:].unflatten(-1, (PAGE, D // BLOCK))[page, :, slot] = scale.view(torch.uint8)


def _prepare_attend(c, g):
    lens = _lens(c, c["q_len"])
    B, hq, hkv, q_len = c["B"], c["hq"], c["hkv"], c["q_len"]
    npg = (lens + PAGE - 1) // PAGE
    P = int(npg.sum()) + 1
    s = {"case": c, "lens": _i32(lens), "indptr": _indptr(npg), "max_len": int(lens.max()),
         "indices": torch.randperm(P, generator=g, device="cuda").to(torch.int32)[:P - 1]}
    for name in ("k", "v"):
        unit = (0.5 + torch.rand(hkv, generator=g, device="cuda")) / 64
        x = torch.randn((P, hkv, PAGE, D), generator=g, device="cuda")
        code, scale = _quantise(x.div_(unit.view(-1, 1, 1)))
        pool = torch.empty((P, hkv, UNIT), dtype=torch.uint8, device="cuda")
        pool[..., :CODES] = (code[..., 0::2] | (code[..., 1::2] << 4)).flatten(2)
        pool[..., CODES:] = scale.view(torch.uint8).flatten(2)
        s[name], s[name + "_scale"] = pool, unit
        del x, code, scale
    # sharper than unit scores: a few keys carry most of a row's weight
    s["q"] = (2.0 * torch.randn((B, q_len, hq, D), generator=g, device="cuda")).to(torch.bfloat16)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((B, q_len, hq), device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms
def _plain_pages(s):
    L, new, row = s["lens"].long(), s["new"].long(), s["rows"].long()
    table = s["table"]
    held = s["held"][row].long()
    need = (L + PAGE - 1) // PAGE
    back, take = (held - need).clamp(min=0), (need - held).clamp(min=0)
    free = s["count"].long() + back.sum()      # pages to give out, the returned ones on top
    ends = torch.cumsum(take, 0)
    served = (take == 0) | (ends <= free)      # in order, while the pages last
    pages = torch.where(served, need, held)
    at = torch.arange(table.shape[1], device=L.device)[None]
    mine = table[row]
    returned = (at >= need[:, None]) & (at < held[:, None])
    n = s["count"].long() + (torch.cumsum(back, 0) - back)[:, None] + at - need[:, None]
    s["free"][n[returned]] = mine[returned]
    fresh = (at >= held[:, None]) & (at < need[:, None]) & served[:, None]
    n = free - 1 - ((ends - take)[:, None] + at - held[:, None])
    mine[fresh] = s["free"][n[fresh]]
    table[row] = mine
    s["held_out"][row] = pages.to(torch.int32)
    s["count_out"][:] = (free - (take * served).sum()).to(torch.int32)
    s["indptr"][1:] = torch.cumsum(pages, 0)
    ids = mine[at < pages[:, None]]
    s["indices"][:ids.shape[0]] = ids
    t = torch.arange(s["slots"].shape[0], device=L.device)
    last = torch.cumsum(new, 0)
    r = torch.searchsorted(last, t, right=True)
    valid = r < L.shape[0]
    r = r.clamp(max=L.shape[0] - 1)
    pos = torch.where(valid, L[r] - last[r] + t, 0)
    good = valid & served[r]
    page = mine[r, torch.where(good, pos // PAGE, 0)].long()
    s["slots"][:] = torch.where(good, page * PAGE + pos % PAGE, -1)
    s["positions"][:] = pos.to(torch.int32)
    return _pages_out(s)


def _pages_out(s):
    return {"table": s["table"], "held": s["held_out"], "free": s["free"], "count": s["count_out"],
            "indptr": s["indptr"], "indices": s["indices"], "slots": s["slots"],
            "positions": s["positions"]}


def _hadamard(dtype):
    h = torch.ones((1, 1), dtype=dtype, device="cuda")
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return h / math.sqrt(D)


def _heads(s, x, w, dtype):
    """Norm, rotation and transform of x [N][heads][d], the norm before or after the rotation."""
    c = s["case"]
    x = x.to(dtype)

    def normed(y):
        return y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.to(dtype)

    if c["norm"] == "before":
        x = normed(x)
    cos, sin = s["cos_sin"].to(dtype)[s["positions"].long()][:, None].chunk(2, -1)
    turn, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["pairs"] == "half":
        a, b = turn.chunk(2, -1)
        turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    x = torch.cat([turn, rest], -1)
    if c["norm"] == "after":
        x = normed(x)
    return x @ _hadamard(dtype) if c["hadamard"] else x


def _plain_store(s):
    c = s["case"]
    live = s["slots"] >= 0
    q = _heads(s, s["q"], s["q_norm"], torch.float32)
    s["q_out"][:] = torch.where(live[:, None, None], q.to(torch.bfloat16), s["q_out"])
    at = s["slots"][live]
    rows = at // PAGE, at % PAGE
    for name in ("k", "v"):
        x = _heads(s, s["k"], s["k_norm"], torch.float32) if name == "k" else s["v"].float()
        x, pool = x[live], s[name + "_pool"]
        if c["kv"] == "bf16":
            pool[rows[0], :, rows[1]] = x.to(torch.bfloat16)
            continue
        x = x * (1.0 / s[name + "_scale"])[:, None]
        if c["kv"] == "e4m3":
            x = x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            pool[rows[0], :, rows[1]] = x.view(torch.uint8)
        else:
            _pack(pool, rows, *_quantise(x))
    return _store_out(s)


def _store_out(s):
    """Queries, and the caches as the values that they hold: 8-bit pools as they are, 4-bit codes
    as E4M3 of a 64th of their value (sign, exponent and fraction bits moved to their places)."""
    kv, out = s["case"]["kv"], {"q": s["q_out"]}
    for name in ("k", "v"):
        pool = s[name + "_pool"]
        if kv == "e2m1":
            words = pool.view(torch.int64)[..., :CODES // 8]
            sign, size = 0x0808080808080808, 0x0707070707070707
            out[name + "_low"] = ((words & sign) << 4 | (words & size) << 2).view(torch.float8_e4m3fn)
            words = words >> 4
            out[name + "_high"] = ((words & sign) << 4 | (words & size) << 2).view(torch.float8_e4m3fn)
            out[name + "_scales"] = pool[..., CODES:].view(torch.float8_e4m3fn)
        else:
            out[name] = pool if kv == "bf16" else pool.view(torch.float8_e4m3fn)
    return out


def _cached(s, name, page, slot, dtype):
    """Rows [..][Hkv][d] of the 4-bit pool at (page, slot)."""
    pool = s[name]
    code = pool[..., :CODES].unflatten(-1, (PAGE, D // 2))[page, :, slot]
    scale = pool[..., CODES:].unflatten(-1, (PAGE, D // BLOCK))[page, :, slot]
    value = torch.tensor(E2M1 + [-x for x in E2M1], device="cuda", dtype=dtype)
    pair = torch.stack([code & 15, code >> 4], -1).flatten(-2).int()
    x = value[pair].unflatten(-1, (-1, BLOCK))
    x *= scale.view(torch.float8_e4m3fn).to(dtype)[..., None]
    return x.flatten(-2).mul_(s[name + "_scale"].to(dtype)[:, None])


def _plain_attend(s):
    c = s["case"]
    B, q_len, hkv = c["B"], c["q_len"], c["hkv"]
    L = s["lens"].long()[:, None]
    j = torch.arange(q_len, device=L.device)
    last = L - q_len + j                                     # [B][q_len] position of token j
    if c["window"]:
        low = (L - q_len + 1 - c["window"]).clamp(min=0)     # first key of token 0's window
        first = low.clamp(max=c["sinks"])                    # sinks before it
        n = torch.arange(min(s["max_len"], c["sinks"] + c["window"] + q_len - 1), device=L.device)
        pos = torch.where(n < first, n, low + n - first)
    else:
        pos = torch.arange(s["max_len"], device=L.device).expand(B, -1)
    valid = pos < L
    pos = torch.where(valid, pos, 0)
    at = s["indptr"].long()[:-1, None] + pos // PAGE
    page, slot = s["indices"].long()[at], pos % PAGE
    see = valid[:, None] & (pos[:, None] <= last[..., None])
    if c["window"]:
        see &= (pos[:, None] > last[..., None] - c["window"]) | (pos[:, None] < c["sinks"])
    q = s["q"].float().view(B, q_len, hkv, -1, D).permute(0, 2, 3, 1, 4)
    G = q.shape[2]
    k = _cached(s, "k", page, slot, torch.float32).permute(0, 2, 3, 1)
    x = torch.matmul(q.flatten(2, 3), k).unflatten(2, (G, q_len)) / math.sqrt(D)
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    v = _cached(s, "v", page, slot, torch.float32).permute(0, 2, 1, 3)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (G, q_len)) / total
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)
    s["out"][:] = o.permute(0, 3, 1, 2, 4).reshape(s["out"].shape)
    s["lse"][:] = lse.reshape(s["lse"].shape)
    return {"out": s["out"], "lse": s["lse"]}


# ----------------------------------------------------------------------------- the library's calls
def _own_pages(s):
    import load_balanced_split_gb300 as hpa
    if "ws" not in s:                          # a serving loop's workspace (no results in it)
        n = hpa.hpa_assign_pages_workspace(s["case"]["B"], s["table"].shape[0])
        s["ws"] = torch.empty((n + 3) // 4, dtype=torch.int32, device="cuda")
    hpa.hpa_assign_pages(s["lens"], s["new"], s["table"], s["held"], s["free"], s["count"],
                         s["indptr"], s["indices"], s["slots"], s["positions"], s["ws"],
                         rows=s["rows"], held_out=s["held_out"], free_count_out=s["count_out"],
                         status=s["status"])
    return _pages_out(s)


def _own_store(s):
    import load_balanced_split_gb300 as hpa
    c = s["case"]
    hpa.hpa_store_qkv(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"],
                      s["k_pool"], s["v_pool"], s["q_out"], s["q_norm"], s["k_norm"], eps=1e-6,
                      norm_after=c["norm"] == "after", interleaved=c["pairs"] == "interleaved",
                      use_hadamard=c["hadamard"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                      status=s["status"])
    return _store_out(s)


def _own_attend(s):
    import load_balanced_split_gb300 as hpa
    c = s["case"]
    if "ws" not in s:
        more = dict(window=c["window"], sinks=c["sinks"]) if c["window"] else {}
        count = hpa.hpa_default_num_ctas_window if c["window"] else hpa.hpa_default_num_ctas
        s["ws"] = hpa.Workspace(c["B"], c["q_len"], c["hq"], D, Hkv=c["hkv"],
                                num_ctas=count(c["hkv"], c["q_len"], hpa.KV_E2M1, c["hq"]), **more)
    hpa.decode_step(s["ws"], s["q"], s["k"], s["v"], s["lens"], s["indptr"], s["indices"],
                    s["out"], s["lse"], s["k_scale"], s["v_scale"])
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"pages": _own_pages, "store": _own_store, "attend": _own_attend}[op](s)
    return {"pages": _plain_pages, "store": _plain_store, "attend": _plain_attend}[op](s)


# ----------------------------------------------------------------------------- 64 bits
def exact(c, seed):
    """The definitions in float64 (page tables are whole numbers and have none)."""
    if c["op"] == "pages":
        return None
    s = prepare(c, seed)
    return _exact_store(s) if c["op"] == "store" else _exact_attend(s)


def _exact_heads(s, x, w):
    """One head's tokens at a time: [N][d] by the matrix of the transform."""
    c, out = s["case"], []
    pos = s["positions"].long()
    half = c["rot"] // 2
    turn = s["cos_sin"][pos].double()
    turn = torch.complex(turn[:, :half], turn[:, half:])
    i = torch.arange(D, device="cuda")
    bits = i[:, None] & i
    odd = sum((bits >> b) & 1 for b in range(7)) % 2
    H = (1.0 - 2.0 * odd.double()) / math.sqrt(D)
    for h in range(x.shape[1]):
        y = x[:, h].double()
        for step in (("norm", "turn") if c["norm"] == "before" else ("turn", "norm")):
            if step == "norm" and c["norm"] != "none":
                y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / D + 1e-6) * w.double()
            if step == "turn":
                z = y[:, :c["rot"]]
                z = (torch.complex(z[:, :half].contiguous(), z[:, half:].contiguous())
                     if c["pairs"] == "half" else torch.view_as_complex(
                         z.reshape(-1, half, 2).contiguous())) * turn
                z = torch.cat([z.real, z.imag], 1) if c["pairs"] == "half" else (
                    torch.view_as_real(z).reshape(-1, c["rot"]))
                y = torch.cat([z, y[:, c["rot"]:]], 1)
        out.append(y @ H if c["hadamard"] else y)
    return torch.stack(out, 1)


def _exact_store(s):
    """Queries, and bf16 and 8-bit rows before their rounding; 4-bit codes and scales round twice
    and have no value of their own in 64 bits."""
    c = s["case"]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
    q[live] = _exact_heads(s, s["q"], s["q_norm"])[live]
    out = {"q": q}
    for name in ("k", "v"):
        if c["kv"] == "e2m1":
            out.update({name + "_low": None, name + "_high": None, name + "_scales": None})
            continue
        x = _exact_heads(s, s["k"], s["k_norm"]) if name == "k" else s["v"].double()
        if c["kv"] == "e4m3":
            x = (x / s[name + "_scale"].double()[:, None]).clamp(-448.0, 448.0)
        pool = torch.zeros(s[name + "_pool"].shape, dtype=torch.float64, device="cuda")
        at = s["slots"][live]
        pool.permute(0, 2, 1, 3)[at // PAGE, at % PAGE] = x[live]
        out[name] = pool
    return out


def _exact_attend(s):
    c = s["case"]
    B, q_len, hq, hkv = c["B"], c["q_len"], c["hq"], c["hkv"]
    out = torch.zeros((B, q_len, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, q_len, hq), dtype=torch.float64, device="cuda")
    lens, indptr = s["lens"].tolist(), s["indptr"].tolist()
    for r in range(B):
        i = torch.arange(lens[r], device="cuda")
        at = lens[r] - q_len + torch.arange(q_len, device="cuda")[:, None]
        see = i <= at
        if c["window"]:
            see &= (i > at - c["window"]) | (i < c["sinks"])
        i = i[see.any(0)]
        see = see[:, i]
        page = s["indices"][indptr[r]:indptr[r + 1]].long()[i // PAGE]
        k = _cached(s, "k", page, i % PAGE, torch.float64)
        v = _cached(s, "v", page, i % PAGE, torch.float64)
        for h in range(hkv):
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = s["q"][r, :, heads].double() @ k[:, h].T / math.sqrt(D)    # [q_len][G][keys]
            x = x.masked_fill(~see[:, None], -math.inf)
            lse[r, :, heads] = z = torch.logsumexp(x, -1)
            out[r, :, heads] = torch.exp(x - z[..., None]) @ v[:, h]
    return {"out": out, "lse": lse}
