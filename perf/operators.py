"""Timed cases of the bounded-cache operators: sliding-window decode attention with
sink tokens, accumulated attention weight per cached key, and eviction by that weight.

Each case is one call a serving loop makes per layer on a paged KV cache.  `run` computes
it in plain torch (`own` false) or through the library (`own` true) on the same state;
`exact` gives the definition in 64 bits.  Outputs go to buffers the state holds, and no
run changes what the next one reads (weights and evicted rows go to pages of their own),
so a state can be run again.
"""
import math

import numpy as np
import torch

own = False

PAGE, D = 64, 128


# ----------------------------------------------------------------------------- cases
def listed():
    """op: window | weights | evict; L: mean length; spread: sigma of the lognormal lengths."""
    return [
        # one chat session generating its next token: launch latency
        _case("window one session", "window", "bf16", 1, 900, 0.0, 64, 8, 1, window=256, sinks=4),
        # an ordinary batch of mid-length sessions
        _case("window batch", "window", "bf16", 32, 8192, 0.5, 64, 8, 1, window=1024, sinks=4),
        # a large 8-bit batch verifying one draft token
        _case("window large 8-bit", "window", "e4m3", 128, 16000, 0.6, 64, 8, 2, window=4096,
              sinks=16),
        # several draft tokens, another head layout, odd window: 20 query rows a KV head
        _case("window drafts", "window", "bf16", 13, 20011, 0.7, 40, 8, 4, window=1001, sinks=70),
        # weights of one short session
        _case("weights one session", "weights", "bf16", 1, 1000, 0.0, 64, 8, 1, decay=1.0),
        _case("weights batch", "weights", "bf16", 16, 8192, 0.5, 64, 8, 1, decay=1.0),
        # long 8-bit sessions, two tokens a step
        _case("weights large 8-bit", "weights", "e4m3", 32, 24000, 0.6, 64, 8, 2, decay=0.97),
        # an observation block of eight tokens over one long prompt: 64 query rows a KV head
        _case("weights observation", "weights", "bf16", 1, 65536, 0.0, 64, 8, 8, decay=1.0),
        # one short session reaching its budget
        _case("evict one session", "evict", "bf16", 1, 1024, 0.0, 64, 8, 1, budget=512, sinks=4,
              recent=64),
        _case("evict batch", "evict", "bf16", 32, 8192, 0.5, 64, 8, 1, budget=2048, sinks=4,
              recent=256),
        _case("evict large 8-bit", "evict", "e4m3", 64, 24000, 0.6, 64, 8, 1, budget=4096,
              sinks=16, recent=512),
        # one long prompt cut down before decoding starts
        _case("evict long prompt", "evict", "e4m3", 1, 196608, 0.0, 64, 8, 1, budget=16384,
              sinks=64, recent=1024),
    ]


def draw(rng):
    """Another case of the same ranges; no costlier than the largest listed one of its operator."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["window", "weights", "evict"])
    kv = rng.choice(["bf16", "e4m3"])
    hq, hkv = rng.choice([(64, 8), (32, 8), (16, 16), (8, 1), (40, 8), (48, 4), (12, 3)])
    q_len = rng.choice([1, 1, 1, 2, 3, 5])
    while hq // hkv * q_len > 64:
        q_len -= 1
    spread = rng.choice([0.0, rng.uniform(0.2, 0.7)])
    es = 2 if kv == "bf16" else 1
    if op == "window":
        # pool tokens x heads and visible tokens x heads, both bounded by the largest case
        B, window = log_int(1, 128), log_int(1, 8192)
        sinks = rng.choice([0, 1, 4, rng.randint(5, 200)])
        B = max(1, min(B, 128 * 4096 * 8 // (es * hkv * (window + sinks + 64))))
        L = log_int(8, max(9, min(64000, 128 * 16000 * 8 // (es * hkv * B))))
        return _case("", op, kv, B, L, spread, hq, hkv, q_len, window=window, sinks=sinks)
    if op == "weights":
        B = log_int(1, 32)
        L = log_int(8, max(9, min(120000, 32 * 24000 * 8 // (es * hkv * B))))
        return _case("", op, kv, B, L, spread, hq, hkv, q_len, decay=rng.choice([1.0, 0.9]))
    B = log_int(1, 64)
    L = log_int(80, max(81, min(196608, 64 * 24000 * 8 // (es * hkv * B))))
    sinks, recent = rng.choice([0, 4, 17]), rng.choice([0, 1, 61])
    top = max(sinks + recent + 1, min(L, 64 * 4096 * 8 // (es * hkv * B)))
    budget = log_int(sinks + recent + 1, top)
    return _case("", op, kv, B, L, spread, hq, hkv, 1, budget=budget, sinks=sinks, recent=recent)


def _case(name, op, kv, B, L, spread, hq, hkv, q_len, **more):
    c = dict(name=name, op=op, kv=kv, B=B, L=L, spread=round(spread, 3), hq=hq, hkv=hkv,
             q_len=q_len, **more)
    return c if name else {k: v for k, v in c.items() if k != "name"}


def _lens(c):
    """The request lengths of a case: L each, or lognormal about L, at most three times L."""
    g = np.random.default_rng([c["B"], c["L"], c["hq"]])
    x = c["L"] * np.exp(c["spread"] * g.standard_normal(c["B"]) - c["spread"] ** 2 / 2)
    return np.clip(np.round(x), c["q_len"], 3 * c["L"]).astype(np.int64)


def _visible(c, lens):
    """Keys of each request that some row of the window sees."""
    low = np.maximum(lens - c["q_len"] + 1 - c["window"], 0)
    return lens - low + np.minimum(c["sinks"], low)


def work(c):
    """Each visible key and value, query, weight and output once; two products of 2 rows d flops."""
    lens, es = _lens(c), 2 if c["kv"] == "bf16" else 1
    B, hq, hkv, q_len = c["B"], c["hq"], c["hkv"], c["q_len"]
    rows = hq // hkv * q_len
    if c["op"] == "window":
        n = int(_visible(c, lens).sum())
        return {"bytes": n * hkv * 2 * D * es + B * q_len * hq * (4 * D + 4),
                "flops": n * hkv * rows * 4 * D}
    n = int(lens.sum())
    if c["op"] == "weights":
        return {"bytes": n * hkv * (D * es + 8) + B * q_len * hq * (2 * D + 4),
                "flops": n * hkv * rows * (2 * D + 4)}
    kept = int(np.minimum(lens, c["budget"]).sum())
    return {"bytes": n * hkv * 4 + kept * hkv * (2 * 2 * D * es + 4 + 4), "flops": 0}


# ----------------------------------------------------------------------------- inputs
def prepare(c, seed):
    lens = _lens(c)
    B, hq, hkv, q_len = c["B"], c["hq"], c["hkv"], c["q_len"]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    npg = (lens + PAGE - 1) // PAGE
    keep = np.minimum(lens, c["budget"]) if c["op"] == "evict" else np.zeros(B, np.int64)
    spare = (keep + PAGE - 1) // PAGE           # pages the evicted cache goes to
    P = int(npg.sum() + spare.sum())
    perm = torch.randperm(P, generator=g, device=dev).to(torch.int32)

    def offsets(n):
        o = np.zeros(B + 1, np.int64)
        np.cumsum(n, out=o[1:])
        return torch.from_numpy(o.astype(np.int32)).to(dev)

    s = {"case": c, "lens": torch.from_numpy(lens.astype(np.int32)).to(dev),
         "indptr": offsets(npg), "indices": perm[:int(npg.sum())].contiguous(),
         "max_len": int(lens.max())}

    def pool():
        x = torch.randn((P, hkv, PAGE, D), generator=g, device=dev, dtype=torch.bfloat16)
        if c["kv"] == "bf16":
            return x, None
        scale = (4.5 + torch.rand(hkv, generator=g, device=dev)) / 448.0
        x = x.div_(scale.view(-1, 1, 1)).clamp_(-448.0, 448.0)
        return x.to(torch.float8_e4m3fn), scale

    s["k"], s["ks"] = pool()
    if c["op"] != "weights":
        s["v"], s["vs"] = pool()
    if c["op"] != "evict":
        # sharper than unit scores: a few keys carry most of a row's weight
        s["q"] = (2.0 * torch.randn((B, q_len, hq, D), generator=g, device=dev)).to(torch.bfloat16)
        s["lse"] = torch.zeros((B, q_len, hq), device=dev)
    if c["op"] == "window":
        s["out"] = torch.zeros_like(s["q"])
    if c["op"] == "weights":
        s["lse"] = _plain_lse(s)
    if c["op"] != "window":
        # accumulated weights are heavy-tailed: few keys hold most of them
        z = torch.randn((P, hkv, PAGE), generator=g, device=dev)
        s["acc"] = torch.exp(1.5 * z) * 1e-2
    if c["op"] == "weights":
        s["acc_out"] = torch.zeros_like(s["acc"])
    if c["op"] == "evict":
        s["dst_indptr"], s["dst_indices"] = offsets(spare), perm[int(npg.sum()):].contiguous()
        s["budgets"] = torch.full((B,), c["budget"], dtype=torch.int32, device=dev)
        s["kept"] = torch.full((B, hkv, c["budget"]), -1, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


# ----------------------------------------------------------------------------- plain form
def _slots(s, req, pos):
    """(page, slot) of key `pos` of request `req` (tensors that broadcast)."""
    at = s["indptr"].long()[req] + pos // PAGE
    return s["indices"].long()[at.clamp_(max=s["indices"].numel() - 1)], pos % PAGE


def _rows(s):
    """Query rows by KV head: [B][Hkv][G q_len][d] in 32 bits, row g * q_len + j."""
    c = s["case"]
    q = s["q"].float().view(c["B"], c["q_len"], c["hkv"], -1, D)
    return q.permute(0, 2, 3, 1, 4).reshape(c["B"], c["hkv"], -1, D)


def _scores(s, pos, valid):
    """Scores [B][Hkv][G][q_len][M] of the keys at pos [B][M], causal; -inf where not valid."""
    c = s["case"]
    req = torch.arange(c["B"], device=pos.device)[:, None]
    page, slot = _slots(s, req, pos.clamp(min=0))
    k = s["k"][page, :, slot].float()                       # [B][M][Hkv][d]
    x = torch.matmul(_rows(s), k.permute(0, 2, 3, 1)) / math.sqrt(D)
    if s["ks"] is not None:
        x = x * s["ks"].view(1, -1, 1, 1)
    x = x.view(c["B"], c["hkv"], -1, c["q_len"], pos.shape[1])
    j = torch.arange(c["q_len"], device=pos.device)
    last = s["lens"].long()[:, None] - c["q_len"] + j        # position of token j
    see = valid[:, None, :] & (pos[:, None, :] <= last[:, :, None])
    if c["op"] == "window":
        see &= (pos[:, None, :] > last[:, :, None] - c["window"]) | (pos[:, None, :] < c["sinks"])
    return x.masked_fill_(~see[:, None, None], -math.inf), page, slot


def _all_keys(s):
    pos = torch.arange(s["max_len"], device=s["lens"].device).expand(s["case"]["B"], -1)
    valid = pos < s["lens"][:, None]
    return torch.where(valid, pos, 0), valid


def _plain_lse(s):
    c = s["case"]
    x, _, _ = _scores(s, *_all_keys(s))
    m = x.amax(-1, keepdim=True)
    lse = m.squeeze(-1) + torch.log(torch.exp(x - m).sum(-1))
    return lse.permute(0, 3, 1, 2).reshape(c["B"], c["q_len"], c["hq"]).contiguous()


def _plain_window(s):
    c = s["case"]
    L = s["lens"].long()[:, None]
    low = (L - c["q_len"] + 1 - c["window"]).clamp(min=0)    # first key of token 0's window
    ns = low.clamp(max=c["sinks"])                           # sinks before it
    n = torch.arange(min(s["max_len"], c["sinks"] + c["window"] + c["q_len"] - 1),
                     device=L.device)[None, :]
    pos = torch.where(n < ns, n, low + n - ns)
    valid = pos < L
    pos = torch.where(valid, pos, 0)
    x, page, slot = _scores(s, pos, valid)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    v = s["v"][page, :, slot].float().permute(0, 2, 1, 3)    # [B][Hkv][M][d]
    o = torch.matmul(p.flatten(2, 3), v).view(*p.shape[:4], D) / l
    if s["vs"] is not None:
        o = o * s["vs"].view(1, -1, 1, 1, 1)
    shape = (c["B"], c["q_len"], c["hq"])
    out = o.permute(0, 3, 1, 2, 4).reshape(*shape, D).to(torch.bfloat16)
    lse = (m + torch.log(l)).squeeze(-1).permute(0, 3, 1, 2).reshape(shape)
    return {"out": out, "lse": lse}


def _plain_weights(s):
    c = s["case"]
    pos, valid = _all_keys(s)
    x, page, slot = _scores(s, pos, valid)
    lse = s["lse"].view(c["B"], c["q_len"], c["hkv"], -1).permute(0, 2, 3, 1)[..., None]
    w = torch.exp(x - lse).sum((2, 3))                       # [B][Hkv][M]
    prior = s["acc"][page, :, slot].permute(0, 2, 1) * c["decay"]
    old = pos < s["lens"][:, None] - c["q_len"]              # the new keys start from zero
    w = torch.where(old[:, None, :], prior, 0.0) + w
    s["acc_out"][page[valid], :, slot[valid]] = w.permute(0, 2, 1)[valid]
    return {"acc": s["acc_out"]}


def _plain_evict(s):
    c = s["case"]
    B, hkv, M = c["B"], c["hkv"], s["max_len"]
    pos, valid = _all_keys(s)
    page, slot = _slots(s, torch.arange(B, device=pos.device)[:, None], pos)
    L = s["lens"].long()[:, None]
    a = s["acc"][page, :, slot].permute(0, 2, 1)             # [B][Hkv][M]
    fixed = (pos < c["sinks"]) | (pos >= L - c["recent"])
    a = torch.where(fixed[:, None], math.inf, a).masked_fill(~valid[:, None], -math.inf)
    rank = torch.argsort(a, dim=-1, descending=True, stable=True)
    n = torch.minimum(L.squeeze(1), s["budgets"].long())     # keys each head keeps
    t = torch.arange(c["budget"], device=pos.device)
    live = t < n[:, None]                                    # [B][budget]
    kept = rank[..., :c["budget"]]
    if kept.shape[-1] < c["budget"]:
        kept = torch.nn.functional.pad(kept, (0, c["budget"] - kept.shape[-1]))
    kept = torch.where(live[:, None], kept, 1 << 30).sort(-1).values
    r, tt = torch.nonzero(live, as_tuple=True)               # one row of the new cache each
    src = kept[r, :, tt]                                     # [N][Hkv]
    h = torch.arange(hkv, device=pos.device)[None, :]
    sp, ss = _slots(s, r[:, None], src)
    dp = s["dst_indices"].long()[s["dst_indptr"].long()[r] + tt // PAGE][:, None]
    ds = (tt % PAGE)[:, None]
    bits = torch.int16 if c["kv"] == "bf16" else torch.uint8
    for pool in (s["k"].view(bits), s["v"].view(bits), s["acc"]):
        pool[dp, h, ds] = pool[sp, h, ss]
    out = torch.where(live[:, None], kept, -1).to(torch.int32)
    return {"kept": out, "lens": n.to(torch.int32), "k": s["k"], "v": s["v"], "acc": s["acc"]}


# ----------------------------------------------------------------------------- the library's calls
def _own_workspace(s):
    """The buffers a serving loop keeps from step to step (no results are held in them)."""
    import load_balanced_split_gb300 as hpa
    c = s["case"]
    if "ws" not in s:
        kv = hpa.KV_BF16 if c["kv"] == "bf16" else hpa.KV_E4M3
        more = {}
        count = hpa.hpa_default_num_ctas
        if c["op"] == "window":
            more = dict(window=c["window"], sinks=c["sinks"])
            count = hpa.hpa_default_num_ctas_window
        s["ws"] = hpa.Workspace(c["B"], c["q_len"], c["hq"], D, Hkv=c["hkv"],
                                num_ctas=count(c["hkv"], c["q_len"], kv, c["hq"]), **more)
    return hpa, s["ws"]


def _own_window(s):
    hpa, ws = _own_workspace(s)
    hpa.decode_step(ws, s["q"], s["k"], s["v"], s["lens"], s["indptr"], s["indices"], s["out"],
                    s["lse"], s["ks"], s["vs"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_weights(s):
    hpa, ws = _own_workspace(s)
    ws.plan(s["lens"])
    hpa.hpa_key_weights(s["q"], s["lse"], s["k"], s["indptr"], s["indices"], ws.taskmap,
                        ws.num_ctas, s["acc"], out=s["acc_out"], k_scale=s["ks"],
                        decay=s["case"]["decay"])
    return {"acc": s["acc_out"]}


def _own_evict(s):
    import load_balanced_split_gb300 as hpa
    c = s["case"]
    hpa.evict_step(s["acc"], s["k"], s["v"], s["lens"], s["indptr"], s["indices"], s["budgets"],
                   c["sinks"], c["recent"], s["kept"], s["new_lens"], dst_indptr=s["dst_indptr"],
                   dst_indices=s["dst_indices"], status=s["status"])
    return {"kept": s["kept"], "lens": s["new_lens"], "k": s["k"], "v": s["v"], "acc": s["acc"]}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"window": _own_window, "weights": _own_weights, "evict": _own_evict}[op](s)
    return {"window": _plain_window, "weights": _plain_weights, "evict": _plain_evict}[op](s)


# ----------------------------------------------------------------------------- 64 bits
def exact(c, seed):
    """The definitions, one request at a time, in float64."""
    s = prepare(c, seed)
    host = {k: s[k].cpu().numpy() for k in ("lens", "indptr", "indices")}
    return {"window": _exact_window, "weights": _exact_weights,
            "evict": _exact_evict}[c["op"]](s, host)


def _exact_pages(s, host, r):
    a, b = host["indptr"][r], host["indptr"][r + 1]
    return torch.from_numpy(host["indices"][a:b].astype(np.int64)).cuda()


def _exact_kv(s, pool, scale, pages, L, h):
    x = pool[pages, h].reshape(-1, D)[:L].double()
    return x if scale is None else x * scale[h].double()


def _exact_scores(s, host, r, h):
    """[q_len][G][L] scores of KV head h with every key, and which of them each token sees."""
    c, L = s["case"], int(host["lens"][r])
    G = c["hq"] // c["hkv"]
    k = _exact_kv(s, s["k"], s["ks"], _exact_pages(s, host, r), L, h)
    x = s["q"][r, :, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D)
    i = torch.arange(L, device=k.device)
    at = L - c["q_len"] + torch.arange(c["q_len"], device=k.device)[:, None]
    see = i <= at
    if c["op"] == "window":
        see = see & ((i >= at - c["window"] + 1) | (i < c["sinks"]))
    return x, see[:, None, :].expand_as(x)


def _exact_window(s, host):
    c = s["case"]
    G = c["hq"] // c["hkv"]
    out = torch.zeros((c["B"], c["q_len"], c["hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["B"], c["q_len"], c["hq"]), dtype=torch.float64, device="cuda")
    for r in range(c["B"]):
        pages = _exact_pages(s, host, r)
        for h in range(c["hkv"]):
            x, see = _exact_scores(s, host, r, h)
            lse[r, :, h * G:(h + 1) * G] = z = torch.logsumexp(x.masked_fill(~see, -math.inf), -1)
            p = torch.exp(x - z[..., None]) * see
            v = _exact_kv(s, s["v"], s["vs"], pages, int(host["lens"][r]), h)
            out[r, :, h * G:(h + 1) * G] = p @ v
    return {"out": out, "lse": lse}


def _exact_weights(s, host):
    c = s["case"]
    G = c["hq"] // c["hkv"]
    acc = s["acc_out"].double()
    for r in range(c["B"]):
        pages, L = _exact_pages(s, host, r), int(host["lens"][r])
        for h in range(c["hkv"]):
            x, see = _exact_scores(s, host, r, h)
            z = s["lse"][r, :, h * G:(h + 1) * G].double()[..., None]
            w = (torch.exp(x - z) * see).sum((0, 1))
            before = s["acc"][pages, h].reshape(-1).double()
            w[:L - c["q_len"]] += c["decay"] * before[:L - c["q_len"]]
            new = acc[pages, h].reshape(-1)
            new[:L] = w
            acc[pages, h] = new.view(-1, PAGE)
    return {"acc": acc}


def _exact_evict(s, host):
    c = s["case"]
    acc = s["acc"].cpu().numpy()
    d_ptr, d_idx = s["dst_indptr"].cpu().numpy(), s["dst_indices"].cpu().numpy()
    kept = np.full((c["B"], c["hkv"], c["budget"]), -1, np.int32)
    n = np.minimum(host["lens"], c["budget"]).astype(np.int32)
    new_acc = acc.copy()
    moves = []
    for r in range(c["B"]):
        L, m = int(host["lens"][r]), int(n[r])
        pages = host["indices"][host["indptr"][r]:host["indptr"][r + 1]]
        to = d_idx[d_ptr[r]:d_ptr[r + 1]]
        free = np.arange(L)[c["sinks"]:max(c["sinks"], L - c["recent"])]
        for h in range(c["hkv"]):
            a = acc[pages, h].reshape(-1)[:L]
            if m < L:
                order = np.lexsort((free, -a[free].astype(np.float64)))
                spare = m - (L - len(free))
                gone = np.ones(L, bool)
                gone[free] = False
                keep = np.sort(np.concatenate([np.nonzero(gone)[0], free[order[:spare]]]))
            else:
                keep = np.arange(L)
            kept[r, h, :m] = keep
            t = np.arange(m)
            new_acc[to[t // PAGE], h, t % PAGE] = acc[pages[keep // PAGE], h, keep % PAGE]
            moves.append(np.stack([(pages[keep // PAGE] * np.int64(c["hkv"]) + h) * PAGE
                                   + keep % PAGE,
                                   (to[t // PAGE] * np.int64(c["hkv"]) + h) * PAGE + t % PAGE]))
    src, dst = torch.from_numpy(np.concatenate(moves, 1)).cuda()
    pools = []
    for pool in (s["k"], s["v"]):
        rows = pool.view(torch.int16 if c["kv"] == "bf16" else torch.uint8).reshape(-1, D)
        fresh = rows.clone()
        fresh[dst] = rows[src]
        pools.append(fresh.view(pool.dtype).view(pool.shape))
    return {"kept": kept, "lens": n, "k": pools[0], "v": pools[1],
            "acc": torch.from_numpy(new_acc.astype(np.float64))}
