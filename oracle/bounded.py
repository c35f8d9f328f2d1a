"""ORACLE -- test infrastructure only (tests).

Reference for the bounded-cache operators, in numpy fp64 and plain loops from their
definitions (the pages have no counterpart):

  window_plan     the pages a sliding window with sink tokens reaches, and the dynamic
                  plan over them;
  attention_rows  attention of any (request, key list) with any visibility rule, with the
                  magnitudes that error bounds are built from;
  key_weights     the attention weight each cached key receives;
  evict           which keys are kept, and the cache after the move.

Token j of request r sits at a = L_r - q_len + j and sees key i <= a; with a window of W
keys and S sinks, when also i > a - W or i < S.
"""
from __future__ import annotations

import math

import numpy as np

from . import fourbit, scheduler

PAGE = 64


def pool_values(pool, kv_dtype, scale=None):
    """fp64 values of a pool [P][Hkv][page][d] (torch tensor, bf16 or E4M3 codes, or 4-bit
    pages [P][Hkv][bytes])."""
    import torch
    if kv_dtype == "e2m1":
        return fourbit.values(pool.cpu().numpy(), scale)
    if kv_dtype == "bf16":
        return pool.cpu().to(torch.float64).numpy()
    x = pool.cpu().view(torch.float8_e4m3fn).to(torch.float64).numpy()
    return x if scale is None else x * np.asarray(scale, np.float64)[None, :, None, None]


def sees(L, q_len, j, i, window=None, sinks=0) -> bool:
    a = L - q_len + j
    return i <= a and (window is None or i > a - window or i < sinks)


def window_pages(L, q_len, window, sinks):
    """Real pages that hold a key of the sinks or of some token's window, ascending; pages
    between them that hold neither are left out.  A page from position
    max(0, L - q_len + 1 - window) on is in, whatever it holds."""
    low = max(0, L - q_len + 1 - window)
    return [g for g in range((L + PAGE - 1) // PAGE)
            if g * PAGE < min(sinks, low) or g >= low // PAGE]


def window_plan(lens, q_len, window, sinks, tile, C):
    """The dynamic plan over the compact sequences: (plan over compact lengths, page lists)."""
    pages = [window_pages(int(L), q_len, window, sinks) for L in lens]
    compact = [int(L) - PAGE * ((int(L) + PAGE - 1) // PAGE - len(p)) for L, p in zip(lens, pages)]
    return scheduler.plan(np.array(compact, np.int32), tile, C), pages


def keys_of(b, values, r, h):
    """[L][d] rows of request r, KV head h, from pool values."""
    L = int(b.seq_lens[r])
    ids = np.asarray(b.page_indices)[int(b.page_indptr[r]):int(b.page_indptr[r + 1])]
    return values[ids, h].reshape(-1, b.d)[:L]


def attention_rows(b, window=None, sinks=0, sm_scale=None, keys=None):
    """fp64 attention over each request's visible keys (or, for a partial, those of the sets
    keys[r] alone).  Returns out, lse, A = sum w |v| and E, the largest sum |q . k| sm_scale
    products of a row: [B][q_len][Hq](, d)."""
    sm = 1.0 / math.sqrt(b.d) if sm_scale is None else sm_scale
    K = pool_values(b.k_pool, b.kv_dtype, b.k_scale)
    V = pool_values(b.v_pool, b.kv_dtype, b.v_scale)
    q = b.q.double().numpy()
    G = b.Hq // b.Hkv
    out = np.zeros(q.shape)
    A = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    E = np.zeros(q.shape[:3])
    for r in range(b.B):
        L = int(b.seq_lens[r])
        for h in range(b.Hkv):
            k, v = keys_of(b, K, r, h), keys_of(b, V, r, h)
            for j in range(b.q_len):
                vis = [i for i in range(L) if sees(L, b.q_len, j, i, window, sinks)
                       and (keys is None or i in keys[r])]
                if not vis:
                    continue
                kk, vv = k[vis], v[vis]
                for g in range(h * G, (h + 1) * G):
                    s = kk @ q[r, j, g] * sm
                    m = s.max()
                    w = np.exp(s - m)
                    l = w.sum()
                    lse[r, j, g] = m + math.log(l)
                    out[r, j, g] = w @ vv / l
                    A[r, j, g] = w @ np.abs(vv) / l
                    E[r, j, g] = (np.abs(kk) @ np.abs(q[r, j, g])).max() * abs(sm)
    return out, lse, A, E


def key_weights(b, lse, acc, decay, window=None, sinks=0, sm_scale=None):
    """(acc after the step [P][Hkv][page], written mask, largest E of the rows per slot)."""
    sm = 1.0 / math.sqrt(b.d) if sm_scale is None else sm_scale
    K = pool_values(b.k_pool, b.kv_dtype, b.k_scale)
    q = b.q.double().numpy()
    G = b.Hq // b.Hkv
    new = np.array(acc, np.float64)
    written = np.zeros(new.shape, bool)
    E = np.zeros(new.shape)
    for r in range(b.B):
        L = int(b.seq_lens[r])
        ids = np.asarray(b.page_indices)[int(b.page_indptr[r]):int(b.page_indptr[r + 1])]
        for h in range(b.Hkv):
            k = keys_of(b, K, r, h)
            for i in range(L):
                rows = [j for j in range(b.q_len) if sees(L, b.q_len, j, i, window, sinks)]
                if not rows:
                    continue
                page, slot = ids[i // PAGE], i % PAGE
                t = decay * float(acc[page, h, slot]) if i < L - b.q_len and decay else 0.0
                qq = q[r, rows, h * G:(h + 1) * G].reshape(-1, b.d)
                z = np.asarray(lse, np.float64)[r, rows, h * G:(h + 1) * G].reshape(-1)
                live = ~np.isneginf(z)
                t += np.exp(qq[live] @ k[i] * sm - z[live]).sum()
                new[page, h, slot] = t
                written[page, h, slot] = True
                E[page, h, slot] = (np.abs(qq) @ np.abs(k[i])).max() * abs(sm)
    return new, written, E


def heavier(a, i, c, j) -> bool:
    """Whether key i of weight a goes before key j of weight c: NaN first, ties by index."""
    na, nc = math.isnan(a), math.isnan(c)
    if na != nc:
        return na
    if na or a == c:
        return i < j
    return a > c


def kept_keys(weights, budget, sinks, recent):
    """Ascending indices one KV head keeps of keys with these weights."""
    L = len(weights)
    if L <= budget:
        return list(range(L))
    free = list(range(sinks, L - recent))
    rank = {i: (-math.inf if math.isnan(weights[i]) else -float(weights[i]), i) for i in free}
    nans = [i for i in free if math.isnan(weights[i])]
    numbers = sorted((i for i in free if not math.isnan(weights[i])), key=rank.get)
    best = (nans + numbers)[:budget - sinks - recent]
    return sorted(list(range(sinks)) + best + list(range(L - recent, L)))
