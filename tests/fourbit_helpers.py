"""Helpers for the tests of 4-bit caches: batches on E2M1 pages, poisoned hidden slots, and one
step through the library."""
import numpy as np
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from oracle import bounded, fourbit


def make_batch(lens, q_len=1, heads=(16, 2), seed=0):
    """A workloads batch whose pools are 4-bit pages; scales differ by head."""
    b = W.make_batch(lens, q_len=q_len, kv_dtype="bf16", seed=seed, Hq=heads[0], Hkv=heads[1])
    g = np.random.default_rng(seed + 77)
    b.kv_dtype = "e2m1"
    b.k_scale = ((0.5 + g.random(b.Hkv)) / 64).astype(np.float32)
    b.v_scale = ((0.5 + g.random(b.Hkv)) / 64).astype(np.float32)
    for name, scale in (("k_pool", b.k_scale), ("v_pool", b.v_scale)):
        x = getattr(b, name).double().numpy() / scale.astype(np.float64)[None, :, None, None]
        setattr(b, name, torch.from_numpy(fourbit.pack(x)))
    return b


def seen_slots(b, window=None, sinks=0):
    seen = np.zeros((b.num_pages, 64), bool)
    for r in range(b.B):
        L = int(b.seq_lens[r])
        ids = b.page_indices[int(b.page_indptr[r]):int(b.page_indptr[r + 1])]
        for i in range(L):
            if any(bounded.sees(L, b.q_len, j, i, window, sinks) for j in range(b.q_len)):
                seen[ids[i // 64], i % 64] = True
    return seen


def rows_of(pool):
    """Views (codes [P][Hkv][64][64], scales [P][Hkv][64][8]) of 4-bit pages."""
    c = pool[..., :fourbit.CODES].unflatten(-1, (64, 64))
    return c, pool[..., fourbit.CODES:].unflatten(-1, (64, 8))


def poison_hidden(b, window=None, sinks=0):
    """NaN scales and the largest codes into every slot that no token of any request sees."""
    hide = torch.from_numpy(~seen_slots(b, window, sinks))[:, None, :, None]
    for pool in (b.k_pool, b.v_pool):
        codes, scales = rows_of(pool)
        codes[hide.expand(codes.shape)] = 0x77
        scales[hide.expand(scales.shape)] = 0x7F


def step(b, db, window=None, sinks=0, C=None, tile=None, stream=None, sm_scale=None):
    """Plan, attention and combine over 4-bit pages: (ws, out, lse) on the device."""
    count = hpa.hpa_default_num_ctas if window is None else hpa.hpa_default_num_ctas_window
    C = C or count(b.Hkv, b.q_len, hpa.KV_E2M1, b.Hq)
    ws = hpa.Workspace(b.B, b.q_len, b.Hq, b.d, num_ctas=C, Hkv=b.Hkv, window=window, sinks=sinks)
    ws.partial_o.fill_(float("nan"))
    ws.partial_lse.fill_(float("nan"))
    out = torch.full((b.B, b.q_len, b.Hq, b.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.B, b.q_len, b.Hq), float("nan"), dtype=torch.float32, device="cuda")
    if stream is not None:
        torch.cuda.synchronize()          # the buffers above were filled on the current stream
    hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks, db.vs,
                    tile=tile, stream=stream, sm_scale=sm_scale)
    return ws, out, lse
