"""Helpers for the bounded-cache GPU tests: error bounds from the arithmetic, poisoned
batches, and one windowed step through the library.

Bounds.  A score is a dot product of 128 products with fp32 accumulation, each addition off
by at most 2^-22 of the running magnitude (a truncating adder loses a whole unit, not half):
128 * 2^-22 * E for E = sm_scale * sum |q k|, and a few roundings of the scaled exponent.  A
weight exp(s - lse) is then off by that much relative to itself; an output, whose numerator
and denominator both hold such weights, by twice as much of A = sum w |v|, plus the rounding
of the probabilities for the second MMA (bf16 2^-8, f16 2^-11 of each) and of the bf16 result
(2^-8 of it)."""
import numpy as np
import torch

import load_balanced_split_gb300 as hpa
from oracle import bounded

DOT = 128 * 2.0 ** -22 + 8 * 2.0 ** -24
EXP = 2.0 ** -20          # exp2 / log2 approximations and fp32 sums of a few terms


def out_bound(ref, A, E, kv, rounded=True):
    p = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    return (p + 2 * DOT * E[..., None] + 2 * EXP) * A + (2.0 ** -8 * np.abs(ref) if rounded else 0)


def lse_bound(ref, E):
    return DOT * E + EXP * (1 + np.abs(ref))


def weight_bound(ref, E, lse_abs=20.0):
    return np.abs(ref) * (DOT * E + EXP * (1 + lse_abs))


def assert_within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    fine = np.isfinite(ref)
    assert (np.isnan(got) == np.isnan(ref)).all(), "%s: NaN pattern differs" % what
    inf = np.isinf(ref)
    assert (got[inf] == ref[inf]).all(), "%s: infinities differ" % what
    d = np.abs(got[fine] - ref[fine])
    bad = ~(d <= np.broadcast_to(bound, ref.shape)[fine])
    assert not bad.any(), "%s: %d of %d out of bound, worst %g at ref %g" % (
        what, bad.sum(), bad.size, d[bad].max(), ref[fine][bad][d[bad].argmax()])


def nan_code(kv):
    return float("nan") if kv == "bf16" else 0x7F


def poison_hidden(b, window=None, sinks=0):
    """NaN into every K and V slot that no token of any request sees."""
    seen = np.zeros((b.num_pages, 64), bool)
    for r in range(b.B):
        L = int(b.seq_lens[r])
        ids = b.page_indices[int(b.page_indptr[r]):int(b.page_indptr[r + 1])]
        for i in range(L):
            if any(bounded.sees(L, b.q_len, j, i, window, sinks) for j in range(b.q_len)):
                seen[ids[i // 64], i % 64] = True
    hide = torch.from_numpy(~seen)[:, None, :, None].expand(b.k_pool.shape)
    for pool in (b.k_pool, b.v_pool):
        pool[hide] = nan_code(b.kv_dtype)
    return seen


def window_step(b, db, window, sinks, C=None, tile=None, acc=None, decay=1.0, stream=None):
    """Plan, windowed attention, combine (and weights): (ws, out, lse) on the device."""
    kv = hpa.KV_BF16 if b.kv_dtype == "bf16" else hpa.KV_E4M3
    C = C or hpa.hpa_default_num_ctas_window(b.Hkv, b.q_len, kv, b.Hq)
    ws = hpa.Workspace(b.B, b.q_len, b.Hq, b.d, num_ctas=C, Hkv=b.Hkv, window=window, sinks=sinks)
    ws.partial_o.fill_(float("nan"))
    ws.partial_lse.fill_(float("nan"))
    out = torch.full((b.B, b.q_len, b.Hq, b.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.B, b.q_len, b.Hq), float("nan"), dtype=torch.float32, device="cuda")
    if stream is not None:
        torch.cuda.synchronize()          # the buffers above were filled on the current stream
    hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks, db.vs,
                    tile=tile, acc=acc, decay=decay, stream=stream)
    return ws, out, lse


def check_attention(b, out, lse, ref, kv):
    o, l, A, E = ref
    assert_within(out.float().cpu().numpy(), o, out_bound(o, A, E, kv), "out")
    assert_within(lse.cpu().numpy(), l, lse_bound(l, E), "lse")
