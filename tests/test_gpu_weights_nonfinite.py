"""Key weights where scores are not finite: a key of score -inf weighs nothing, whatever the
number of query rows, and a row whose lse is -inf adds nothing, whatever its query holds."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from bounded_helpers import assert_within, weight_bound
from gpu_helpers import DeviceBatch
from oracle import bounded

pytestmark = pytest.mark.gpu

HEADS = [((8, 1), 1), ((5, 1), 1), ((3, 1), 1), ((12, 3), 1), ((5, 1), 2), ((17, 1), 1),
         ((40, 8), 5), ((33, 1), 1), ((7, 1), 7), ((8, 1), 8)]


def _run(b, lse, decay, window=None, sinks=0):
    acc0 = torch.rand((b.num_pages, b.Hkv, 64), generator=torch.Generator().manual_seed(1))
    kv = hpa.KV_BF16 if b.kv_dtype == "bf16" else hpa.KV_E4M3
    db = DeviceBatch(b)
    ws = hpa.Workspace(b.B, b.q_len, b.Hq, b.d, Hkv=b.Hkv, window=window, sinks=sinks,
                       num_ctas=hpa.hpa_default_num_ctas(b.Hkv, b.q_len, kv, b.Hq))
    ws.plan(db.lens)
    acc = acc0.cuda()
    hpa.hpa_key_weights(db.q, torch.from_numpy(lse).cuda(), db.k, db.indptr, db.indices,
                        ws.taskmap, ws.num_ctas, acc, k_scale=db.ks, decay=decay)
    torch.cuda.synchronize()
    assert ws.status() == 0
    return acc.cpu().numpy(), acc0.numpy()


def _check(b, lse, decay=0.5, window=None, sinks=0):
    """Rows whose lse is -inf have no part in the sums; their queries are zero in the copy that
    the definition sees, so that the bound does not go by them."""
    got, acc0 = _run(b, lse, decay, window, sinks)
    q = b.q.clone()
    q[torch.from_numpy(np.isneginf(lse))] = 0
    ref, written, E = bounded.key_weights(dataclasses.replace(b, q=q), lse, acc0, decay, window,
                                          sinks)
    E = np.where(np.isfinite(E), E, 0.0)                      # a weight of zero is exact
    bound = weight_bound(ref, E) + 2.0 ** -23 * np.abs(acc0)  # and is added to the prior
    assert_within(got[written], ref[written], bound[written], "acc")
    assert (got[~written] == acc0[~written]).all()
    return got


def _lse(b, window=None, sinks=0):
    return bounded.attention_rows(b, window, sinks)[1].astype(np.float32)


@pytest.mark.parametrize("heads,q_len", HEADS)
@pytest.mark.parametrize("windowed", [False, True])
def test_infinite_keys_of_score_minus_infinity(heads, q_len, windowed):
    """Dim 7 of every query is negative, and +inf in some keys: the last new one, the first,
    one inside a page and a whole page of them."""
    win = dict(window=150, sinks=3) if windowed else {}
    b = W.make_batch([q_len + 1, 200, 333], q_len=q_len, seed=heads[0], Hq=heads[0], Hkv=heads[1])
    b.q[..., 7] = -b.q[..., 7].abs() - 0.25
    for r, keys in ((0, [0]), (1, [0, 77, 199]), (2, list(range(192, 256)) + [332])):
        ids = b.page_indices[b.page_indptr[r]:b.page_indptr[r + 1]]
        for i in keys:
            b.k_pool[ids[i // 64], :, i % 64, 7] = math.inf
    got = _check(b, _lse(b, **win), **win)
    assert not np.isnan(got).any()


@pytest.mark.parametrize("heads,q_len", HEADS)
def test_a_score_of_plus_infinity_stays_infinite(heads, q_len):
    """With a finite lse the weight is infinite, and that of the other keys is not touched."""
    b = W.make_batch([200], q_len=q_len, seed=heads[0], Hq=heads[0], Hkv=heads[1])
    lse = _lse(b)
    b.q[..., 7] = b.q[..., 7].abs() + 0.25
    lse += 20.0
    b.k_pool[b.page_indices[1], :, 5, 7] = math.inf
    got = _check(b, lse)
    assert np.isposinf(got[b.page_indices[1], :, 5]).all() and np.isinf(got).sum() == heads[1]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("fill", [math.nan, math.inf, 1e38])
@pytest.mark.parametrize("heads,q_len", HEADS)
def test_rows_of_lse_minus_infinity_add_nothing(kv, fill, heads, q_len):
    """A batch whose padded rows hold anything: the first token's, some heads', and all of one
    request's, whose keys hold NaN as well."""
    b = W.make_batch([300, 130, 65], q_len=q_len, kv_dtype=kv, seed=heads[0], Hq=heads[0],
                     Hkv=heads[1])
    lse = _lse(b)
    if q_len > 1:
        lse[0, 0] = -math.inf
    lse[1, :, ::3] = -math.inf
    lse[2] = -math.inf
    b.q[torch.from_numpy(np.isneginf(lse))] = fill
    ids = b.page_indices[b.page_indptr[2]:b.page_indptr[3]]
    b.k_pool[ids[0], :, 9] = math.nan if kv == "bf16" else 0x7F
    got = _check(b, lse)
    assert not np.isnan(got).any()


@pytest.mark.parametrize("heads,q_len", [((5, 1), 2), ((8, 1), 8), ((12, 3), 3)])
def test_hidden_rows_and_dead_rows_together(heads, q_len):
    """The one live row of a request does not see its last keys, which are infinite: they
    receive nothing, and the live row's own keys their weight."""
    b = W.make_batch([130, 257], q_len=q_len, seed=3, Hq=heads[0], Hkv=heads[1])
    lse = _lse(b)
    lse[:, 1:] = -math.inf
    for r, L in enumerate((130, 257)):
        ids = b.page_indices[b.page_indptr[r]:b.page_indptr[r + 1]]
        for i in range(L - q_len + 1, L):
            b.k_pool[ids[i // 64], :, i % 64, ::2] = math.inf
            b.k_pool[ids[i // 64], :, i % 64, 1::2] = math.nan
    got = _check(b, lse)
    assert not np.isnan(got).any()
