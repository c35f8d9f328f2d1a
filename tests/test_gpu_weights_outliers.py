"""Key weights with outlier query elements: rows whose largest element is thousands of times
the others, and rows of very different size side by side."""
import math

import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from bounded_helpers import DOT, EXP, assert_within
from gpu_helpers import DeviceBatch
from oracle import bounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("power", [4, 9, 12, 15])
@pytest.mark.parametrize("heads,q_len", [((8, 1), 1), ((5, 1), 2), ((32, 1), 2)])
def test_outlier_elements(kv, power, heads, q_len):
    """Dim 7 of a row is 2^power times the others, against keys that are small there.

    With E4M3 pages a query element is two E4M3 terms of a row scaled so that its largest
    element amax lies in [128, 256): hi to 4 significant bits, and 16 times the rest, which a
    bf16 leaves at most 4 bits, so it is exact but where E4M3 is subnormal: then off by at most
    half of 2^-9, over 16, of the scaled row: 2^-14 / 128 = 2^-21 of amax.  A score is off by
    sm_scale times that times sum |k|, beyond the accumulation's share."""
    b = W.make_batch([200, 333], q_len=q_len, kv_dtype=kv, seed=power, Hq=heads[0],
                     Hkv=heads[1])
    sizes = torch.tensor([1.0, 2.0 ** -3, 2.0 ** -6])[torch.arange(heads[0]) % 3]
    b.q *= sizes[:, None].to(b.q.dtype)
    b.q[..., 7] = (b.q[..., 8].abs() + 0.1 * sizes) * 2.0 ** power
    if kv == "bf16":
        b.k_pool[..., 7] *= 2.0 ** -power
    else:
        b.k_pool[..., 7] &= 0x83                         # subnormal codes: up to 3 * 2^-9
    lse = bounded.attention_rows(b)[1].astype(np.float32)
    db = DeviceBatch(b)
    ws = hpa.Workspace(2, q_len, heads[0], 128, Hkv=heads[1], num_ctas=5)
    ws.plan(db.lens)
    acc = torch.zeros((b.num_pages, heads[1], 64), device="cuda")
    hpa.hpa_key_weights(db.q, torch.from_numpy(lse).cuda(), db.k, db.indptr, db.indices,
                        ws.taskmap, 5, acc, k_scale=db.ks)
    ref, written, E = bounded.key_weights(b, lse, np.zeros(acc.shape), 1.0)
    assert ws.status() == 0
    K = np.abs(bounded.pool_values(b.k_pool, kv, b.k_scale)).sum(-1)         # [P][Hkv][page]
    amax = float(b.q.abs().max())
    terms = 2.0 ** -21 * amax * K / math.sqrt(128) if kv == "e4m3" else 0.0
    # |lse| is at most ln(333) + the largest score, E
    bound = np.abs(ref) * (np.expm1(DOT * E + terms) + EXP * (8 + E))
    assert_within(acc.cpu().numpy()[written], ref[written], bound[written], "acc")
    assert ref[written].max() > 1e-3
    assert power > 12 or (bound[written] < 0.05 * ref[written]).all()
