"""Key weights under a window map that was altered after the plan: no accumulator but those the
undamaged map updates is touched."""
import pytest
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from gpu_helpers import DeviceBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["request", "tiles", "owner", "partition", "window", "sinks",
                                 "length"])
def test_damaged_window_maps_change_no_other_weight(how):
    """Every accumulator is what it was or what the undamaged map gives it, and slots that no
    token sees are what they were."""
    b = W.make_batch([700, 300], q_len=1, seed=72, Hq=16, Hkv=2)
    db = DeviceBatch(b)
    lse = torch.full((2, 1, 16), 5.0, device="cuda")
    n_b, n_c = 2, 6
    segs = ((16 + n_b + 2 * (n_b + 1) + 2 * (n_c + 1)) + 3) & ~3
    cta_seg = 16 + n_b + (n_b + 1) + (n_c + 1)
    where, value = {"request": (segs, 5), "tiles": (segs + 2, 10000), "owner": (segs + 3, 3),
                    "partition": (cta_seg + 1, 1000), "window": (11, 0), "sinks": (12, -1),
                    "length": (16, 0)}[how]
    results = []
    for damaged in (False, True):
        ws = hpa.Workspace(2, 1, 16, 128, num_ctas=6, Hkv=2, window=256, sinks=4)
        ws.plan(db.lens)
        if damaged:
            ws.taskmap[where] = value
        acc = torch.full((b.num_pages, 2, 64), 3.0, device="cuda")
        hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, db.indices, ws.taskmap, 6, acc)
        torch.cuda.synchronize()
        assert bool(ws.status() & (32 | 1)) == damaged
        results.append(acc)
    whole, acc = results
    assert ((acc == 3.0) | (acc == whole)).all()
    assert (acc != 3.0).any() == (how not in ("window", "sinks"))
    pos = {int(p): (r, i) for r in range(2)
           for i, p in enumerate(b.page_indices[b.page_indptr[r]:b.page_indptr[r + 1]])}
    lens, low = (700, 300), (700 - 256, 300 - 256)
    for p in range(b.num_pages):
        r, i = pos[p]
        key = torch.arange(64 * i, 64 * i + 64, device="cuda")
        seen = (key < lens[r]) & ((key < 4) | (key >= low[r]))
        assert (acc[p][:, ~seen] == 3.0).all()
