"""A map planned once for many layers is the one that decode_step plans by itself."""
import pytest
import torch

import load_balanced_split_gb300 as hpa
from fourbit_helpers import make_batch
from gpu_helpers import DeviceBatch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [None, 300])
@pytest.mark.parametrize("lens", [[900], [3000, 200, 64, 1000]])
def test_planned_once_and_planned_each_time(lens, window):
    b = make_batch(lens, 2, (16, 2), seed=130)
    db = DeviceBatch(b)
    count = hpa.hpa_default_num_ctas if window is None else hpa.hpa_default_num_ctas_window
    maps, results = [], []
    for kv in (hpa.KV_E2M1, None):
        ws = hpa.Workspace(b.B, 2, b.Hq, 128, num_ctas=count(b.Hkv, 2, hpa.KV_E2M1, b.Hq), Hkv=b.Hkv,
                           window=window, kv_dtype=kv)
        out = torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(b.q.shape[:3], device="cuda")
        once = kv is not None
        if once:
            ws.plan(db.lens)
        for _ in range(2):
            hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks,
                            db.vs, plan=not once)
        torch.cuda.synchronize()
        assert ws.status() == 0
        maps.append(ws.taskmap)
        results.append((out, lse))
    assert torch.equal(*maps)
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
