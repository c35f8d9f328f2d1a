"""The keys a tile of a plan: one default for 4-bit pages, whoever makes the plan (no GPU: the plan's
call is recorded)."""
import pytest

import load_balanced_split_gb300 as hpa
from load_balanced_split_gb300 import hpa as binding


@pytest.mark.parametrize("kv,window,tile", [(hpa.KV_E2M1, None, 256), (hpa.KV_E4M3, None, 512),
                                            (hpa.KV_BF16, None, 512), (None, None, 512),
                                            (hpa.KV_E2M1, 100, 64), (None, 100, 64)])
def test_default_tile(kv, window, tile, monkeypatch):
    seen = []
    monkeypatch.setattr(binding, "hpa_plan", lambda lens, t, *a: seen.append(t))
    monkeypatch.setattr(binding, "hpa_plan_window", lambda lens, q, w, s, t, *a: seen.append(t))
    ws = hpa.Workspace(2, 1, 16, 128, num_ctas=4, device="cpu", Hkv=2, window=window, kv_dtype=kv)
    ws.plan(None)
    ws.plan(None, 128)
    assert seen == [tile, 128]
