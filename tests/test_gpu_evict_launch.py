"""How many blocks a selection gets does not hang on how small the budget is."""
import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa

pytestmark = pytest.mark.gpu


def _time(B, Hkv, L, budget, spare=1, reps=15):
    """(us of one selection, median of `reps` on flushed caches; kept; weights by request)."""
    npg = (L + 63) // 64
    P = B * npg * spare
    g = torch.Generator(device="cuda").manual_seed(L)
    acc = torch.rand((P, Hkv, 64), generator=g, device="cuda")
    idx = torch.randperm(P, generator=g, device="cuda")[:B * npg].to(torch.int32)
    ptr = (torch.arange(B + 1, device="cuda") * npg).to(torch.int32)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    budgets = torch.full((B,), budget, dtype=torch.int32, device="cuda")
    kept = torch.full((B, Hkv, budget), -9, dtype=torch.int32, device="cuda")
    new, st = torch.zeros_like(lens), torch.zeros(1, dtype=torch.int32, device="cuda")
    flush = torch.empty(192 << 20, dtype=torch.uint8, device="cuda")
    times = []
    for _ in range(reps):
        flush.zero_()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        hpa.hpa_evict_select(acc, lens, ptr, idx, budgets, 0, 0, kept, new, st)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    assert int(st.item()) == 0 and (new == budget).all()
    w = acc[idx.long()].view(B, npg, Hkv, 64).permute(0, 2, 1, 3).reshape(B, Hkv, -1)[..., :L]
    return float(np.median(times)), kept, w


@pytest.mark.parametrize("B,L", [(1, 196608), (1, 100000), (4, 190001)])
def test_small_budgets_of_long_requests(B, L):
    """Cut to 64 or 2 keys as to 16384: the weights are walked by as many blocks.  With the
    blocks chosen by the budget they took several times as long."""
    wide = _time(B, 8, L, 16384)[0]
    for budget in (2, 64, 300):
        us, kept, w = _time(B, 8, L, budget)
        # of equal weights (a 24-bit uniform of 190000 has a few) the lower index stays
        order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
        assert torch.equal(kept.long(), order.sort(-1).values), budget
        assert us < 1.5 * wide, (budget, us, wide)
