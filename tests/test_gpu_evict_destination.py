"""Eviction to other pages whose list is too short or wrong: the request is refused whole
(length -1, nothing moved), and the others are served."""
import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from gpu_helpers import DeviceBatch
from oracle import bounded

pytestmark = pytest.mark.gpu

LENS, BUDGETS, HKV = [300, 500, 90, 20000], [100, 130, 200, 9000], 2
PAGES = [(min(L, n) + 63) // 64 for L, n in zip(LENS, BUDGETS)]


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("who", [0, 1, 2, 3])
@pytest.mark.parametrize("how", ["short", "empty", "backwards", "negative", "beyond", "last",
                                 "none"])
def test_a_bad_destination_refuses_its_request(kv, who, how):
    """Request 2 is within its budget (moved whole), request 3 takes a cluster of blocks."""
    spare = sum(PAGES)
    b = W.make_batch(LENS, kv_dtype=kv, seed=7, Hq=HKV, Hkv=HKV)
    db = DeviceBatch(b)
    k = torch.cat([db.k, torch.full_like(db.k[:1], 3).expand(spare, -1, -1, -1)]).contiguous()
    v = torch.cat([db.v, torch.full_like(db.v[:1], 4).expand(spare, -1, -1, -1)]).contiguous()
    acc = torch.rand((k.shape[0], HKV, 64), device="cuda")
    lists = np.split(b.num_pages + np.random.default_rng(1).permutation(spare),
                     np.cumsum(PAGES)[:-1])
    n = np.array(PAGES)
    if how == "short":
        lists[who] = lists[who][:-1]
    elif how == "empty":
        lists[who] = lists[who][:0]
    elif how in ("negative", "beyond", "last"):
        lists[who][-1 if how == "last" else 0] = {"negative": -1, "beyond": k.shape[0],
                                                  "last": 1 << 30}[how]
    ptr = np.concatenate([[0], np.cumsum([len(x) for x in lists])])
    if how == "backwards":                   # a list that ends before it begins
        ptr[who + 1:] = ptr[who] - 1 if who else -1
        ptr = np.maximum(ptr, 0) if who == 0 else ptr
    kept = torch.full((4, HKV, max(BUDGETS)), -9, dtype=torch.int32, device="cuda")
    new, st = _dev([7] * 4), _dev([0])
    k0, v0, a0 = k.clone(), v.clone(), acc.clone()
    hpa.evict_step(acc, k, v, db.lens, db.indptr, db.indices, _dev(BUDGETS), 2, 20, kept, new,
                   dst_indptr=_dev(ptr), dst_indices=_dev(np.concatenate(lists)), status=st)
    torch.cuda.synchronize()
    if how == "backwards":                   # the lists after it have moved: only its own counts
        assert int(st.item()) == 4 and int(new[who]) == -1 and (kept[who] == -9).all()
        return
    refused = [] if how == "none" else [who]
    assert int(st.item()) == (4 if refused else 0)
    ek, ev, ea = k0.clone(), v0.clone(), a0.clone()
    for r, (L, budget) in enumerate(zip(LENS, BUDGETS)):
        m = min(L, budget)
        if r in refused:
            assert int(new[r]) == -1 and (kept[r] == -9).all()
            continue
        assert int(new[r]) == m and len(lists[r]) == n[r]
        ids = b.page_indices[b.page_indptr[r]:b.page_indptr[r + 1]]
        t = np.arange(m)
        for h in range(HKV):
            w = a0[ids, h].reshape(-1)[:L].cpu().numpy()
            want = np.array(bounded.kept_keys(list(w), budget, 2, 20))
            assert (kept[r, h, :m].cpu().numpy() == want).all()
            src, dst = (ids[want // 64], h, want % 64), (lists[r][t // 64], h, t % 64)
            for e, x in ((ek, k0), (ev, v0), (ea, a0)):
                e[dst] = x[src]
    raw = lambda x: x.view(torch.int16 if kv == "bf16" else torch.uint8)  # noqa: E731
    assert torch.equal(raw(k), raw(ek)) and torch.equal(raw(v), raw(ev)) and torch.equal(acc, ea)


def test_selection_alone_and_in_place_know_no_destination():
    """hpa_evict without a second table, and hpa_evict_select, go by the source alone."""
    b = W.make_batch(LENS, seed=8, Hq=HKV, Hkv=HKV)
    db = DeviceBatch(b)
    acc = torch.rand((b.num_pages, HKV, 64), device="cuda")
    outs = []
    for call in ("select", "step"):
        kept = torch.full((4, HKV, max(BUDGETS)), -9, dtype=torch.int32, device="cuda")
        new, st = _dev([7] * 4), _dev([0])
        if call == "select":
            hpa.hpa_evict_select(acc, db.lens, db.indptr, db.indices, _dev(BUDGETS), 2, 20, kept,
                                 new, st)
        else:
            hpa.evict_step(acc, db.k, db.v, db.lens, db.indptr, db.indices, _dev(BUDGETS), 2, 20,
                           kept, new, status=st)
        assert int(st.item()) == 0 and new.tolist() == [min(a, c) for a, c in zip(LENS, BUDGETS)]
        outs.append(kept)
    assert torch.equal(*outs)
