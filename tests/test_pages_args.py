"""Page tables: refusals on the host (nothing is launched) and the oracle's own properties, on CPU."""
import random

import pytest
import torch

import load_balanced_split_gb300 as hpa
from oracle import paging

FAKE = 1 << 20  # a 16-byte aligned non-null value; never dereferenced by these calls


def _call(**kw):
    at = iter(range(FAKE, FAKE + (100 << 16), 1 << 16))
    a = dict(lens=next(at), new=next(at), rows=next(at), off=next(at), B=3, num_rows=5,
             table=next(at), stride=7, held=None, held_out=next(at), free=next(at), fin=None,
             fout=next(at), P=40, page=64, ip=next(at), ix=next(at), cap=40, slots=next(at),
             pos=next(at), tokens=9, ws=next(at), nb=hpa.hpa_assign_pages_workspace(3, 5), st=None)
    a["held"], a["fin"] = a["held_out"], a["fout"]
    a.update(kw)
    return hpa.lib().hpa_assign_pages(*a.values(), None)


def test_argument_checks():
    for name in ("lens", "table", "held", "held_out", "free", "fin", "fout", "ip", "ix", "ws",
                 "slots", "pos"):
        assert _call(**{name: None}) == -1, name
    for bad in (dict(B=0), dict(num_rows=0), dict(stride=0), dict(P=0), dict(cap=-1),
                dict(tokens=-1), dict(rows=None, B=6, nb=1 << 20)):
        assert _call(**bad) == -1, bad
    assert _call(page=32) == -2
    assert _call(nb=hpa.hpa_assign_pages_workspace(3, 5) - 4) == -3
    assert _call(ws=FAKE + (90 << 16) + 8) == -4 and _call(slots=FAKE + (90 << 16) + 4) == -4
    for name in ("lens", "new", "rows", "off", "table", "free", "ip", "ix", "pos", "st"):
        assert _call(**{name: FAKE + (90 << 16) + 2}) == -4, name
    # arrays that are written lie apart
    table = FAKE + (70 << 16)
    for name in ("lens", "new", "rows", "off", "free", "ip", "ix", "slots", "pos", "ws", "held"):
        other = table + 4 * 5 * 7 - 4
        other -= other % 16
        assert _call(table=table, **{name: other}) == -1, name


def test_workspace_sizes():
    assert hpa.hpa_assign_pages_workspace(0, 4) == 0 and hpa.hpa_assign_pages_workspace(4, 0) == 0
    assert hpa.hpa_assign_pages_workspace(10, 20) > hpa.hpa_assign_pages_workspace(10, 10) > 0


def test_binding_refusals():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(hpa.HpaError, match="CUDA tensor"):
        hpa.hpa_assign_pages(t, None, t.view(2, 2), t, t, t, t, t, None, None, t)
    with pytest.raises(hpa.HpaError, match="out of range"):
        hpa.PageTable(0, 4, 4, device="cpu")
    pt = hpa.PageTable(8, 4, 4, max_batch=2, device="cpu")
    assert pt.free_pages.tolist() == [7, 6, 5, 4, 3, 2, 1, 0] and pt.free_count.tolist() == [8]
    with pytest.raises(hpa.HpaError, match="room for 2"):
        pt.assign(torch.zeros(3, dtype=torch.int32))


def test_oracle_keeps_every_page_once():
    rng = random.Random(1)
    rows, stride, P = 7, 9, 30
    table, held, free = [[-1] * stride for _ in range(rows)], [0] * rows, list(range(P))
    full = 0
    for _ in range(300):
        B = rng.randint(1, rows)
        which = rng.sample(range(rows), B)
        lens = [rng.choice([0, rng.randint(1, 64 * stride)]) for _ in range(B)]
        new = [rng.randint(0, x) for x in lens]
        (table, held, free), (indptr, ix), (slots, pos), status = paging.assign(
            lens, new, table, held, free, P, which)
        owned = [p for r in range(rows) for p in table[r][:held[r]]]
        assert sorted(owned + free) == list(range(P))
        full += status == paging.NO_PAGES
        assert status in (0, paging.NO_PAGES) and len(slots) == len(pos) == sum(new)
        for r in range(B):
            mine = ix[indptr[r]:indptr[r + 1]]
            assert mine == table[which[r]][:held[which[r]]]
            t = slots[sum(new[:r]):sum(new[:r + 1])]
            assert all(x == -1 for x in t) or [x // 64 for x in t] == [
                mine[i // 64] for i in range(lens[r] - new[r], lens[r])]
    assert 0 < full < 300


def test_oracle_order():
    """Returned pages go on top in order, and the top comes off first."""
    (table, held, free), _, (slots, pos), _ = paging.assign(
        [64, 0, 129], [1, 0, 129], [[5, 6, 7], [8, 9, 0], [0, 0, 0]], [3, 2, 0], [1, 2], 10)
    assert free == [1, 2, 6] and held == [1, 0, 3]     # the stack was 1 2 6 7 8 9 before r = 2
    assert table[2] == [9, 8, 7] and slots[0] == 5 * 64 + 63 and slots[1] == 9 * 64
    assert pos[:3] == [63, 0, 1]
