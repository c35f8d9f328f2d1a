"""Host-side refusals of the bounded-cache entry points (nothing is launched), on CPU."""
import pytest
import torch

import load_balanced_split_gb300 as hpa

FAKE = 1 << 20  # a 16-byte aligned non-null value; never dereferenced by these calls


def test_plan_window_argument_checks():
    L = hpa.lib()
    nb = hpa.hpa_taskmap_bytes(3, 4)

    def call(**kw):
        a = dict(lens=FAKE, B=3, q_len=1, window=100, sinks=4, tile=64, C=4, tm=FAKE, nb=nb)
        a.update(kw)
        return L.hpa_plan_window(a["lens"], a["B"], a["q_len"], a["window"], a["sinks"], a["tile"],
                                 a["C"], a["tm"], a["nb"], None)

    for bad in (dict(lens=None), dict(tm=None), dict(B=0), dict(q_len=0), dict(window=0),
                dict(window=-5), dict(sinks=-1), dict(tile=100), dict(tile=0), dict(C=0)):
        assert call(**bad) == -1, bad
    assert call(nb=nb - 4) == -3
    assert call(tm=FAKE + 4) == -4


def test_window_attention_argument_checks():
    L = hpa.lib()

    def call(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, kv=0, ks=None, vs=None, P=100, ip=FAKE, ix=FAKE, page=64,
                 B=3, q_len=1, Hq=64, Hkv=8, d=128, scale=0.088, tm=FAKE, C=4, po=FAKE, pl=FAKE)
        a.update(kw)
        return L.hpa_decode_attn_window(*a.values(), None)

    assert call(q=None) == -1 and call(kv=2) == -1 and call(kv=1) == -1
    assert call(scale=float("inf")) == -1
    assert call(d=64) == -2 and call(page=16) == -2 and call(Hq=60) == -2 and call(q_len=9) == -2
    assert call(k=FAKE + 8) == -4


def test_key_weights_argument_checks():
    L = hpa.lib()

    def call(**kw):
        a = dict(q=FAKE, lse=FAKE, k=FAKE, kv=0, ks=None, P=100, ip=FAKE, ix=FAKE, page=64, B=3,
                 q_len=1, Hq=64, Hkv=8, d=128, scale=0.088, decay=1.0, tm=FAKE, C=4, a0=FAKE,
                 a1=FAKE)
        a.update(kw)
        return L.hpa_key_weights(*a.values(), None)

    for name in ("q", "lse", "k", "ip", "ix", "tm", "a1"):
        assert call(**{name: None}) == -1, name
    assert call(kv=1) == -1 and call(kv=9) == -1 and call(C=0) == -1 and call(q_len=0) == -1
    for decay in (-0.5, float("nan"), float("inf")):
        assert call(decay=decay) == -1
    assert call(d=64) == -2 and call(page=32) == -2 and call(q_len=9) == -2
    assert call(P=1 << 29) == -2 and call(Hq=63) == -2
    for name in ("a0", "a1", "k", "tm"):
        assert call(**{name: FAKE + 8}) == -4, name
    for name in ("lse", "ip", "ix"):
        assert call(**{name: FAKE + 2}) == -4, name
    size = 100 * 8 * 64 * 4                          # a pool of weights that overlaps the other
    for a0, a1 in ((FAKE, FAKE + size - 16), (FAKE + size - 16, FAKE)):
        assert call(a0=a0, a1=a1) == -1


def test_evict_select_argument_checks():
    L = hpa.lib()

    def call(**kw):
        a = dict(acc=FAKE, lens=FAKE, ip=FAKE, ix=FAKE, P=100, page=64, budgets=FAKE + 64, sinks=4,
                 recent=8, B=3, Hkv=8, kept=FAKE, stride=100, new=FAKE + 128, st=None)
        a.update(kw)
        return L.hpa_evict_select(*a.values(), None)

    for name in ("acc", "lens", "ip", "ix", "budgets", "kept", "new"):
        assert call(**{name: None}) == -1, name
    for bad in (dict(sinks=-1), dict(recent=-1), dict(B=0), dict(Hkv=0), dict(stride=0),
                dict(P=0), dict(new=FAKE), dict(new=FAKE + 64)):    # new_lens over its inputs
        assert call(**bad) == -1, bad
    assert call(page=32) == -2 and call(B=1 << 24, Hkv=1000) == -2
    assert call(acc=FAKE + 4) == -4 and call(st=FAKE + 2) == -4
    for name in ("lens", "ip", "ix", "budgets", "kept"):
        assert call(**{name: FAKE + 66}) == -4, name
    assert call(new=FAKE + 130) == -4
    assert call(new=FAKE + 8) == -1 and call(new=FAKE + 60) == -1  # overlaps lens, budgets


def test_evict_compact_argument_checks():
    L = hpa.lib()

    def call(**kw):
        a = dict(k=FAKE, v=2 * FAKE + (100 << 17), kv=0, acc=None, P=100, ip=FAKE, ix=FAKE, dip=None, dix=None,
                 page=64, kept=FAKE, stride=100, new=FAKE, B=3, Hkv=8, d=128, st=None)
        a.update(kw)
        return L.hpa_evict_compact(*a.values(), None)

    for name in ("k", "v", "ip", "ix", "kept", "new"):
        assert call(**{name: None}) == -1, name
    assert call(dip=FAKE) == -1 and call(dix=FAKE) == -1           # one half of a page table
    assert call(v=FAKE) == -1 and call(v=FAKE + (100 << 17) - 16) == -1   # one pool over the other
    assert call(k=FAKE + (100 << 17), v=2 * FAKE) == -1
    for name in ("ip", "ix", "kept", "new", "acc"):
        assert call(**{name: FAKE + 2}) == -4, name
    assert call(dip=FAKE + 2, dix=FAKE) == -4 and call(dip=FAKE, dix=FAKE + 2) == -4
    assert call(kv=3) == -1 and call(stride=0) == -1
    assert call(d=64) == -2 and call(page=128) == -2
    assert call(k=FAKE + 8) == -4


def test_store_kv_at_argument_checks():
    L = hpa.lib()

    def call(**kw):
        a = dict(k=FAKE, v=FAKE, lens=FAKE, text=FAKE, ip=FAKE, ix=FAKE, P=10, page=64, cs=FAKE,
                 maxpos=100, w=FAKE, eps=1e-6, had=1, kv=0, ks=None, vs=None, kp=FAKE, vp=FAKE,
                 B=2, q=1, Hkv=8, d=128, st=None)
        a.update(kw)
        return L.hpa_store_kv_at(*a.values(), None)

    assert call(text=None) == -1 and call(k=None) == -1 and call(kv=1) == -1
    assert call(d=64) == -2
    assert call(cs=FAKE + 4) == -4


def test_workspace_and_step_combinations():
    with pytest.raises(hpa.HpaError, match="dynamic plan"):
        hpa.Workspace(2, 1, 8, 128, splits=2, window=10, device="cpu", Hkv=1)
    with pytest.raises(hpa.HpaError, match="dynamic plan"):
        hpa.Workspace(2, 1, 8, 128, num_ctas=2, window=10, weighted=True, device="cpu", Hkv=1)
    with pytest.raises(hpa.HpaError, match="with a window"):
        hpa.Workspace(2, 1, 8, 128, num_ctas=2, sinks=4, device="cpu", Hkv=1)
    ws = hpa.Workspace(2, 1, 8, 128, num_ctas=2, window=10, sinks=4, device="cpu", Hkv=1)
    t = torch.zeros(1)
    for kw in (dict(fused=True), dict(tc=True), dict(allheads=True), dict(mma=True)):
        with pytest.raises(hpa.HpaError, match="one attention kernel"):
            hpa.decode_step(ws, t, t, t, t, t, t, t, **kw)
    with pytest.raises(hpa.HpaError, match="out_lse"):
        hpa.decode_step(ws, t, t, t, t, t, t, t, acc=t)
    plain = hpa.Workspace(2, 1, 8, 128, num_ctas=2, device="cpu", Hkv=1)
    with pytest.raises(hpa.HpaError, match="per KV head"):
        hpa.decode_step(plain, t, t, t, t, t, t, t, t, acc=t, allheads=True)


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4, 1, 64)
    with pytest.raises(hpa.HpaError, match="CUDA tensor"):
        hpa.hpa_evict_select(f, t, t, t, t, 0, 0, t, t)
    with pytest.raises(hpa.HpaError, match="CUDA tensor"):
        hpa.hpa_plan_window(t, 1, 10, 0, 64, 2, t)
