"""Accumulated key weights, selection and compaction against the 64-bit definitions."""
import math

import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from bounded_helpers import assert_within, check_attention, poison_hidden, weight_bound
from gpu_helpers import DeviceBatch
from oracle import bounded, feeder

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- key weights
def _weights(b, window=None, sinks=0, decay=1.0, C=None, splits=None, weighted=False,
             in_place=True, seed=0, acc0=None):
    kv = hpa.KV_BF16 if b.kv_dtype == "bf16" else hpa.KV_E4M3
    _, lse, _, _ = bounded.attention_rows(b, window, sinks)
    poison_hidden(b, window, sinks)
    db = DeviceBatch(b)
    if splits is None:
        C = C or hpa.hpa_default_num_ctas(b.Hkv, b.q_len, kv, b.Hq)
    ws = hpa.Workspace(b.B, b.q_len, b.Hq, b.d, num_ctas=C, Hkv=b.Hkv, window=window, sinks=sinks,
                       splits=splits, weighted=weighted)
    ws.plan(db.lens)
    g = torch.Generator().manual_seed(seed)
    if acc0 is None:
        acc0 = torch.rand((b.num_pages, b.Hkv, 64), generator=g) * 2
    lse = torch.from_numpy(lse.astype(np.float32))
    acc = acc0.cuda()
    out = acc if in_place else torch.full_like(acc, -7.0)
    hpa.hpa_key_weights(db.q, lse.cuda(), db.k, db.indptr, db.indices, ws.taskmap, ws.num_ctas,
                        acc, out=None if in_place else out, k_scale=db.ks, decay=decay)
    torch.cuda.synchronize()
    assert ws.status() == 0
    new, written, E = bounded.key_weights(b, lse.numpy(), acc0.numpy(), decay, window, sinks)
    got = out.cpu().numpy()
    assert_within(got[written], new[written], weight_bound(new, E)[written], "acc")
    if in_place:
        assert (got[~written] == acc0.numpy()[~written]).all(), "an unseen slot was written"
    else:
        same = torch.equal(acc.cpu().view(torch.int32), acc0.view(torch.int32))   # NaN too
        assert (got[~written] == -7.0).all() and same


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,q_len", [((8, 1), 1), ((16, 2), 2), ((5, 1), 1), ((12, 3), 1),
                                         ((8, 1), 3), ((8, 1), 8), ((32, 1), 2), ((17, 1), 1),
                                         ((2, 2), 1), ((40, 8), 5), ((40, 1), 1), ((8, 1), 6)])
def test_weights_head_layouts(kv, heads, q_len):
    b = W.make_batch([q_len, 64, 65, 300, 530], q_len=q_len, kv_dtype=kv, seed=heads[0] + q_len,
                     Hq=heads[0], Hkv=heads[1])
    _weights(b, decay=0.9)


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (70, 65), (300, 1), (1 << 30, 0)])
@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_weights_under_a_window(window, sinks, q_len, kv):
    b = W.make_batch([q_len, 65, 200, 449, 700], q_len=q_len, kv_dtype=kv, seed=window % 91,
                     Hq=8, Hkv=2)
    _weights(b, window, sinks, decay=0.5)


@pytest.mark.parametrize("kw", [dict(C=1), dict(C=50), dict(splits=3), dict(C=7, weighted=True),
                                dict(C=4, in_place=False), dict(C=4, decay=0.0)])
def test_weights_of_every_plan(kw):
    b = W.make_batch([1, 900, 64, 333], seed=11, Hq=16, Hkv=2)
    _weights(b, **kw)


def test_weights_without_prior():
    """acc None starts from zero; decay 0 reads no prior, NaN among it or not."""
    b = W.make_batch([100, 30], seed=12, Hq=8, Hkv=1)
    _weights(b, decay=0.0, acc0=torch.full((b.num_pages, 1, 64), math.nan), in_place=False)
    db = DeviceBatch(b)
    _, lse, _, _ = bounded.attention_rows(b)
    ws = hpa.Workspace(2, 1, 8, 128, num_ctas=3, Hkv=1)
    ws.plan(db.lens)
    out = torch.full((b.num_pages, 1, 64), 5.0, device="cuda")
    z = torch.from_numpy(lse.astype(np.float32))
    z[1] = -math.inf                                       # a row without a key weighs nothing
    hpa.hpa_key_weights(db.q, z.cuda(), db.k, db.indptr, db.indices, ws.taskmap, 3, None, out=out)
    new, written, E = bounded.key_weights(b, z.numpy(), np.full(out.shape, 5.0), 0.0)
    assert_within(out.cpu().numpy(), new, weight_bound(new, E), "acc")


def test_weights_are_the_same_on_every_run():
    b = W.make_batch([5000, 777, 64], q_len=2, kv_dtype="e4m3", seed=13)
    db = DeviceBatch(b)
    lse = torch.full((3, 2, 64), 6.0, device="cuda")
    ws = hpa.Workspace(3, 2, 64, 128, num_ctas=38)
    ws.plan(db.lens)
    runs = []
    for _ in range(3):
        acc = torch.ones((b.num_pages, 8, 64), device="cuda")
        hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, db.indices, ws.taskmap, 38, acc,
                            k_scale=db.ks)
        runs.append(acc)
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_weights_device_side_refusals():
    b = W.make_batch([400, 100], q_len=2, seed=14, Hq=16, Hkv=2)
    db = DeviceBatch(b)
    lse = torch.full((2, 2, 16), 5.0, device="cuda")

    def run(lens, indices, plan_lens=None, C=4):
        ws = hpa.Workspace(2, 2, 16, 128, num_ctas=4, Hkv=2)
        ws.plan(lens)
        acc = torch.full((b.num_pages, 2, 64), 3.0, device="cuda")
        hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, indices, ws.taskmap, C, acc)
        torch.cuda.synchronize()
        return ws.status(), acc.cpu().numpy()

    short = torch.tensor([400, 1], dtype=torch.int32, device="cuda")
    st, acc = run(short, db.indices)
    ids = b.page_indices[int(b.page_indptr[1]):]
    assert st == 1 and (acc[ids] == 3.0).all()             # its keys are left alone
    bad = db.indices.clone()
    bad[2] = -1
    st, acc = run(db.lens, bad)
    assert st == 4 and (acc[int(b.page_indices[2])] == 3.0).all()
    st, acc = run(db.lens, db.indices, C=3)
    assert st == 2 and (acc == 3.0).all()


# ----------------------------------------------------------------------------- selection
def _select(weights, lens, budgets, sinks, recent, stride=None, Hkv=2, seed=0, spare=0):
    """weights: per request [Hkv][L] fp32; spare: pages of the pool that no request has."""
    _, indices, P = W.page_table(seed, np.maximum(np.array(lens), 1), 64, True)
    indptr = np.concatenate([[0], np.cumsum((np.maximum(lens, 1) + 63) // 64)]).astype(np.int32)
    acc = np.full((P + spare, Hkv, 64), 1e30, np.float32)
    for r, L in enumerate(lens):
        for i in range(L):
            acc[indices[indptr[r] + i // 64], :, i % 64] = weights[r][:, i]
    stride = stride or max(1, min(max(budgets), max(lens)))
    kept = torch.full((len(lens), Hkv, stride), -9, dtype=torch.int32, device="cuda")
    new = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    hpa.hpa_evict_select(dev(acc), dev(np.array(lens, np.int32)), dev(indptr), dev(indices),
                         dev(np.array(budgets, np.int32)), sinks, recent, kept, new, st)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), new.cpu().numpy(), int(st.item())


def _check_select(weights, lens, budgets, sinks, recent, **kw):
    kept, new, st = _select(weights, lens, budgets, sinks, recent, **kw)
    assert st == 0
    for r, L in enumerate(lens):
        n = min(L, budgets[r])
        assert new[r] == n
        for h in range(kept.shape[1]):
            assert list(kept[r, h, :n]) == bounded.kept_keys(weights[r][h], budgets[r], sinks,
                                                             recent), (r, h)
            assert (kept[r, h, n:] == -9).all()


@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 0), (0, 7), (3, 64), (65, 1)])
def test_select_lengths_and_budgets(sinks, recent):
    g = np.random.default_rng(sinks + recent)
    lens = [1, 2, 63, 64, 65, 130, 200, 500, 1027, 2050, 5000]
    low = sinks + recent
    budgets = [max(1, low, min(L, int(g.integers(max(1, low), max(low + 2, L + 5))))) for L in lens]
    budgets[4], budgets[6], budgets[8] = max(1, low), 199, 1 << 20     # the fewest, all but one, all
    weights = [np.exp(g.standard_normal((2, L)) * 2).astype(np.float32) for L in lens]
    _check_select(weights, lens, budgets, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "special", "close", "negative"])
def test_select_ties_and_special_weights(kind):
    g = np.random.default_rng(5)
    L = 1500
    w = {"equal": np.full((2, L), 0.25),
         "few": g.integers(0, 3, (2, L)).astype(float),
         "zeros": np.where(g.random((2, L)) < 0.5, 0.0, -0.0),
         "special": g.choice([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, 1.0, 3e38], (2, L)),
         "close": 1 + g.integers(0, 9, (2, L)) * 2.0 ** -23,
         "negative": -np.exp(g.standard_normal((2, L)))}[kind].astype(np.float32)
    for budget in (5, 6, 700, 1499):
        _check_select([w], [L], [budget], 2, 3)


@pytest.mark.parametrize("L", [48 * 1024 - 1, 48 * 1024 + 1, 100003, 250000])
def test_select_long_requests(L):
    """Lengths around and beyond what one block, or a cluster, holds in shared memory."""
    g = np.random.default_rng(L)
    w = np.exp(g.standard_normal((1, L)) * 1.5).astype(np.float32)
    w[0, ::7] = w[0, 3]
    order = np.lexsort((np.arange(L), -w[0].astype(np.float64)))
    for budget in (1, 4099, L - 1):
        kept, new, st = _select([w], [L], [budget], 0, 0, Hkv=1)
        assert st == 0 and new[0] == budget
        assert (kept[0, 0] == np.sort(order[:budget])).all()


def test_select_many_requests():
    g = np.random.default_rng(8)
    lens = list(g.integers(1, 400, size=500))
    weights = [g.random((1, L)).astype(np.float32) for L in lens]
    _check_select(weights, lens, [100] * 500, 1, 10, Hkv=1)


def test_select_one_long_among_many():
    """A length far beyond the mean that the blocks per (request, head) are chosen by."""
    g = np.random.default_rng(10)
    lens = [70] * 200 + [60001] + [70] * 100
    weights = [g.random((1, L)).astype(np.float32) for L in lens]
    kept, new, st = _select(weights, lens, [64] * 200 + [2000] + [64] * 100, 2, 30, Hkv=1)
    assert st == 0
    for r in (0, 199, 200, 300):
        n = int(new[r])
        assert list(kept[r, 0, :n]) == bounded.kept_keys(weights[r][0], n, 2, 30)


@pytest.mark.parametrize("B,Hkv", [(2, 160), (57, 8), (127, 3), (128, 3), (129, 3)])
def test_select_more_blocks_than_the_gpu_holds(B, Hkv):
    """The longest requests go first then: equal lengths, none and every other order."""
    g = np.random.default_rng(B)
    lens = [int(x) for x in g.choice([1, 64, 65, 100, 100, 190, 300], size=B)]
    weights = [g.random((Hkv, L)).astype(np.float32) for L in lens]
    _check_select(weights, lens, [70] * B, 1, 10, Hkv=Hkv)
    lens[B // 2] = 0
    kept, new, st = _select(weights, lens, [70] * B, 1, 10, Hkv=Hkv)
    assert st == 1 and list(new) == [min(L, 70) if L else -1 for L in lens]
    assert (kept[B // 2] == -9).all()


def test_select_short_requests_in_a_large_pool():
    """Blocks are launched by the pool's size; those that a request does not need leave."""
    g = np.random.default_rng(11)
    lens = [1, 100, 4096, 4097, 8192, 8193, 16385, 0, 32768, 33000]
    weights = [g.random((1, L)).astype(np.float32) for L in lens]
    budgets = [50, 50, 2000, 2000, 8192, 1, 16384, 5, 7000, 32999]
    kept, new, st = _select(weights, lens, budgets, 0, 0, Hkv=1, spare=8192)
    assert st == 1
    for r, L in enumerate(lens):
        n = min(L, budgets[r])
        assert new[r] == (n if L else -1) and (kept[r, 0, n:] == -9).all()
        order = np.lexsort((np.arange(L), -weights[r][0].astype(np.float64)))
        assert (kept[r, 0, :n] == np.sort(order[:n])).all()


def test_select_refusals():
    g = np.random.default_rng(9)
    lens = [100, 100, 100, 100, 0]
    w = [g.random((2, max(1, L))).astype(np.float32) for L in lens]
    kept, new, st = _select(w, lens, [0, 9, 60, 50, 10], 5, 5, stride=50)
    assert list(new) == [-1, -1, -1, 50, -1] and st == 64 | 1
    assert (kept[[0, 1, 2, 4]] == -9).all()
    acc = torch.zeros((4, 2, 64), device="cuda")
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for indices, n in (((0, 4), 100), ((0, -1), 100), ((0,), 100), ((0, 7), 65)):
        for budget in (40, 200):
            kept = torch.full((1, 2, 200), -9, dtype=torch.int32, device="cuda")
            new, st = one(5), one(0)
            hpa.hpa_evict_select(acc, one(n), one(0, len(indices)), one(*indices), one(budget), 0,
                                 0, kept, new, st)
            assert int(st.item()) == 4 and int(new.item()) == -1 and (kept == -9).all()
    for n in (2 ** 31 - 1, 2 ** 31 - 65536):        # positions that int32 does not hold
        new, st = one(5), one(0)
        hpa.hpa_evict_select(acc, one(n), one(0, 2), one(0, 1), one(40), 0, 0, kept, new, st)
        assert int(st.item()) == 16 and int(new.item()) == -1 and (kept == -9).all()


# ----------------------------------------------------------------------------- compaction
def _cache(lens, kv, Hkv, spare=0, seed=0):
    b = W.make_batch(lens, kv_dtype=kv, seed=seed, Hq=Hkv, Hkv=Hkv)
    db = DeviceBatch(b)
    if spare:
        db.k = torch.cat([db.k, torch.full_like(db.k[:1], 3).expand(spare, -1, -1, -1)]).contiguous()
        db.v = torch.cat([db.v, torch.full_like(db.v[:1], 4).expand(spare, -1, -1, -1)]).contiguous()
    g = torch.Generator().manual_seed(seed)
    acc = torch.rand((db.k.shape[0], Hkv, 64), generator=g).cuda()
    return b, db, acc


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,budget,Hkv", [([1], 1, 1), ([300], 100, 1), ([300, 200], 250, 1), ([64, 700, 65, 30], 64, 3),
                                             ([5000, 130, 2500], 2049, 2),
                                             (list(range(60, 260)), 90, 2),
                                             ([40000, 9000], 3001, 1),      # clusters
                                             ([30000], 20000, 1)])
@pytest.mark.parametrize("elsewhere", [False, True])
@pytest.mark.parametrize("calls", [1, 2])
def test_evict_step(kv, lens, budget, Hkv, elsewhere, calls):
    pages = [(min(L, budget) + 63) // 64 for L in lens]
    b, db, acc = _cache(lens, kv, Hkv, sum(pages) if elsewhere else 0, seed=len(lens) + budget)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    dst = {}
    d_ptr, d_idx = b.page_indptr, b.page_indices
    if elsewhere:
        d_ptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        d_idx = (b.num_pages + np.random.default_rng(1).permutation(sum(pages))).astype(np.int32)
        dst = dict(dst_indptr=dev(d_ptr), dst_indices=dev(d_idx))
    budgets = np.full(len(lens), budget, np.int32)
    k0, v0, a0 = (x.clone().cpu() for x in (db.k, db.v, acc))
    kept = torch.full((len(lens), Hkv, budget), -9, dtype=torch.int32, device="cuda")
    new = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sinks, recent = min(2, budget // 2), min(5, budget // 2)
    if calls == 1:
        hpa.evict_step(acc, db.k, db.v, db.lens, db.indptr, db.indices, dev(budgets), sinks,
                       recent, kept, new, status=st, **dst)
    else:
        hpa.hpa_evict_select(acc, db.lens, db.indptr, db.indices, dev(budgets), sinks, recent,
                             kept, new, st)
        hpa.hpa_evict_compact(db.k, db.v, db.indptr, db.indices, kept, new, acc, status=st, **dst)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ek, ev, ea = k0.clone(), v0.clone(), a0.clone()
    for r, L in enumerate(lens):
        ids = b.page_indices[b.page_indptr[r]:b.page_indptr[r + 1]]
        to = d_idx[d_ptr[r]:d_ptr[r + 1]]
        for h in range(Hkv):
            w = a0[ids, h].reshape(-1)[:L].numpy()
            want = np.array(bounded.kept_keys(list(w), budget, sinks, recent))
            assert (kept[r, h, :len(want)].cpu().numpy() == want).all()
            t = np.arange(len(want))
            src, dst_at = (ids[want // 64], h, want % 64), (to[t // 64], h, t % 64)
            for e, x in ((ek, k0), (ev, v0), (ea, a0)):
                e[dst_at] = x[src]
    raw = lambda x: x.cpu().view(torch.int16 if kv == "bf16" else torch.uint8)  # noqa: E731
    assert torch.equal(raw(db.k), raw(ek)) and torch.equal(raw(db.v), raw(ev))
    assert torch.equal(acc.cpu(), ea)


def test_compact_passes_over_what_selection_refused():
    b, db, acc = _cache([100, 200], "bf16", 2, seed=20)
    k0 = db.k.clone()
    kept = torch.zeros((2, 2, 64), dtype=torch.int32, device="cuda")
    new = torch.tensor([-1, 65], dtype=torch.int32, device="cuda")     # 65 > stride
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    hpa.hpa_evict_compact(db.k, db.v, db.indptr, db.indices, kept, new, acc, status=st)
    assert torch.equal(db.k, k0) and int(st.item()) == 0
    new[0], new[1] = 64, 1
    kept[0] = torch.arange(64, device="cuda") * 3                       # up to 189: no such page
    kept[1] = 7
    hpa.hpa_evict_compact(db.k, db.v, db.indptr, db.indices, kept, new, acc, status=st)
    assert int(st.item()) == 4


# ----------------------------------------------------------------------------- together
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(None, 0), (90, 4)])
def test_serving_loop_with_evictions(kv, window, sinks):
    """Twelve steps of two tokens: store at text positions, attend, accumulate, evict when a
    cache passes its mark.  The outputs and weights of every step are checked against the
    64-bit definition on the cache as it then is, and every cache row against the feeder's
    rotation at its text position."""
    q_len, Hkv, Hq, budget, mark = 2, 2, 16, 70, 90
    lens = np.array([80, 30, 88], np.int64)
    text = lens.copy()
    b = W.make_batch(lens + 64, q_len=q_len, kv_dtype=kv, seed=21, Hq=Hq, Hkv=Hkv)
    db = DeviceBatch(b)
    acc = torch.zeros((b.num_pages, Hkv, 64), device="cuda")
    state = [[[(int(i), -1) for i in range(lens[r])] for _ in range(Hkv)] for r in range(3)]
    cs = torch.from_numpy(W.rope_cos_sin_table(400)).cuda()
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvc = hpa.KV_BF16 if kv == "bf16" else hpa.KV_E4M3
    C = hpa.hpa_default_num_ctas(Hkv, q_len, kvc, Hq)
    evicted = False
    for step in range(12):
        lens += q_len
        fi = W.make_feeder_inputs(100 + step, 3, q_len, max_pos=400, Hkv=Hkv)
        hpa.hpa_store_kv_at(fi.k_new.cuda(), fi.v_new.cuda(), dev(lens), dev(text), db.indptr,
                            db.indices, cs, torch.from_numpy(fi.norm_w).cuda(), db.k, db.v,
                            eps=fi.eps, k_scale=db.ks, v_scale=db.vs, status=st)
        for r in range(3):
            for h in range(Hkv):
                state[r][h] += [(int(text[r]) + j, step) for j in range(q_len)]
        text += q_len
        b.seq_lens = lens.astype(np.int32)
        b.q = W.make_q(200 + step, 3, q_len, Hq)
        db.q, db.lens = b.q.cuda(), dev(lens)
        b.k_pool, b.v_pool = db.k.cpu(), db.v.cpu()
        before = acc.cpu().numpy().astype(np.float64)
        ws = hpa.Workspace(3, q_len, Hq, 128, num_ctas=C, Hkv=Hkv, window=window, sinks=sinks)
        out = torch.empty((3, q_len, Hq, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((3, q_len, Hq), dtype=torch.float32, device="cuda")
        hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks,
                        db.vs, acc=acc, decay=0.95)
        torch.cuda.synchronize()
        assert ws.status() == 0
        check_attention(b, out, lse, bounded.attention_rows(b, window, sinks), kv)
        new, written, E = bounded.key_weights(b, lse.cpu().numpy(), before, 0.95, window, sinks)
        assert_within(acc.cpu().numpy(), new, weight_bound(new, E), "acc")
        if (lens > mark).any():
            evicted = True
            budgets = np.where(lens > mark, budget, lens)
            kept = torch.zeros((3, Hkv, 200), dtype=torch.int32, device="cuda")
            n = torch.zeros(3, dtype=torch.int32, device="cuda")
            hpa.evict_step(acc, db.k, db.v, db.lens, db.indptr, db.indices, dev(budgets), 4, 20,
                           kept, n, status=st)
            lens = n.cpu().numpy().astype(np.int64)
            assert (lens <= mark).all()
            for r in range(3):
                for h in range(Hkv):
                    state[r][h] = [state[r][h][i] for i in kept[r, h, :lens[r]].tolist()]
    assert evicted and int(st.item()) == 0
    # the keys that the steps stored: rotation by text position, whatever slot they are in now
    K = bounded.pool_values(db.k, kv, b.k_scale)
    for r in range(3):
        for h in range(Hkv):
            ids = b.page_indices[b.page_indptr[r]:b.page_indptr[r + 1]]
            for slot, (pos, step) in enumerate(state[r][h]):
                if step < 0:
                    continue
                fi = W.make_feeder_inputs(100 + step, 3, q_len, max_pos=400, Hkv=Hkv)
                j = pos - (int(text[r]) - q_len * (12 - step))
                x = feeder.rope_rotate_half(fi.k_new[r, j, h].double().numpy(),
                                            fi.cos_sin[pos].astype(np.float64))
                x = feeder.hadamard(128) @ feeder.rms_norm(x, fi.norm_w.astype(np.float64), fi.eps)
                tol = 2.0 ** -8 * np.abs(x) + 3e-5
                if kv == "e4m3":   # half a step, of a normal or of the subnormals (2^-10 scales)
                    tol = 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * float(b.k_scale[h]) + 3e-5
                    x = np.clip(x, -448 * b.k_scale[h], 448 * b.k_scale[h])
                got = K[ids[slot // 64], h, slot % 64]
                assert (np.abs(got - x) <= tol).all(), (r, h, slot, pos, np.abs(got - x).max())
