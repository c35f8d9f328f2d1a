"""The bounded-cache operators as a serving loop uses them: captured and replayed, on other
streams, two at once, in pools whose offsets pass 32 bits, between guard bands, and the KV
writer at text positions."""
import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from bounded_helpers import check_attention
from gpu_helpers import DeviceBatch
from oracle import bounded

pytestmark = pytest.mark.gpu


def _dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype)).cuda()


# ----------------------------------------------------------------------------- graphs and streams
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_captured_step_with_weights_and_eviction_replays_on_new_inputs(kv):
    """decode_step with accumulation, then evict_step, in one graph; replayed after queries,
    lengths, budgets and weights change in place, against the same calls made eagerly."""
    b = W.make_batch([500, 260, 129], q_len=2, kv_dtype=kv, seed=31, Hq=16, Hkv=2)
    kvc = hpa.KV_BF16 if kv == "bf16" else hpa.KV_E4M3
    C = hpa.hpa_default_num_ctas_window(2, 2, kvc, 16)

    def state():
        db = DeviceBatch(b)
        s = dict(db=db, ws=hpa.Workspace(3, 2, 16, 128, num_ctas=C, Hkv=2, window=200, sinks=3),
                 out=torch.zeros((3, 2, 16, 128), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros((3, 2, 16), device="cuda"),
                 acc=torch.zeros((b.num_pages, 2, 64), device="cuda"),
                 budgets=_dev([400, 128, 129]), new=_dev([0, 0, 0]), st=_dev([0]),
                 kept=torch.zeros((3, 2, 500), dtype=torch.int32, device="cuda"))
        return s

    def step(s):
        db = s["db"]
        hpa.decode_step(s["ws"], db.q, db.k, db.v, db.lens, db.indptr, db.indices, s["out"],
                        s["lse"], db.ks, db.vs, acc=s["acc"], decay=0.9)
        hpa.evict_step(s["acc"], db.k, db.v, db.lens, db.indptr, db.indices, s["budgets"], 3, 60,
                       s["kept"], s["new"], status=s["st"])

    eager, graphed = state(), state()
    stream = torch.cuda.Stream()
    warm = state()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step(warm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step(graphed)
    torch.cuda.synchronize()
    for i, (lens, budgets) in enumerate((([500, 260, 129], [400, 128, 129]),
                                         ([400, 128, 2], [64, 70, 200]),
                                         ([333, 65, 100], [333, 64, 99]))):
        q = W.make_q(40 + i, 3, 2, 16).cuda()
        for s in (eager, graphed):
            s["db"].q.copy_(q)
            s["db"].lens.copy_(_dev(lens))
            s["budgets"].copy_(_dev(budgets))
            s["acc"] += 0.25 * (i + 1)
        torch.cuda.synchronize()
        step(eager)
        g.replay()
        torch.cuda.synchronize()
        assert int(graphed["st"].item()) == int(eager["st"].item()) == 0
        assert graphed["new"].tolist() == [min(a, c) for a, c in zip(lens, budgets)]
        for name in ("out", "lse", "acc", "kept", "new"):
            assert torch.equal(eager[name], graphed[name]), (i, name)
        assert torch.equal(eager["db"].k.view(torch.uint8), graphed["db"].k.view(torch.uint8))
        assert torch.equal(eager["db"].v.view(torch.uint8), graphed["db"].v.view(torch.uint8))


def test_two_streams_at_once():
    """Independent steps on two streams, interleaved: each equals the step made alone."""
    results, jobs = [], []
    for i, (kv, rows) in enumerate((("e4m3", (64, 8, 1)), ("bf16", (16, 2, 8)))):
        hq, hkv, q_len = rows
        b = W.make_batch([3000, 900, 70, 2000], q_len=q_len, kv_dtype=kv, seed=50 + i, Hq=hq,
                         Hkv=hkv)
        db = DeviceBatch(b)
        kvc = hpa.KV_BF16 if kv == "bf16" else hpa.KV_E4M3
        C = hpa.hpa_default_num_ctas(hkv, q_len, kvc, hq)

        def once(stream, db=db, b=b, C=C):
            ws = hpa.Workspace(4, b.q_len, b.Hq, 128, num_ctas=C, Hkv=b.Hkv)
            out = torch.zeros((4, b.q_len, b.Hq, 128), dtype=torch.bfloat16, device="cuda")
            lse = torch.zeros((4, b.q_len, b.Hq), device="cuda")
            acc = torch.ones((b.num_pages, b.Hkv, 64), device="cuda")
            kept = torch.zeros((4, b.Hkv, 1000), dtype=torch.int32, device="cuda")
            new, bud = _dev([0] * 4), _dev([1000, 500, 100, 900])
            torch.cuda.synchronize()

            def go():
                for _ in range(4):
                    hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse,
                                    db.ks, db.vs, acc=acc, stream=stream)
                    hpa.hpa_evict_select(acc, db.lens, db.indptr, db.indices, bud, 2, 20, kept,
                                         new, stream=stream)
            return go, (out, lse, acc, kept, new)
        alone, want = once(torch.cuda.current_stream())
        alone()
        alone()
        torch.cuda.synchronize()
        jobs.append(once(torch.cuda.Stream()))
        results.append(want)
    for go, _ in jobs * 2:
        go()
    torch.cuda.synchronize()
    for (go, got), want in zip(jobs, results):
        for name, x, y in zip(("out", "lse", "acc", "kept", "new"), got, want):
            assert torch.equal(x, y), name


# ----------------------------------------------------------------------------- far offsets
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_past_32_bit_offsets(kv):
    """A pool of 3 * 2^30 elements (6 GB bf16): the request's pages lie beyond element 2^31,
    the copy's too.  Window attention, weights and eviction against the same request in a
    small pool."""
    hkv, L, q_len = 8, 300, 2
    P = 3 * (1 << 30) // (hkv * 64 * 128)
    b = W.make_batch([L], q_len=q_len, kv_dtype=kv, seed=61, Hq=16, Hkv=hkv)
    db = DeviceBatch(b)
    n = len(b.page_indices)
    far = P - 1 - np.arange(n) * 7
    to = P - 2 - np.arange(3) * 7
    big = {}
    for name, pool in (("k", db.k), ("v", db.v)):
        big[name] = torch.zeros((P, hkv, 64, 128), dtype=pool.dtype, device="cuda")
        big[name][torch.from_numpy(far).cuda()] = pool[db.indices.long()]
    acc = torch.zeros((P, hkv, 64), device="cuda")
    small_acc = torch.rand((b.num_pages, hkv, 64), device="cuda")
    acc[torch.from_numpy(far).cuda()] = small_acc[db.indices.long()]
    idx, dst = _dev(far), _dev(to)
    outs = []
    for k, v, ix, a in ((db.k, db.v, db.indices, small_acc), (big["k"], big["v"], idx, acc)):
        ws = hpa.Workspace(1, q_len, 16, 128, num_ctas=7, Hkv=hkv, window=100, sinks=5)
        out = torch.zeros((1, q_len, 16, 128), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros((1, q_len, 16), device="cuda")
        hpa.decode_step(ws, db.q, k, v, db.lens, db.indptr, ix, out, lse, db.ks, db.vs, acc=a)
        outs.append((out, lse, a[ix.long()].clone()))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    kept = torch.zeros((1, hkv, 150), dtype=torch.int32, device="cuda")
    new, st = _dev([0]), _dev([0])
    hpa.evict_step(acc, big["k"], big["v"], db.lens, db.indptr, idx, _dev([150]), 5, 20, kept, new,
                   dst_indptr=_dev([0, 3]), dst_indices=dst, status=st)
    assert int(st.item()) == 0 and int(new.item()) == 150
    for h in range(hkv):
        w = small_acc[db.indices.long(), h].reshape(-1)[:L].cpu().numpy()
        want = np.array(bounded.kept_keys(list(w), 150, 5, 20))
        assert (kept[0, h].cpu().numpy() == want).all()
        t = np.arange(150)
        for name, pool in (("k", db.k), ("v", db.v)):
            got = big[name][torch.from_numpy(to[t // 64]).cuda(), h, torch.from_numpy(t % 64).cuda()]
            src = pool[db.indices.long()[torch.from_numpy(want // 64).cuda()], h,
                       torch.from_numpy(want % 64).cuda()]
            assert torch.equal(got.view(torch.uint8), src.view(torch.uint8))


# ----------------------------------------------------------------------------- guard bands
def _guarded(shape, dtype, fill):
    n = int(np.prod(shape))
    raw = torch.full((n + 2048,), fill, dtype=dtype, device="cuda")
    return raw, raw[1024:1024 + n].view(shape)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_guard_bands_untouched(kv):
    b = W.make_batch([700, 64, 1, 333], q_len=1, kv_dtype=kv, seed=71, Hq=16, Hkv=2)
    db = DeviceBatch(b)
    bands = []

    def guard(shape, dtype, fill=7):
        raw, t = _guarded(shape, dtype, fill)
        bands.append((raw, t.numel(), raw.clone()))
        return t

    k, v = guard(db.k.shape, db.k.dtype), guard(db.v.shape, db.v.dtype)
    k.copy_(db.k), v.copy_(db.v)
    acc = guard((b.num_pages, 2, 64), torch.float32)
    acc.uniform_()
    kept, new, st = guard((4, 2, 200), torch.int32), guard((4,), torch.int32), guard((1,),
                                                                                     torch.int32)
    st.zero_()
    ws = hpa.Workspace(4, 1, 16, 128, num_ctas=11, Hkv=2, window=300, sinks=70)
    ws.taskmap = guard(ws.taskmap.shape, torch.int32)
    ws.partial_o = guard(ws.partial_o.shape, torch.float32)
    ws.partial_lse = guard(ws.partial_lse.shape, torch.float32)
    out, lse = guard((4, 1, 16, 128), torch.bfloat16), guard((4, 1, 16), torch.float32)
    hpa.decode_step(ws, db.q, k, v, db.lens, db.indptr, db.indices, out, lse, db.ks, db.vs, acc=acc)
    check_attention(b, out, lse, bounded.attention_rows(b, 300, 70), kv)
    hpa.evict_step(acc, k, v, db.lens, db.indptr, db.indices, _dev([200, 60, 1, 200]), 3, 20, kept,
                   new, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and new.tolist() == [200, 60, 1, 200]
    for raw, n, before in bands:
        x, y = raw.view(torch.uint8), before.view(torch.uint8)
        e = raw.element_size()
        assert torch.equal(x[:1024 * e], y[:1024 * e])
        assert torch.equal(x[(1024 + n) * e:], y[(1024 + n) * e:])


@pytest.mark.parametrize("how", ["request", "tiles", "owner", "partition", "window", "sinks",
                                 "length"])
def test_corrupted_window_maps_are_reported(how):
    """A map altered after the plan: the status says so, the step's outputs of the damaged
    request are NaN, and no accumulator outside the buffers' extents or of another request
    changes because of it."""
    b = W.make_batch([700, 300], q_len=1, seed=72, Hq=16, Hkv=2)
    db = DeviceBatch(b)
    ws = hpa.Workspace(2, 1, 16, 128, num_ctas=6, Hkv=2, window=256, sinks=4)
    ws.plan(db.lens)
    B, C = 2, 6
    tm = ws.taskmap.cpu()
    segs = ((16 + B + 2 * (B + 1) + 2 * (C + 1)) + 3) & ~3
    cta_seg = 16 + B + (B + 1) + (C + 1)
    if how == "request":
        tm[segs] = 5
    elif how == "tiles":
        tm[segs + 2] = 10000
    elif how == "owner":
        tm[segs + 3] = 3
    elif how == "partition":
        tm[cta_seg + 1] = 1000
    elif how == "window":
        tm[11] = 0
    elif how == "sinks":
        tm[12] = -1
    elif how == "length":
        tm[16] = 0
    ws.taskmap.copy_(tm)
    bands = []
    acc_raw, acc = _guarded((b.num_pages, 2, 64), torch.float32, 7)
    acc.fill_(3.0)
    bands.append(acc_raw.clone())
    lse = torch.full((2, 1, 16), 5.0, device="cuda")
    hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, db.indices, ws.taskmap, 6, acc)
    torch.cuda.synchronize()
    assert ws.status() & (32 | 1)
    assert torch.equal(acc_raw[:1024], bands[0][:1024])
    assert torch.equal(acc_raw[-1024:], bands[0][-1024:])
    tm[6] = 0
    ws.taskmap.copy_(tm)
    out = torch.zeros((2, 1, 16, 128), dtype=torch.bfloat16, device="cuda")
    hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, plan=False)
    torch.cuda.synchronize()
    assert ws.status() & (32 | 1)
    assert out[0].isnan().all()


# ----------------------------------------------------------------------------- writer
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_store_at_text_positions(kv):
    lens, q_len = [3, 64, 130, 700], 3
    b = W.make_batch(lens, q_len=q_len, kv_dtype=kv, seed=81, Hq=8, Hkv=1)
    fi = W.make_feeder_inputs(81, 4, q_len, max_pos=1000, Hkv=1)
    cs, w = torch.from_numpy(fi.cos_sin).cuda(), torch.from_numpy(fi.norm_w).cuda()
    kn, vn = fi.k_new.cuda(), fi.v_new.cuda()

    def store(fn, *pos, status=None):
        db = DeviceBatch(b)
        fn(kn, vn, db.lens, *pos, db.indptr, db.indices, cs, w, db.k, db.v, k_scale=db.ks,
           v_scale=db.vs, status=status)
        return db.k.view(torch.uint8), db.v.view(torch.uint8)

    plain = store(hpa.hpa_store_kv)
    same = store(hpa.hpa_store_kv_at, _dev(np.array(lens) - q_len))
    assert torch.equal(plain[0], same[0]) and torch.equal(plain[1], same[1])
    # cache position 0.. with text position 900..: the row a fresh cache of that length has
    moved = store(hpa.hpa_store_kv_at, _dev([997, 500, 0, 699]))
    long = W.make_batch([1000, 503, 3, 702], q_len=q_len, kv_dtype=kv, seed=81, Hq=8, Hkv=1)
    ldb = DeviceBatch(long)
    if kv == "e4m3":
        long.k_scale = b.k_scale
        ldb.ks, ldb.vs = _dev(b.k_scale, np.float32), _dev(b.v_scale, np.float32)
    hpa.hpa_store_kv(kn, vn, ldb.lens, ldb.indptr, ldb.indices, cs, w, ldb.k, ldb.v,
                     k_scale=ldb.ks, v_scale=ldb.vs)
    lk = ldb.k.view(torch.uint8)
    for r in range(4):
        for j in range(q_len):
            at, far = lens[r] - q_len + j, int(long.seq_lens[r]) - q_len + j
            page = b.page_indices[b.page_indptr[r] + at // 64]
            there = long.page_indices[long.page_indptr[r] + far // 64]
            assert torch.equal(moved[0][page, 0, at % 64], lk[there, 0, far % 64]), (r, j)
    # text positions outside the table: reported, nothing written
    for bad in ([998, 500, 0, 699], [-1, 500, 0, 699], [2**31 - 1, 500, 0, 699]):
        st = _dev([0])
        k, _ = store(hpa.hpa_store_kv_at, _dev(bad), status=st)
        assert int(st.item()) == 1
        page = b.page_indices[b.page_indptr[0]]
        untouched = DeviceBatch(b).k.view(torch.uint8)[page, 0]
        first_bad = 2 if bad[0] == 998 else 0
        assert torch.equal(k[page, 0, first_bad], untouched[first_bad])


def test_binding_refusals():
    b = W.make_batch([100, 50], seed=91, Hq=16, Hkv=2)
    db = DeviceBatch(b)
    acc = torch.zeros((b.num_pages, 2, 64), device="cuda")
    lse = torch.zeros((2, 1, 16), device="cuda")
    ws = hpa.Workspace(2, 1, 16, 128, num_ctas=3, Hkv=2)
    ws.plan(db.lens)

    def weights(**kw):
        a = dict(q=db.q, lse=lse, k_pool=db.k, page_indptr=db.indptr, page_indices=db.indices,
                 taskmap=ws.taskmap, num_ctas=3, acc=acc)
        a.update(kw)
        hpa.hpa_key_weights(**a)

    weights()
    for kw, text in ((dict(lse=lse[:, :, :8].contiguous()), "lse"), (dict(acc=acc[1:]), "acc"),
                     (dict(acc=None), "out"), (dict(out=acc.half()), "out"),
                     (dict(q=db.q.transpose(2, 3)), "contiguous"), (dict(q=db.q.float()), "q"),
                     (dict(page_indptr=db.indptr[:2]), "page_indptr"),
                     (dict(taskmap=ws.taskmap[:40]), "taskmap"), (dict(decay=-1.0), "invalid"),
                     (dict(k_pool=db.k.view(torch.uint8)[..., :128].contiguous()), "k_scale")):
        with pytest.raises(hpa.HpaError, match=text):
            weights(**kw)
    kept = torch.zeros((2, 2, 60), dtype=torch.int32, device="cuda")
    new, bud = _dev([0, 0]), _dev([60, 60])

    def evict(**kw):
        a = dict(acc=acc, k_pool=db.k, v_pool=db.v, seq_lens=db.lens, page_indptr=db.indptr,
                 page_indices=db.indices, budgets=bud, sinks=1, recent=2, kept=kept, new_lens=new)
        a.update(kw)
        hpa.evict_step(**a)

    for kw, text in ((dict(budgets=bud[:1]), "budgets"), (dict(kept=kept[:, :1]), "kept"),
                     (dict(kept=kept[:1]), "kept"), (dict(new_lens=new[:1]), "new_lens"),
                     (dict(new_lens=db.lens), "invalid"), (dict(sinks=-1), "invalid"),
                     (dict(v_pool=db.k), "invalid"), (dict(dst_indptr=db.indptr), "together"),
                     (dict(acc=acc.double()), "float32"), (dict(v_pool=db.v[:, :1]), "contiguous"),
                     (dict(page_indptr=db.indptr[:1]), "page_indptr")):
        with pytest.raises(hpa.HpaError, match=text):
            evict(**kw)
    torch.cuda.synchronize()
    assert new.tolist() == [0, 0] and not kept.any()
