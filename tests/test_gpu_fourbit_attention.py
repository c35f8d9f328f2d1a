"""Attention over 4-bit pages (hpa_decode_attn and hpa_decode_attn_window with HPA_KV_E2M1)
against the 64-bit definition; slots that no token sees hold NaN scales throughout."""
import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
from bounded_helpers import check_attention, lse_bound, out_bound
from fourbit_helpers import make_batch, poison_hidden, rows_of, step
from gpu_helpers import DeviceBatch
from oracle import bounded, fourbit

pytestmark = pytest.mark.gpu


def _run(lens, q_len, window=None, sinks=0, heads=(16, 2), C=None, tile=None, seed=0):
    b = make_batch(lens, q_len, heads, seed)
    poison_hidden(b, window, sinks)
    db = DeviceBatch(b)
    ws, out, lse = step(b, db, window, sinks, C, tile)
    torch.cuda.synchronize()
    assert ws.status() == 0
    check_attention(b, out, lse, bounded.attention_rows(b, window, sinks), "e2m1")


@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (63, 4), (65, 64), (128, 65), (200, 3),
                                          (1 << 30, 1 << 30)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_lengths_around_every_border(window, sinks, q_len):
    lens = [q_len, 16, 63, 64, 65, 127, 130, 191, 200, 257, 449, 700, 1111]
    _run(lens, q_len, window, sinks, seed=3 + q_len)


@pytest.mark.parametrize("heads,q_len", [((2, 2), 1), ((8, 1), 1), ((8, 1), 2), ((8, 1), 8),
                                         ((5, 1), 1), ((9, 1), 1), ((40, 8), 4), ((32, 2), 1),
                                         ((48, 4), 2), ((12, 3), 5), ((64, 8), 5), ((17, 1), 3)])
@pytest.mark.parametrize("window", [None, 130])
def test_head_layouts(heads, q_len, window):
    _run([q_len, 90, 400, 777], q_len, window, 7 if window else 0, heads, seed=heads[0])


@pytest.mark.parametrize("C,tile", [(1, 64), (3, 128), (23, 64), (40, 512), (200, 64)])
def test_partitions_and_tiles(C, tile):
    _run([1, 500, 1300, 40, 640], 1, C=C, tile=tile, seed=C)


@pytest.mark.parametrize("window,sinks", [(None, 0), (70, 3)])
@pytest.mark.parametrize("C,q_len", [(1, 1), (1, 3), (2, 5), (3, 2)])
def test_partitions_of_many_requests(C, q_len, window, sinks):
    """More segments in a partition than are read at once (32), some of them two pages short of a
    ring's length, some with many pages."""
    g = np.random.default_rng(50 + C)
    lens = [int(n) for n in g.integers(q_len, 200, size=75)] + [2500, q_len, 64, 65, 2100, 70]
    _run(lens, q_len, window, sinks, heads=(8, 1), C=C, tile=64, seed=51)


def test_one_long_request_and_a_large_batch():
    _run([70000], 2, heads=(8, 1), seed=3)
    g = np.random.default_rng(4)
    _run(list(g.integers(1, 300, size=400)), 1, heads=(4, 1), seed=4)


@pytest.mark.parametrize("window,sinks", [(None, 0), (70, 0), (5, 130)])
@pytest.mark.parametrize("heads,q_len", [((8, 2), 3), ((8, 1), 2), ((40, 8), 4)])
def test_nan_scales_reach_only_the_rows_that_see_them(window, sinks, heads, q_len):
    """A NaN block scale of a value marks its 16 dims of the rows that see the key, one of a key
    the whole row; all other rows are as without it."""
    lens = [200, 131, 64 + q_len]
    for which in ("v", "k"):
        b = make_batch(lens, q_len, heads, seed=21)
        poison_hidden(b, window, sinks)
        bad = []
        for r, L in enumerate(lens):
            # the last key (one token sees it), the first token's, and one at the windows' start
            for i in {L - 1, L - q_len, max(0, L - (window or 0) - 1), max(0, L - (window or 0))}:
                h, block = i % b.Hkv, (5 * i + r) % 8
                page = int(b.page_indices[int(b.page_indptr[r]) + i // 64])
                bad.append((r, i, h, block, page))
        ref = bounded.attention_rows(b, window, sinks)
        for r, i, h, block, page in bad:
            rows_of(b.k_pool if which == "k" else b.v_pool)[1][page, h, i % 64, block] = 0x7F
        ws, out, lse = step(b, DeviceBatch(b), window, sinks)
        torch.cuda.synchronize()
        assert ws.status() == 0
        want, seen = ref[0].copy(), np.zeros(ref[1].shape, bool)
        G = b.Hq // b.Hkv
        for r, i, h, block, page in bad:
            for j in range(q_len):
                if bounded.sees(lens[r], q_len, j, i, window, sinks):
                    dims = slice(16 * block, 16 * block + 16) if which == "v" else slice(None)
                    want[r, j, h * G:(h + 1) * G, dims] = np.nan
                    seen[r, j, h * G:(h + 1) * G] = which == "k"
        got, l = out.float().cpu().numpy(), lse.cpu().numpy()
        assert (np.isnan(got) == np.isnan(want)).all()
        fine = ~np.isnan(want)
        bound = out_bound(ref[0], ref[2], ref[3], "e2m1")
        assert (np.abs(got - want)[fine] <= bound[fine]).all()
        assert (np.abs(l - ref[1])[~seen] <= lse_bound(ref[1], ref[3])[~seen]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_row_stays_alone(bad):
    b = make_batch([300, 70], 2, (16, 2), seed=22)
    ref = bounded.attention_rows(b)
    b.q[0, 1, 3, 77] = bad
    b.q[1, 0, 12, 0] = bad
    ws, out, lse = step(b, DeviceBatch(b))
    got = out.float().cpu().numpy()
    hit = np.zeros(got.shape[:3], bool)
    hit[0, 1, 3] = hit[1, 0, 12] = True
    assert np.isnan(got[hit]).all()
    bound = out_bound(ref[0], ref[2], ref[3], "e2m1")
    assert (np.abs(got - ref[0])[~hit] <= bound[~hit]).all()


@pytest.mark.parametrize("case", ["large", "tiny", "mixed_rows", "negative", "zero"])
def test_query_scales(case):
    b = make_batch([500, 64, 130], 2, (16, 2), seed=23)
    sm, q = 1 / np.sqrt(128), b.q.float()
    if case == "large":
        q, sm = q * 1e5, sm / 1e5
    elif case == "tiny":
        q, sm = q * 1e-6, sm * 1e6
    elif case == "mixed_rows":
        q[:, :, ::3] *= 1e5
        q[:, :, 1::3] *= 1e-6
    else:
        sm = -sm if case == "negative" else 0.0
    b.q = q.to(torch.bfloat16)
    ws, out, lse = step(b, DeviceBatch(b), sm_scale=sm)
    torch.cuda.synchronize()
    check_attention(b, out, lse, bounded.attention_rows(b, sm_scale=sm), "e2m1")


@pytest.mark.parametrize("q_len", [1, 2, 3])
def test_many_small_probabilities_beside_a_large_one(q_len):
    """20000 keys of 2^-26 of the first one's weight, whose value is zero: what is left is their
    sum.  2^-26 is 2^-19 as it is held, where f16's half step is 2^-25, 2^-6 of it; the queries and
    the result add 2^-8 at most."""
    L = 20000
    b = make_batch([L], q_len, (8, 1), seed=24)
    k, v = np.zeros((b.num_pages, 1, 64, 128)), np.full((b.num_pages, 1, 64, 128), 6.0)
    first = int(b.page_indices[0])
    k[first, 0, 0], v[first, 0, 0] = 6.0, 0.0
    b.k_pool, b.v_pool = torch.from_numpy(fourbit.pack(k)), torch.from_numpy(fourbit.pack(v))
    b.q = torch.ones_like(b.q)
    b.k_scale[:], b.v_scale[:] = 1.0, 1.0
    sm = 26 * np.log(2) / (128 * 6)
    ws, out, lse = step(b, DeviceBatch(b), C=1, tile=64, sm_scale=sm)
    torch.cuda.synchronize()
    assert ws.status() == 0
    small = (L - q_len + np.arange(q_len)) * 2.0 ** -26
    want = (6 * small / (1 + small))[None, :, None, None]
    got = out.double().cpu().numpy()
    assert (np.abs(got / want - 1) <= 2.0 ** -5).all()
    check = 26 * np.log(2) + np.log1p(small)
    assert np.abs(lse.double().cpu().numpy() - check[None, :, None]).max() <= 1e-4


@pytest.mark.parametrize("heads,q_len", [((8, 1), 4), ((25, 1), 1), ((17, 1), 1), ((8, 1), 8),
                                         ((50, 2), 2), ((33, 1), 1), ((32, 1), 1)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (100, 20), (1, 0)])
def test_more_than_16_rows(heads, q_len, window, sinks):
    """Every count of pages around a tile's two and the teams' six, in partitions of one to many
    segments."""
    lens = [q_len, 63, 64, 65, 127, 128, 129, 200, 330, 385, 450, 700, 1100, 1500]
    _run(lens, q_len, window, sinks, heads, C=3, tile=128, seed=60)
    _run([q_len, 2000, 130, 900], q_len, window, sinks, heads, seed=61)


@pytest.mark.parametrize("case", ["large", "tiny", "mixed_rows", "negative", "zero"])
def test_query_scales_of_many_rows(case):
    b = make_batch([500, 64, 130], 4, (16, 2), seed=62)
    sm, q = 1 / np.sqrt(128), b.q.float()
    if case == "large":
        q, sm = q * 1e5, sm / 1e5
    elif case == "tiny":
        q, sm = q * 1e-6, sm * 1e6
    elif case == "mixed_rows":
        q[:, :, ::3] *= 1e5
        q[:, :, 1::3] *= 1e-6
    else:
        sm = -sm if case == "negative" else 0.0
    b.q = q.to(torch.bfloat16)
    ws, out, lse = step(b, DeviceBatch(b), sm_scale=sm)
    torch.cuda.synchronize()
    check_attention(b, out, lse, bounded.attention_rows(b, sm_scale=sm), "e2m1")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_query_row_stays_alone_among_many(bad):
    b = make_batch([300, 70], 4, (16, 2), seed=63)
    ref = bounded.attention_rows(b)
    b.q[0, 1, 3, 77] = bad
    b.q[1, 0, 12, 0] = bad
    ws, out, lse = step(b, DeviceBatch(b))
    got = out.float().cpu().numpy()
    hit = np.zeros(got.shape[:3], bool)
    hit[0, 1, 3] = hit[1, 0, 12] = True
    assert np.isnan(got[hit]).all()
    bound = out_bound(ref[0], ref[2], ref[3], "e2m1")
    assert (np.abs(got - ref[0])[~hit] <= bound[~hit]).all()


def test_rising_scores_of_many_rows():
    """The maximum moves with nearly every tile, each row's at its own keys."""
    b = make_batch([3000, 1300], 3, (16, 2), seed=64)
    _, scales = rows_of(b.k_pool)
    for r, L in enumerate([3000, 1300]):
        ids = b.page_indices[int(b.page_indptr[r]):int(b.page_indptr[r + 1])]
        for n, page in enumerate(ids):   # scales of a page, 2^(n / 4) times as large in all
            scales[page] = (scales[page].to(torch.int32) // 4 + 2 * min(n, 40)).to(torch.uint8)
    ws, out, lse = step(b, DeviceBatch(b))
    torch.cuda.synchronize()
    assert ws.status() == 0
    check_attention(b, out, lse, bounded.attention_rows(b), "e2m1")


@pytest.mark.parametrize("q_len", [3, 4])
def test_many_rows_captured_twice_and_on_two_streams(q_len):
    b = make_batch([900, 64, 2000, 130], q_len, (16, 2), seed=65)
    poison_hidden(b)
    db = DeviceBatch(b)
    want = step(b, db)
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for s in streams:
        got.append(step(b, db, stream=s))
    torch.cuda.synchronize()
    for ws, out, lse in got:
        assert ws.status() == 0
        assert torch.equal(out, want[1]) and torch.equal(lse, want[2])
    ws, out, lse = want
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks,
                            db.vs)
    first = out.clone()
    out.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert ws.status() == 0 and torch.equal(out, first)


def test_queries_and_scales_near_the_smallest():
    """Scores of nothing at all: hidden keys stay hidden, the rest is a mean."""
    b = make_batch([130, 70], 2, (16, 2), seed=25)
    poison_hidden(b)
    b.q = (b.q.float() * 1e-36).to(torch.bfloat16)
    b.k_scale[:] = 1e-10
    ws, out, lse = step(b, DeviceBatch(b))
    torch.cuda.synchronize()
    assert ws.status() == 0
    check_attention(b, out, lse, bounded.attention_rows(b), "e2m1")


@pytest.mark.parametrize("kind", ["static", "weighted"])
def test_other_plans(kind):
    b = make_batch([900, 33, 1500, 64], 1, (16, 2), seed=24)
    db = DeviceBatch(b)
    more = dict(splits=3) if kind == "static" else dict(num_ctas=7, weighted=True)
    ws = hpa.Workspace(b.B, 1, b.Hq, 128, Hkv=b.Hkv, **more)
    out = torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(b.q.shape[:3], device="cuda")
    hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks, db.vs,
                    tile=128)
    check_attention(b, out, lse, bounded.attention_rows(b), "e2m1")


def test_same_bits_again_and_without_allocation():
    b = make_batch([3000, 200, 64, 1000], 2, (16, 2), seed=25)
    db = DeviceBatch(b)
    ws, out, lse = step(b, db)
    first = out.clone(), lse.clone()
    for _ in range(3):
        hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks, db.vs)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    out.zero_()
    hpa.hpa_decode_attn_combine_noalloc(db.q, db.k, db.v, db.indptr, db.indices, ws.taskmap,
                                        ws.num_ctas, out, lse, db.ks, db.vs)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_captured_and_on_two_streams():
    b, b2 = make_batch([700, 90], 1, (16, 2), seed=26), make_batch([400, 1300], 3, (16, 2), seed=27)
    db, db2 = DeviceBatch(b), DeviceBatch(b2)
    refs = bounded.attention_rows(b), bounded.attention_rows(b2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        r1, r2 = step(b, db, stream=s1), step(b2, db2, stream=s2)
    torch.cuda.synchronize()
    check_attention(b, r1[1], r1[2], refs[0], "e2m1")
    check_attention(b2, r2[1], r2[2], refs[1], "e2m1")
    ws, out, lse = r1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks, db.vs)
    out.zero_(), lse.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check_attention(b, out, lse, refs[0], "e2m1")


def test_pages_past_32_bit_offsets():
    """A pool of 4.8 GB whose last pages and those past 2^31 and 2^32 bytes are read."""
    b = make_batch([400, 300], 1, (8, 8), seed=28)
    P, unit = 130000, 8 * 4608
    far = [P - 1, (1 << 31) // unit, (1 << 31) // unit + 1, (1 << 32) // unit, (1 << 32) // unit + 1, 0]
    far += [P - 2 - i for i in range(len(b.page_indices) - len(far))]
    ref = bounded.attention_rows(b)
    db = DeviceBatch(b)
    big = []
    for pool in (db.k, db.v):
        t = torch.full((P, 8, 4608), 0x7F, dtype=torch.uint8, device="cuda")
        for old, new in zip(b.page_indices.tolist(), far):
            t[new] = pool[old]
        big.append(t)
    db.k, db.v = big
    db.indices = torch.tensor(far, dtype=torch.int32, device="cuda")
    ws, out, lse = step(b, db)
    check_attention(b, out, lse, ref, "e2m1")


def test_errors_are_reported_and_the_result_is_nan():
    def run(b, C=9, **kw):
        db = DeviceBatch(b)
        for k, v in kw.items():
            setattr(db, k, v)
        ws, out, lse = step(b, db, C=C)
        torch.cuda.synchronize()
        return ws.status(), out

    b = make_batch([300, 70], 1, (16, 2), seed=29)
    ix = torch.from_numpy(b.page_indices).cuda()
    for at, bad in ((1, b.num_pages), (2, -1), (4, 2 ** 31 - 1)):
        x = ix.clone()
        x[at] = bad
        status, out = run(b, indices=x)
        assert status == 4 and torch.isnan(out).all()
    short = torch.from_numpy(b.page_indptr).cuda()
    short[1] -= 1                                  # a page list too short for its request
    status, out = run(b, indptr=short)
    assert status & 4 and torch.isnan(out).all()
    b.seq_lens[1] = 2
    b3 = make_batch([300, 70], 3, (16, 2), seed=29)
    b3.seq_lens[1] = 2                             # fewer keys than new tokens
    status, out = run(b3)
    assert status == 1 and torch.isnan(out).all()


def test_maps_of_other_calls_are_refused():
    b = make_batch([300, 70], 2, (16, 2), seed=30)
    db = DeviceBatch(b)
    win, out, lse = step(b, db, 50, 3, C=6)
    plain, _, _ = step(b, db, C=6)
    torch.cuda.synchronize()
    args = (db.q, db.k, db.v, db.indptr, db.indices)
    for ws, kw, bit in ((win, {}, 32), (plain, dict(window=True), 32)):
        ws.plan(db.lens)
        hpa.hpa_decode_attn(*args, ws.taskmap, 6, ws.partial_o, ws.partial_lse, db.ks, db.vs, **kw)
        assert ws.status() == bit
    ws = plain
    ws.plan(db.lens)
    ws.taskmap[3] = 5                              # planned for another count
    hpa.hpa_decode_attn(*args, ws.taskmap, 6, ws.partial_o, ws.partial_lse, db.ks, db.vs)
    assert ws.status() == 2


def test_guard_bands():
    """Nothing is written outside the partials and the results."""
    b = make_batch([800, 90, 64, 1], 3, (40, 8), seed=31)
    db = DeviceBatch(b)
    C = 11
    ws = hpa.Workspace(b.B, b.q_len, b.Hq, 128, num_ctas=C, Hkv=b.Hkv)
    n = ws.partial_lse.numel()
    po = torch.full((n * 128 + 512,), 3.25, device="cuda")
    pl = torch.full((n + 512,), 3.25, device="cuda")
    ws.plan(db.lens)
    hpa.hpa_decode_attn(db.q, db.k, db.v, db.indptr, db.indices, ws.taskmap, C, po[256:-256],
                        pl[256:-256], db.ks, db.vs)
    torch.cuda.synchronize()
    S = int(ws.taskmap[5])
    assert (po[:256] == 3.25).all() and (po[-256:] == 3.25).all()
    assert (pl[:256] == 3.25).all() and (pl[-256:] == 3.25).all()
    rows = b.q_len * b.Hq
    assert (po[256 + S * rows * 128:] == 3.25).all() and (pl[256 + S * rows:] == 3.25).all()
    assert not (pl[256:256 + S * rows] == 3.25).any()


def test_errors_and_guard_bands_of_many_rows():
    b = make_batch([800, 90, 300, 4], 4, (16, 2), seed=33)
    ix = torch.from_numpy(b.page_indices).cuda()
    for at, bad in ((1, b.num_pages), (2, -1), (14, 2 ** 31 - 1)):
        db = DeviceBatch(b)
        db.indices = ix.clone()
        db.indices[at] = bad
        ws, out, lse = step(b, db, C=5)
        torch.cuda.synchronize()
        assert ws.status() == 4 and torch.isnan(out).all()
    short = make_batch([300, 70], 4, (16, 2), seed=33)
    short.seq_lens[1] = 3                          # fewer keys than new tokens
    ws, out, lse = step(short, DeviceBatch(short), C=5)
    torch.cuda.synchronize()
    assert ws.status() == 1 and torch.isnan(out).all()
    db, C = DeviceBatch(b), 11
    ws = hpa.Workspace(b.B, b.q_len, b.Hq, 128, num_ctas=C, Hkv=b.Hkv)
    n = ws.partial_lse.numel()
    po = torch.full((n * 128 + 512,), 3.25, device="cuda")
    pl = torch.full((n + 512,), 3.25, device="cuda")
    ws.plan(db.lens)
    hpa.hpa_decode_attn(db.q, db.k, db.v, db.indptr, db.indices, ws.taskmap, C, po[256:-256],
                        pl[256:-256], db.ks, db.vs)
    torch.cuda.synchronize()
    assert ws.status() == 0
    S, rows = int(ws.taskmap[5]), b.q_len * b.Hq
    assert (po[:256] == 3.25).all() and (pl[:256] == 3.25).all()
    assert (po[256 + S * rows * 128:] == 3.25).all() and (pl[256 + S * rows:] == 3.25).all()
    assert not (pl[256:256 + S * rows] == 3.25).any()


def test_calls_without_a_4bit_form_refuse_it():
    b = make_batch([300, 70], 1, (16, 2), seed=32)
    db = DeviceBatch(b)
    ws = hpa.Workspace(b.B, 1, b.Hq, 128, num_ctas=5, Hkv=b.Hkv)
    out = torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(b.q.shape[:3], device="cuda")
    base = (db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, db.ks, db.vs)
    for kw in (dict(fused=True), dict(tc=True), dict(mma=True), dict(allheads=True)):
        with pytest.raises(hpa.HpaError, match="failed"):
            hpa.decode_step(ws, *base, **kw)
    acc = torch.zeros(b.num_pages, b.Hkv, 64, device="cuda")
    with pytest.raises(hpa.HpaError, match="no 4-bit form"):
        hpa.decode_step(ws, *base, acc=acc)
    with pytest.raises(hpa.HpaError):
        hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, db.indices, ws.taskmap, 5, acc)
    kept = torch.zeros(b.B, b.Hkv, 64, dtype=torch.int32, device="cuda")
    with pytest.raises(hpa.HpaError):
        hpa.hpa_evict_compact(db.k, db.v, db.indptr, db.indices, kept, db.lens.clone())
    trace = torch.zeros(4 * 5 * 2, dtype=torch.int64, device="cuda")
    with pytest.raises(hpa.HpaError, match="failed"):
        hpa.hpa_decode_attn_traced(db.q, db.k, db.v, db.indptr, db.indices, ws.taskmap, 5,
                                   ws.partial_o, ws.partial_lse, trace, db.ks, db.vs)
