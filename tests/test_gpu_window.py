"""Sliding-window decode attention with sink tokens (hpa_plan_window, hpa_decode_attn_window)
against the 64-bit definition, every hidden slot holding NaN."""
import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from bounded_helpers import check_attention, nan_code, poison_hidden, window_step
from gpu_helpers import DeviceBatch, decode_taskmap, run_gpu
from oracle import bounded

pytestmark = pytest.mark.gpu


def _check_map(ws, b, window, sinks, tile):
    tm = decode_taskmap(ws.taskmap.cpu().numpy(), b.B, ws.num_ctas)
    ref, _ = bounded.window_plan(b.seq_lens, b.q_len, window, sinks, tile, ws.num_ctas)
    assert tm["status"] == 0 and tm["kind"] == 3
    for k in ("T", "base", "rem", "C", "B", "S", "tile"):
        assert tm[k] == ref[k], (k, tm[k], ref[k])
    assert list(tm["header_tail"]) == [window, sinks, b.q_len, 0, 0]
    np.testing.assert_array_equal(tm["lens"], b.seq_lens)
    for k in ("cu_tiles", "cta_begin", "cta_seg", "seg_off", "segs"):
        np.testing.assert_array_equal(tm[k], ref[k], err_msg=k)


def _run(lens, q_len, kv, window, sinks, heads=(16, 2), C=None, tile=None, seed=0):
    b = W.make_batch(lens, q_len=q_len, kv_dtype=kv, seed=seed, Hq=heads[0], Hkv=heads[1])
    poison_hidden(b, window, sinks)
    db = DeviceBatch(b)
    ws, out, lse = window_step(b, db, window, sinks, C, tile)
    torch.cuda.synchronize()
    _check_map(ws, b, window, sinks, tile or 64)
    check_attention(b, out, lse, bounded.attention_rows(b, window, sinks), kv)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 4), (64, 0), (65, 64), (128, 65),
                                          (200, 3), (1000, 300), (1 << 30, 1 << 30)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_lengths_around_every_border(kv, window, sinks, q_len):
    lens = [q_len, 63, 64, 65, 127, 130, 191, 200, 257, 449, 700, 1111]
    _run(lens, q_len, kv, window, sinks, seed=window % 97 + sinks % 89)


@pytest.mark.parametrize("heads,q_len", [((2, 2), 1), ((8, 1), 8), ((5, 1), 1), ((40, 8), 4),
                                         ((32, 2), 1), ((48, 4), 2), ((12, 3), 5),
                                         ((64, 8), 5)])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_head_layouts(kv, heads, q_len):
    _run([q_len, 90, 400, 777], q_len, kv, 130, 7, heads, seed=heads[0])


@pytest.mark.parametrize("C,tile", [(1, 64), (3, 128), (23, 64), (40, 512), (200, 64)])
def test_partitions_and_tiles(C, tile):
    _run([1, 500, 1300, 40, 640], 1, "bf16", 333, 70, C=C, tile=tile, seed=C)


def test_one_long_request_and_a_large_batch():
    _run([70000], 2, "e4m3", 1500, 100, (8, 1), seed=3)
    g = np.random.default_rng(4)
    _run(list(g.integers(1, 300, size=400)), 1, "bf16", 50, 2, (4, 1), seed=4)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_wide_window_gives_the_full_step(kv):
    """A window beyond every length: the same partials as the mma.sync kernel, bit for bit."""
    b = W.make_batch([700, 64, 3, 2000], q_len=2, kv_dtype=kv, seed=5)
    db = DeviceBatch(b)
    full = run_gpu(b, num_ctas=9, tile=128, db=db, mma=True)
    ws, out, lse = window_step(b, db, 1 << 20, 0, C=9, tile=128)
    torch.cuda.synchronize()
    assert (out.float().cpu().numpy() == full["out"]).all()
    assert (lse.cpu().numpy() == full["lse"]).all()


@pytest.mark.parametrize("kv,bad", [("bf16", float("nan")), ("bf16", float("inf")),
                                    ("bf16", float("-inf")), ("e4m3", float("nan"))])
def test_nonfinite_values_reach_only_the_rows_that_see_them(kv, bad):
    window, sinks, q_len = 70, 5, 4
    b = W.make_batch([300, 33, 641], q_len=q_len, kv_dtype=kv, seed=6, Hq=8, Hkv=2)
    poison_hidden(b, window, sinks)
    for r in range(b.B):
        L = int(b.seq_lens[r])
        ids = b.page_indices[int(b.page_indptr[r]):int(b.page_indptr[r + 1])]
        low = max(0, L - q_len + 1 - window)
        for i, dim in ((L - 1, 3), (L - 2, 77), (low, 127), (low + 1, 0)):
            if L > 33 or i >= L - 2:
                b.v_pool[ids[i // 64], :, i % 64, dim] = nan_code(kv) if bad != bad else bad
    db = DeviceBatch(b)
    ws, out, lse = window_step(b, db, window, sinks)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        o, l, A, E = bounded.attention_rows(b, window, sinks)
    assert np.isfinite(o).any(axis=(2, 3)).all() and not np.isfinite(o).all()
    check_attention(b, out, lse, (o, l, np.where(np.isfinite(A), A, 0), E), kv)


def test_graph_replay_follows_new_lengths():
    """A captured step replayed after lengths and queries change in place, on its own stream."""
    b = W.make_batch([900, 300], q_len=1, seed=7, Hq=16, Hkv=2)
    db = DeviceBatch(b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws, out, lse = window_step(b, db, 100, 4, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse)
    for lens in ([900, 300], [555, 1], [64, 299]):
        b.seq_lens = np.array(lens, np.int32)
        db.lens.copy_(torch.from_numpy(b.seq_lens))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check_attention(b, out, lse, bounded.attention_rows(b, 100, 4), "bf16")


def _status_after(b, db, lens=None, indices=None, q_len=None):
    ws = hpa.Workspace(b.B, b.q_len, b.Hq, b.d, num_ctas=5, Hkv=b.Hkv, window=100, sinks=4)
    ws.q_len = q_len or b.q_len
    out = torch.zeros((b.B, b.q_len, b.Hq, b.d), dtype=torch.bfloat16, device="cuda")
    hpa.decode_step(ws, db.q, db.k, db.v, db.lens if lens is None else lens, db.indptr,
                    db.indices if indices is None else indices, out)
    torch.cuda.synchronize()
    return ws.status(), out


def test_device_side_refusals():
    b = W.make_batch([400, 200], q_len=2, seed=8, Hq=16, Hkv=2)
    db = DeviceBatch(b)
    st, out = _status_after(b, db, lens=torch.tensor([400, 1], dtype=torch.int32, device="cuda"))
    assert st & 1 and out.isnan().all()                        # shorter than its new tokens
    bad = db.indices.clone()
    bad[6] = b.num_pages
    st, out = _status_after(b, db, indices=bad)                # the page of request 0's last keys
    assert st & 4 and out.isnan().all()
    st, out = _status_after(b, db, q_len=1)                    # planned for another q_len
    assert st & 2 and out.isnan().all()


def test_other_attention_calls_refuse_a_window_map():
    b = W.make_batch([400, 200], seed=9, Hq=16, Hkv=2)
    db = DeviceBatch(b)
    for kernel in ({}, {"tc": True}, {"mma": True}):
        ws = hpa.Workspace(b.B, 1, b.Hq, b.d, num_ctas=5, Hkv=b.Hkv, window=100, sinks=4)
        ws.plan(db.lens)
        hpa.hpa_decode_attn(db.q, db.k, db.v, db.indptr, db.indices, ws.taskmap, 5, ws.partial_o,
                            ws.partial_lse, **kernel)
        torch.cuda.synchronize()
        assert ws.status() == 32
    ws = hpa.Workspace(b.B, 1, b.Hq, b.d, num_ctas=5, Hkv=b.Hkv)
    ws.plan(db.lens)
    hpa.hpa_decode_attn_window(db.q, db.k, db.v, db.indptr, db.indices, ws.taskmap, 5,
                               ws.partial_o, ws.partial_lse)
    torch.cuda.synchronize()
    assert ws.status() == 32
