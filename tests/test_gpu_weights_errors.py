"""Key weights with an error in one request: every other request's weights are updated in full,
whenever its partitions run."""
import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
import workloads as W
from gpu_helpers import DeviceBatch

pytestmark = pytest.mark.gpu

B, C, HKV = 300, 4000, 4          # 16000 blocks, tens of times what the GPU holds at once


def _state(q_len=2):
    lens = [640] * B
    b = W.make_batch(lens, q_len=q_len, seed=5, Hq=2 * HKV, Hkv=HKV)
    db = DeviceBatch(b)
    lse = torch.full((B, q_len, 2 * HKV), 3.0, device="cuda")
    acc0 = torch.rand((b.num_pages, HKV, 64), device="cuda")
    return b, db, lse, acc0


def _weights(db, lse, acc0, lens=None, indices=None, corrupt=None, calls=1):
    ws = hpa.Workspace(B, db.q.shape[1], 2 * HKV, 128, num_ctas=C, Hkv=HKV)
    ws.plan(db.lens if lens is None else lens, tile=64)
    if corrupt:
        tm = ws.taskmap.cpu()
        corrupt(tm)
        ws.taskmap.copy_(tm)
    acc = acc0.clone()
    for _ in range(calls):                                  # an error stops those that follow
        hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, db.indices if indices is None else indices,
                            ws.taskmap, C, acc, decay=0.5)
    torch.cuda.synchronize()
    assert ws.taskmap[14:16].tolist() == [0, 0]
    return ws.status(), acc


@pytest.mark.parametrize("calls", [1, 3])
@pytest.mark.parametrize("what", ["page", "length", "segment"])
def test_other_requests_are_updated_in_full(what, calls):
    b, db, lse, acc0 = _state()
    st, want = _weights(db, lse, acc0)
    assert st == 0
    touched = np.ones(b.num_pages, bool)
    if what == "page":
        bad = db.indices.clone()
        bad[3] = -1
        st, got = _weights(db, lse, acc0, indices=bad, calls=calls)
        assert st == 4
        touched[b.page_indices[3]] = False
    elif what == "length":
        lens = db.lens.clone()
        lens[0] = 1
        st, got = _weights(db, lse, acc0, lens=lens, calls=calls)
        assert st == 1
        touched[b.page_indices[:10]] = False
    else:
        segs = ((16 + B + 2 * (B + 1) + 2 * (C + 1)) + 3) & ~3

        def corrupt(tm):
            tm[segs] = -7                                   # the first segment's request
        st, got = _weights(db, lse, acc0, corrupt=corrupt, calls=calls)
        assert st == 32
        touched[b.page_indices[0]] = False
    want[torch.from_numpy(~touched).cuda()] = acc0[torch.from_numpy(~touched).cuda()]
    assert torch.equal(got, want), int((got != want).sum())


def test_errors_of_earlier_kernels_stop_the_call():
    """A status that the plan or the attention step set leaves every accumulator as it was."""
    b, db, lse, acc0 = _state()
    for bit in (1, 4, 8, 32):
        def corrupt(tm):
            tm[6] = bit
        st, got = _weights(db, lse, acc0, corrupt=corrupt)
        assert st == bit and torch.equal(got, acc0)


def test_the_attention_step_still_reports_what_key_weights_found():
    b, db, lse, acc0 = _state()
    ws = hpa.Workspace(B, 2, 2 * HKV, 128, num_ctas=C, Hkv=HKV)
    ws.plan(db.lens, tile=64)
    bad = db.indices.clone()
    bad[3] = -1
    hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, bad, ws.taskmap, C, acc0.clone())
    out = torch.zeros((B, 2, 2 * HKV, 128), dtype=torch.bfloat16, device="cuda")
    hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, plan=False)
    torch.cuda.synchronize()
    assert ws.status() == 4 and out.isnan().all()
    hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, tile=64)
    torch.cuda.synchronize()
    assert ws.status() == 0 and not out.isnan().any()        # a new plan starts afresh


def test_a_step_after_an_error_adds_nothing():
    """Layer after layer on one plan: the first one's weights meet a bad page of their own, the
    attention of the next gives NaN, and its weights leave every accumulator as it was."""
    b, db, lse, acc0 = _state()
    ws = hpa.Workspace(B, 2, 2 * HKV, 128, num_ctas=C, Hkv=HKV)
    ws.plan(db.lens, tile=64)
    bad = db.indices.clone()
    bad[3] = -1
    hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, bad, ws.taskmap, C, acc0.clone())
    out = torch.zeros((B, 2, 2 * HKV, 128), dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        acc = acc0.clone()
        hpa.decode_step(ws, db.q, db.k, db.v, db.lens, db.indptr, db.indices, out, lse, acc=acc,
                        plan=False)
        torch.cuda.synchronize()
        assert ws.status() == 4 and lse.isnan().all() and torch.equal(acc, acc0)


def test_calls_over_one_map_on_two_streams():
    """Two layers' weights at once, over and over: each as if alone, the map's two words zero
    again, and an error in a later call still reported."""
    b, db, lse, acc0 = _state()
    _, want = _weights(db, lse, acc0)
    ws = hpa.Workspace(B, 2, 2 * HKV, 128, num_ctas=C, Hkv=HKV)
    ws.plan(db.lens, tile=64)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    accs = [[acc0.clone() for _ in range(4)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(4):
        for s, a in zip(streams, accs):
            hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, db.indices, ws.taskmap, C, a[i],
                                decay=0.5, stream=s)
    torch.cuda.synchronize()
    assert ws.status() == 0 and ws.taskmap[14:16].tolist() == [0, 0]
    assert all(torch.equal(a, want) for group in accs for a in group)
    bad = db.indices.clone()
    bad[-1] = -1                                            # the last blocks' page
    hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, bad, ws.taskmap, C, acc0.clone())
    assert ws.status() == 4


def test_calls_of_other_head_counts_one_after_the_other():
    """The blocks of a call are counted in the map: a call of another size begins from zero."""
    b, db, lse, acc0 = _state()
    ws = hpa.Workspace(B, 2, 2 * HKV, 128, num_ctas=C, Hkv=HKV)
    ws.plan(db.lens, tile=64)
    for heads in (1, 3, HKV):
        k, a = db.k[:, :heads].contiguous(), acc0[:, :heads].contiguous()
        hpa.hpa_key_weights(db.q[:, :, :2 * heads].contiguous(),
                            lse[:, :, :2 * heads].contiguous(), k, db.indptr, db.indices,
                            ws.taskmap, C, a)
        assert ws.status() == 0 and ws.taskmap[14:16].tolist() == [0, 0]
    bad = db.indices.clone()
    bad[-1] = -1
    hpa.hpa_key_weights(db.q, lse, db.k, db.indptr, bad, ws.taskmap, C, acc0.clone())
    assert ws.status() == 4 and ws.taskmap[14:16].tolist() == [0, 0]
