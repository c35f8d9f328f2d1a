"""The lse of 4-bit attention's rows that see a NaN: NaN, not the -inf of a row without keys, from
one segment and from many, through either form of the combine."""
import numpy as np
import pytest
import torch

from bounded_helpers import lse_bound, out_bound
from fourbit_helpers import make_batch, poison_hidden, rows_of, step
from gpu_helpers import DeviceBatch
from oracle import bounded

pytestmark = pytest.mark.gpu

# lengths, partitions, keys a tile: a request of one segment, requests of a few (a warp for each
# row merges them), one request of more than four (a block for each row)
CUTS = [([40, 64], 1, 512), ([300, 200, 131], 5, 64), ([1500], 12, 64)]
ROWS = [((8, 2), 2), ((16, 2), 2), ((8, 1), 3), ((16, 2), 4)]


@pytest.mark.parametrize("lens,C,tile", CUTS)
@pytest.mark.parametrize("heads,q_len", ROWS)
@pytest.mark.parametrize("window,sinks", [(None, 0), (70, 3)])
def test_a_nan_key(heads, q_len, lens, C, tile, window, sinks):
    b = make_batch(lens, q_len, heads, seed=110)
    poison_hidden(b, window, sinks)
    ref = bounded.attention_rows(b, window, sinks)
    hit = np.zeros(ref[1].shape, bool)
    G = b.Hq // b.Hkv
    for r, L in enumerate(lens):
        i, h = L - 1, r % b.Hkv                # the last token alone sees it
        page = int(b.page_indices[int(b.page_indptr[r]) + i // 64])
        rows_of(b.k_pool)[1][page, h, i % 64, r] = 0x7F
        hit[r, q_len - 1, h * G:(h + 1) * G] = True
    ws, out, lse = step(b, DeviceBatch(b), window, sinks, C, tile)
    torch.cuda.synchronize()
    assert ws.status() == 0
    got, l = out.float().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(got[hit]).all() and not np.isnan(got[~hit]).any()
    assert np.isnan(l[hit]).all()
    assert (np.abs(l - ref[1])[~hit] <= lse_bound(ref[1], ref[3])[~hit]).all()


@pytest.mark.parametrize("lens,C,tile", CUTS)
@pytest.mark.parametrize("heads,q_len", ROWS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_query_row(heads, q_len, lens, C, tile, bad):
    b = make_batch(lens, q_len, heads, seed=111)
    ref = bounded.attention_rows(b)
    hit = np.zeros(ref[1].shape, bool)
    for r in range(len(lens)):
        b.q[r, r % q_len, 3 * r + 1, 5 * r] = bad
        hit[r, r % q_len, 3 * r + 1] = True
    ws, out, lse = step(b, DeviceBatch(b), C=C, tile=tile)
    torch.cuda.synchronize()
    assert ws.status() == 0
    got, l = out.float().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(got[hit]).all() and not np.isnan(got[~hit]).any()
    assert np.isnan(l[hit]).all()
    assert (np.abs(l - ref[1])[~hit] <= lse_bound(ref[1], ref[3])[~hit]).all()


@pytest.mark.parametrize("heads,q_len", ROWS)
def test_a_nan_value_leaves_the_lse(heads, q_len):
    b = make_batch([300, 200], q_len, heads, seed=112)
    ref = bounded.attention_rows(b)
    rows_of(b.v_pool)[1][int(b.page_indices[1]), :, 5, 2] = 0x7F
    ws, out, lse = step(b, DeviceBatch(b))
    torch.cuda.synchronize()
    assert np.isnan(out.float().cpu().numpy()[0, ..., 32:48]).all()
    assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= lse_bound(ref[1], ref[3])).all()


@pytest.mark.parametrize("at", [5, 700, 1999])
@pytest.mark.parametrize("heads,q_len", ROWS)
def test_a_nan_key_among_rising_scores(heads, q_len, at):
    """The maximum moves with nearly every tile, before and after the NaN."""
    b = make_batch([2000, 1300], q_len, heads, seed=113)
    _, scales = rows_of(b.k_pool)
    for r in range(2):
        ids = b.page_indices[int(b.page_indptr[r]):int(b.page_indptr[r + 1])]
        for n, page in enumerate(ids):   # scales of a page, 2^(n / 4) times as large in all
            scales[page] = (scales[page].to(torch.int32) // 4 + 2 * min(n, 40)).to(torch.uint8)
    ref = bounded.attention_rows(b)
    scales[int(b.page_indices[at // 64]), 0, at % 64, 3] = 0x7F
    hit = np.zeros(ref[1].shape, bool)
    sees = [j for j in range(q_len) if at <= 2000 - q_len + j]
    hit[0, sees, :b.Hq // b.Hkv] = True
    ws, out, lse = step(b, DeviceBatch(b), C=2, tile=512)
    torch.cuda.synchronize()
    assert ws.status() == 0
    got, l = out.float().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isnan(got[hit]).all() and np.isnan(l[hit]).all()
    bound = out_bound(ref[0], ref[2], ref[3], "e2m1")
    assert (np.abs(got - ref[0])[~hit] <= bound[~hit]).all()
    assert (np.abs(l - ref[1])[~hit] <= lse_bound(ref[1], ref[3])[~hit]).all()
