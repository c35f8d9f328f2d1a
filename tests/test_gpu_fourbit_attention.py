"""Attention over 4-bit pages (hpa_decode_attn and hpa_decode_attn_window with HPA_KV_E2M1)
against the 64-bit definition; slots that no token sees hold NaN scales throughout."""
import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
from bounded_helpers import check_attention
from fourbit_helpers import make_batch, poison_hidden, rows_of, step
from gpu_helpers import DeviceBatch
from oracle import bounded

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


def test_one_long_request_and_a_large_batch():
    _run([70000], 2, heads=(8, 1), seed=3)
    g = np.random.default_rng(4)
    _run(list(g.integers(1, 300, size=400)), 1, heads=(4, 1), seed=4)
