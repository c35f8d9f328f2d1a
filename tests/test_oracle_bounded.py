"""The bounded-cache oracle against closed forms, brute force and the unsplit oracle."""
import math

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from oracle import bounded


@pytest.mark.parametrize("L,q_len,window,sinks", [
    (1, 1, 1, 0), (64, 1, 64, 0), (65, 1, 1, 0), (200, 1, 10, 0), (200, 3, 10, 4),
    (1000, 2, 100, 70), (1000, 2, 100, 870), (1000, 8, 5000, 3), (513, 1, 64, 64)])
def test_window_pages_are_those_with_a_visible_key(L, q_len, window, sinks):
    seen = {i // 64 for i in range(L) for j in range(q_len)
            if bounded.sees(L, q_len, j, i, window, sinks)}
    got = bounded.window_pages(L, q_len, window, sinks)
    assert set(got) == seen and got == sorted(got)


def test_wide_window_is_causal_attention():
    b = W.make_batch([3, 70, 130], q_len=2, Hq=4, Hkv=2, seed=1)
    ref, ref_lse = oracle.attention(b)
    for window, sinks in ((None, 0), (1 << 20, 0), (1, 1 << 20)):
        out, lse, _, _ = bounded.attention_rows(b, window, sinks)
        np.testing.assert_allclose(out, ref, atol=1e-12)
        np.testing.assert_allclose(lse, ref_lse, atol=1e-12)


def test_window_of_one_key_is_its_value():
    b = W.make_batch([100], q_len=3, Hq=2, Hkv=1, seed=2)
    out, _, _, _ = bounded.attention_rows(b, window=1)
    V = bounded.keys_of(b, bounded.pool_values(b.v_pool, "bf16"), 0, 0)
    for j in range(3):
        np.testing.assert_allclose(out[0, j, 0], V[97 + j], atol=1e-14)


def test_weights_of_a_step_sum_to_its_rows():
    """With the true lse every row spreads a weight of 1 over its keys."""
    for window, sinks in ((None, 0), (40, 3)):
        b = W.make_batch([2, 150], q_len=2, Hq=6, Hkv=2, kv_dtype="e4m3", seed=3)
        _, lse, _, _ = bounded.attention_rows(b, window, sinks)
        acc = np.zeros((b.num_pages, 2, 64))
        new, written, _ = bounded.key_weights(b, lse, acc, 1.0, window, sinks)
        assert new[~written].sum() == 0
        np.testing.assert_allclose(new.sum(axis=(0, 2)), [2 * 2 * 3] * 2, rtol=1e-12)


def test_weights_start_and_decay():
    b = W.make_batch([5], q_len=2, Hq=1, Hkv=1, seed=4)
    b.q = torch.zeros_like(b.q)                      # uniform: 1/4 and 1/5 a key
    lse = np.array([[[math.log(4)], [math.log(5)]]])
    new, written, _ = bounded.key_weights(b, lse, np.full((1, 1, 64), 8.0), 0.5)
    np.testing.assert_allclose(new[0, 0, :6], [4.45, 4.45, 4.45, .45, .2, 8.0], rtol=1e-12)
    assert written[0, 0].sum() == 5


def test_kept_keys_by_hand_and_by_comparison():
    nan, inf = math.nan, math.inf
    assert bounded.kept_keys([5, 1, 2, 2, 2, 9], 4, 1, 1) == [0, 2, 3, 5]
    assert bounded.kept_keys([1, 2, 3], 3, 0, 0) == [0, 1, 2]
    assert bounded.kept_keys([0.0, -0.0, 1, -1, nan, inf, -inf], 4, 0, 0) == [0, 2, 4, 5]
    assert bounded.kept_keys([1, 2, 3, 4], 2, 1, 1) == [0, 3]
    g = np.random.default_rng(5)
    for _ in range(50):
        n = int(g.integers(4, 40))
        w = [float(x) for x in g.integers(0, 5, n)]
        if g.random() < 0.3:
            w[int(g.integers(n))] = nan
        s, rec = int(g.integers(0, 2)), int(g.integers(0, 2))
        budget = int(g.integers(max(1, s + rec), n))
        kept = bounded.kept_keys(w, budget, s, rec)
        free = range(s, n - rec)
        ahead = {i: sum(bounded.heavier(w[j], j, w[i], i) for j in free if j != i) for i in free}
        want = sorted([*range(s), *(i for i in free if ahead[i] < budget - s - rec),
                       *range(n - rec, n)])
        assert kept == want
