"""4-bit attention at scores far beyond what fp32 resolves: a row's largest score then has all of
its weight.  The kernels' scores are off by DOT * E (bounded_helpers), so rows whose two largest
lie further apart than that, and than what leaves the second a weight, have the value of one key."""
import numpy as np
import pytest
import torch

from bounded_helpers import DOT, lse_bound
from fourbit_helpers import make_batch, poison_hidden, rows_of, step
from gpu_helpers import DeviceBatch
from oracle import bounded, fourbit

pytestmark = pytest.mark.gpu

ROWS = [((8, 1), 1), ((5, 1), 1), ((16, 2), 2), ((9, 1), 1), ((24, 1), 1), ((8, 1), 3), ((8, 1), 4),
        ((16, 2), 4), ((17, 1), 1), ((8, 1), 8)]


def one_key(b, window, sinks):
    """(value of the largest score's key, score, E, whether it is the only one that counts)."""
    k = fourbit.values(b.k_pool.numpy(), b.k_scale)
    v = fourbit.values(b.v_pool.numpy(), b.v_scale)
    q, G = b.q.double().numpy(), b.Hq // b.Hkv
    shape = (b.B, b.q_len, b.Hq)
    val, top, E, alone = (np.zeros(shape + (128,)), np.zeros(shape), np.zeros(shape),
                          np.zeros(shape, bool))
    for r in range(b.B):
        L = int(b.seq_lens[r])
        ids = b.page_indices[int(b.page_indptr[r]):int(b.page_indptr[r + 1])]
        for j in range(b.q_len):
            i = np.array([x for x in range(L) if bounded.sees(L, b.q_len, j, x, window, sinks)])
            for h in range(b.Hq):
                kk, vv = k[ids[i // 64], h // G, i % 64], v[ids[i // 64], h // G, i % 64]
                s = kk @ q[r, j, h] / np.sqrt(128)
                e = (np.abs(kk) @ np.abs(q[r, j, h]) / np.sqrt(128)).max()
                best = int(s.argmax())
                second = np.partition(s, -2)[-2] if len(s) > 1 else -np.inf
                val[r, j, h], top[r, j, h], E[r, j, h] = vv[best], s[best], e
                alone[r, j, h] = s[best] - second > 2 * DOT * e + 60
    return val, top, E, alone


def check(b, window=None, sinks=0, C=None, tile=None):
    want, s, E, alone = one_key(b, window, sinks)
    poison_hidden(b, window, sinks)
    ws, out, lse = step(b, DeviceBatch(b), window, sinks, C, tile)
    torch.cuda.synchronize()
    assert ws.status() == 0
    got, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert alone.mean() > 0.9
    assert np.isfinite(got).all() and np.isfinite(l).all()
    # its probability as f16 (2^-11), the sum's exponential and the division (2^-20 each), bf16
    bound = (2.0 ** -8 + 2.0 ** -10) * np.abs(want)
    assert (np.abs(got - want)[alone] <= bound[alone]).all()
    assert (np.abs(l - s) <= lse_bound(s, E) + np.log(int(max(b.seq_lens)))).all()


@pytest.mark.parametrize("scale", [1e7, 2.0 ** 25, 2.0 ** 26, 2.0 ** 27, 1e9, 1e12, 1e20, 1e33])
@pytest.mark.parametrize("heads,q_len", ROWS)
def test_scores_beyond_what_fp32_resolves(heads, q_len, scale):
    """The largest score is not a whole number of fp32's steps there: a weight taken from the exact
    product less the rounded maximum would be zero, or beyond f16."""
    b = make_batch([300, 70, 1000], q_len, heads, seed=80 + q_len)
    b.q = (b.q.float() * scale).to(torch.bfloat16)
    check(b)


@pytest.mark.parametrize("window,sinks", [(70, 3), (200, 0)])
@pytest.mark.parametrize("heads,q_len", ROWS[::2])
def test_such_scores_in_windows_and_many_segments(heads, q_len, window, sinks):
    for scale in (2.0 ** 26, 1e12):
        b = make_batch([300, 70, 1000], q_len, heads, seed=90 + q_len)
        b.q = (b.q.float() * scale).to(torch.bfloat16)
        check(b, window, sinks)
        b = make_batch([900, 1300], q_len, heads, seed=91 + q_len)
        b.q = (b.q.float() * scale).to(torch.bfloat16)
        check(b, C=14, tile=64)


def one_step_apart(heads, q_len, window=None, C=1):
    """Scores of 2^26 and one slack, 8, more in base 2 (8 is fp32's step there), exact in every
    type on the way; all others are 0.  The weights are 256 to 1, whatever the order of the keys."""
    for first, second in ((0, 400), (400, 0), (3, 5)):
        b = make_batch([600], q_len, heads, seed=120)
        keep = torch.zeros(b.q.shape, dtype=torch.bool)
        keep[..., :2] = True
        b.q[~keep] = 0
        b.q[..., 0], b.q[..., 1] = 2.0 ** 20, 0.25
        b.k_scale[:] = 1.0
        codes, scales = rows_of(b.k_pool)
        codes.zero_()
        scales[:] = int(fourbit.e4m3_byte(32.0))
        v = fourbit.values(b.v_pool.numpy(), b.v_scale)
        at = {}
        for i, code in ((first, 0x04), (second, 0x24)):      # (64, 0) and (64, 32)
            page = int(b.page_indices[i // 64])
            codes[page, :, i % 64, 0] = code
            at[i] = v[page, :, i % 64]
        sm = np.float32(np.log(2.0))
        while np.float32(sm * np.float32(1.4426950408889634)) < 1:
            sm = np.nextafter(sm, np.float32(1))
        assert np.float32(sm * np.float32(1.4426950408889634)) == 1
        ws, out, lse = step(b, DeviceBatch(b), window, 0, C, 64, sm_scale=float(sm))
        torch.cuda.synchronize()
        assert ws.status() == 0
        got = out.double().cpu().numpy()
        a, z = at[first], at[second]
        want = ((256 * z + a) / 257).repeat(b.Hq // b.Hkv, 0)[None, None]
        size = ((256 * np.abs(z) + np.abs(a)) / 257).repeat(b.Hq // b.Hkv, 0)[None, None]
        # f16 probabilities (exact powers of two), sums and division (2^-20), merged partials, whose
        # lse is off by fp32's step at 2^26 ln 2, 4 (1 with C == 1), and bf16
        if C == 1:
            assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size).all()
        lo, hi = np.minimum(a, z), np.maximum(a, z)          # in any case a mean of the two
        lo, hi = (x.repeat(b.Hq // b.Hkv, 0)[None, None] for x in (lo, hi))
        slack = 2.0 ** -7 * np.maximum(np.abs(lo), np.abs(hi))
        assert (got >= lo - slack).all() and (got <= hi + slack).all()
        assert np.abs(lse.double().cpu().numpy() - 2.0 ** 26 * np.log(2)).max() <= 16


@pytest.mark.parametrize("C", [1, 7])
@pytest.mark.parametrize("heads,q_len", [((8, 1), 1), ((5, 1), 1), ((16, 2), 2), ((9, 1), 1),
                                         ((17, 1), 1), ((24, 1), 1), ((8, 1), 4), ((40, 1), 1)])
def test_two_keys_one_step_apart(heads, q_len, C):
    one_step_apart(heads, q_len, None, C)
    one_step_apart(heads, q_len, 650, C)


@pytest.mark.parametrize("window,sinks", [(None, 0), (70, 3)])
@pytest.mark.parametrize("heads,q_len", ROWS)
def test_a_first_maximum_below_any_constant(heads, q_len, window, sinks):
    """Every score of every row is near -1e33 (keys without a negative element, queries without a
    positive one), in tiles without a row of padding too."""
    b = make_batch([300, 70, 500, q_len], q_len, heads, seed=100 + q_len)
    b.k_pool[..., :fourbit.CODES] &= 0x77
    b.q = (-b.q.float().abs() * 1e33).to(torch.bfloat16)
    check(b, window, sinks)
