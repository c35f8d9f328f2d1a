"""hpa_store_qkv: refusals on the host (nothing is launched), and the oracle's pins, on CPU."""
import math

import numpy as np
import pytest
import torch

import load_balanced_split_gb300 as hpa
from oracle import feeder, fourbit, qkv

FAKE = 1 << 20


def _call(**kw):
    a = dict(q=FAKE, sq=1024, k=2 * FAKE, sk=256, v=3 * FAKE, sv=256, n=4, Hq=8, Hkv=2, d=128,
             pos=FAKE, slots=FAKE, cs=FAKE, max_pos=100, rot=128, qn=FAKE, kn=FAKE, eps=1e-6, flags=0,
             qo=4 * FAKE, so=1024, kv=0, ks=None, vs=None, kp=FAKE, vp=FAKE, P=10, page=64, st=None)
    a.update(kw)
    return hpa.lib().hpa_store_qkv(*a.values(), None)


def test_argument_checks():
    for bad in (dict(k=None), dict(v=None), dict(q=None, k=None, v=None), dict(pos=None),
                dict(slots=None), dict(cs=None), dict(qo=None), dict(kp=None), dict(vp=None),
                dict(kv=3), dict(kv=1), dict(kv=2), dict(kv=2, ks=FAKE), dict(n=-1), dict(Hq=0),
                dict(Hkv=0), dict(P=0), dict(max_pos=0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(flags=8), dict(flags=-1), dict(sq=1016), dict(so=1016), dict(sk=248),
                dict(sv=248)):
        assert _call(**bad) == -1, bad
    for bad in (dict(d=64), dict(page=16), dict(rot=96), dict(rot=256), dict(rot=-16), dict(rot=8),
                dict(P=1 << 30), dict(P=1 << 33)):
        assert _call(**bad) == -2, bad
    for bad in (dict(q=FAKE + 8), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(qo=FAKE + 8),
                dict(kp=FAKE + 8), dict(vp=FAKE + 8), dict(sq=1028), dict(sk=260), dict(sv=257),
                dict(so=1028), dict(pos=FAKE + 2), dict(slots=FAKE + 4), dict(cs=FAKE + 8),
                dict(qn=FAKE + 2), dict(kn=FAKE + 1), dict(st=FAKE + 2)):
        assert _call(**bad) == -4, bad
    # queries written over others that are still to be read
    for bad in (dict(qo=FAKE + 16), dict(qo=FAKE + 2048), dict(qo=FAKE, so=1032)):
        assert _call(**bad) == -1, bad
    assert _call(n=0) == 0


def test_what_is_written_lies_apart():
    """Queries over keys or values still to be read, and pools over anything, are refused."""
    far = dict(q=FAKE, k=2 * FAKE, v=3 * FAKE, qo=4 * FAKE, kp=8 * FAKE, vp=16 * FAKE)
    for bad in (dict(qo=2 * FAKE), dict(qo=2 * FAKE + 256), dict(qo=3 * FAKE - 2048),
                dict(qo=2 * FAKE - 256, n=1), dict(vp=8 * FAKE), dict(vp=8 * FAKE + 16384),
                dict(kp=FAKE), dict(vp=4 * FAKE - 32768), dict(kp=2 * FAKE), dict(vp=3 * FAKE + 512),
                # packed rows of 12 heads: queries reaching into the keys, keys before the queries
                dict(q=FAKE, qo=FAKE, k=FAKE + 7 * 256, v=FAKE + 10 * 256, sq=1536, sk=1536,
                     sv=1536, so=1536),
                dict(q=FAKE, qo=FAKE, k=FAKE + 8 * 256, v=FAKE + 11 * 256, sq=1536, sk=1536,
                     sv=1536, so=1536)):
        assert _call(**{**far, **bad}) == -1, bad


def test_binding_refusals():
    t = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(hpa.HpaError, match="neither"):
        hpa.hpa_store_qkv(None, None, None, i, i.long(), None)
    with pytest.raises(hpa.HpaError, match="go together"):
        hpa.hpa_store_qkv(t, t, None, i, i.long(), None)
    with pytest.raises(hpa.HpaError, match="CUDA tensor"):
        hpa.hpa_store_qkv(t, None, None, i, i.long(), None)


def test_oracle_head():
    g = np.random.default_rng(0)
    x = g.standard_normal(128)
    cs = np.zeros((2, 128))
    cs[0, :64] = 1.0
    w = 1 + 0.1 * g.standard_normal(128)
    y, m = qkv.head(x, 0, cs, w, 1e-6, False, False, False)
    np.testing.assert_allclose(y, feeder.rms_norm(x, w, 1e-6), rtol=1e-14)
    assert (m >= np.abs(y) * (1 - 1e-12)).all()
    ang = g.random(64) * 6
    cs[1] = np.concatenate([np.cos(ang), np.sin(ang)])
    y, m = qkv.head(x, 1, cs, w, 1e-6, True, False, True)
    ref = feeder.hadamard(128) @ feeder.rms_norm(feeder.rope_rotate_half(x, cs[1]), w, 1e-6)
    np.testing.assert_allclose(y, ref, rtol=1e-12, atol=1e-14)
    y, _ = qkv.head(x, 1, cs[:, 48:80], None, 0.0, False, True, False)
    z = (x[0:32:2] + 1j * x[1:32:2]) * (cs[1, 48:64] + 1j * cs[1, 64:80])
    np.testing.assert_allclose(y[0:32:2] + 1j * y[1:32:2], z, rtol=1e-13)
    np.testing.assert_array_equal(y[32:], x[32:])


def test_oracle_4bit():
    assert fourbit.decode_e2m1(np.arange(16)).tolist() == [
        0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 7.0, -100.0, 0.0]
    assert fourbit.decode_e2m1(fourbit.encode_e2m1(ties)).tolist() == [
        0, 1, 1, 2, 2, 4, 4, 0, -4, 6, -6, 0]
    g = np.random.default_rng(2)
    y = g.standard_normal((3, 2, 64, 128)) * np.exp(g.standard_normal((3, 2, 64, 1)))
    x = fourbit.values(fourbit.pack(y))
    amax = np.abs(y).reshape(3, 2, 64, 8, 16).max(-1).repeat(16, -1)
    # half the widest step (1 of 6) at a scale that its rounding raised by up to 2^-4, and what
    # saturates when the rounding lowered it
    assert (np.abs(x - y) <= amax / 6 * (1 + 2 ** -4) + 2.0 ** -10 * 6).all()
    codes, scales = fourbit.encode(y)
    c, s = fourbit.unpack(fourbit.pack(y))
    assert (c == codes).all() and (fourbit.e4m3_value(s) == scales).all()
    assert math.isnan(fourbit.e4m3_value(np.array([0x7F]))[0])
