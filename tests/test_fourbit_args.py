"""4-bit caches at the C entry points: refusals on the host (nothing is launched), on CPU."""
import load_balanced_split_gb300 as hpa

FAKE = 1 << 20
E2M1 = hpa.KV_E2M1


def _attn(entry, *more, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, kv=E2M1, ks=FAKE, vs=FAKE, P=100, ip=FAKE, ix=FAKE, page=64, B=3,
             q_len=1, Hq=64, Hkv=8, d=128, scale=0.088, tm=FAKE, C=4, po=FAKE, pl=FAKE)
    a.update(kw)
    return getattr(hpa.lib(), entry)(*a.values(), *more, None)


def test_attention_checks():
    for entry in ("hpa_decode_attn", "hpa_decode_attn_window"):
        assert _attn(entry, ks=None) == -1 and _attn(entry, vs=None) == -1
        assert _attn(entry, kv=3) == -1 and _attn(entry, C=0) == -1
        assert _attn(entry, d=64) == -2 and _attn(entry, page=32) == -2 and _attn(entry, q_len=9) == -2
        assert _attn(entry, P=1 << 29) == -2
        assert _attn(entry, k=FAKE + 8) == -4 and _attn(entry, v=FAKE + 4) == -4


def test_calls_without_a_4bit_form():
    assert _attn("hpa_decode_attn_mma") == -2 and _attn("hpa_decode_attn_tc") == -2
    assert _attn("hpa_decode_attn_traced", FAKE) == -2
    assert _attn("hpa_decode_attn_allheads", None) == -2
    assert _attn("hpa_decode_attn_fused", FAKE, None, FAKE) == -2
    L = hpa.lib()
    assert L.hpa_store_kv(FAKE, FAKE, FAKE, FAKE, FAKE, 10, 64, FAKE, 100, FAKE, 1e-6, 1, E2M1, FAKE,
                          FAKE, FAKE, FAKE, 2, 1, 8, 128, None, None) == -1
    assert L.hpa_key_weights(FAKE, FAKE, FAKE, E2M1, FAKE, 100, FAKE, FAKE, 64, 3, 1, 64, 8, 128, 0.1,
                             1.0, FAKE, 4, FAKE, FAKE, None) == -1
    assert L.hpa_evict_compact(FAKE, FAKE << 1, E2M1, None, 10, FAKE, FAKE, None, None, 64, FAKE, 100,
                               FAKE, 3, 8, 128, None, None) == -1
    assert L.hpa_default_num_ctas_mma(64, 8, 1, E2M1) == -1
    assert L.hpa_default_num_ctas_tc(64, 8, 1, E2M1) == -1
    for bad in ((63, 8, 1), (64, 0, 1), (64, 8, 0), (64, 8, 9)):
        assert L.hpa_default_num_ctas(*bad, E2M1) == -1
        assert L.hpa_default_num_ctas_window(*bad, E2M1) == -1


def test_page_size_constant():
    assert hpa.E2M1_PAGE_BYTES == 64 * 64 + 64 * 8
