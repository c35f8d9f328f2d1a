"""Refusals of the binding that protect memory, on CPU: page tables and scales shorter than the
batch, and tensors on a device other than the current one, never reach the library."""
import pytest
import torch

import load_balanced_split_gb300 as pkg
import load_balanced_split_gb300.hpa as H

B, Q_LEN, HQ, HKV, D, P = 3, 2, 16, 2, 128, 20


class _Lib:
    """Stands in for the library: records the calls that get through."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    fake = _Lib()
    monkeypatch.setattr(H, "lib", lambda: fake)

    def host_dev(t, name, dtype=None):           # as _dev, without the GPU
        if not (isinstance(t, torch.Tensor) and t.is_contiguous()):
            raise pkg.HpaError("%s must be a contiguous CUDA tensor" % name)
        if dtype is not None and t.dtype is not dtype:
            raise pkg.HpaError("%s must be %s, got %s" % (name, dtype, t.dtype))
        return t
    monkeypatch.setattr(H, "_dev", host_dev)
    monkeypatch.setattr(H, "_n_devices", 1)
    monkeypatch.setattr(H, "_stream", lambda s: 0)
    return fake


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def _store(**kw):
    a = dict(k_new=torch.zeros(B, Q_LEN, HKV, D, dtype=torch.bfloat16),
             v_new=torch.zeros(B, Q_LEN, HKV, D, dtype=torch.bfloat16), seq_lens=_i32(9, 9, 9),
             text_pos=_i32(0, 0, 0), page_indptr=_i32(0, 1, 2, 3), page_indices=_i32(0, 1, 2),
             cos_sin=torch.zeros(50, D), norm_w=torch.zeros(D),
             k_pool=torch.zeros(P, HKV, 64, D, dtype=torch.bfloat16),
             v_pool=torch.zeros(P, HKV, 64, D, dtype=torch.bfloat16), status=_i32(0))
    a.update(kw)
    pkg.hpa_store_kv_at(**a)


def _workspace(window=100):
    return pkg.Workspace(B, Q_LEN, HQ, D, num_ctas=4, Hkv=HKV, device="cpu", window=window)


def _step(monkeypatch, ws=None, **kw):
    a = dict(q=torch.zeros(B, Q_LEN, HQ, D, dtype=torch.bfloat16),
             k_pool=torch.zeros(P, HKV, 64, D, dtype=torch.bfloat16),
             v_pool=torch.zeros(P, HKV, 64, D, dtype=torch.bfloat16), seq_lens=_i32(9, 9, 9),
             page_indptr=_i32(0, 1, 2, 3), page_indices=_i32(0, 1, 2),
             out=torch.zeros(B, Q_LEN, HQ, D, dtype=torch.bfloat16))
    a.update(kw)
    pkg.decode_step(ws or _sized(monkeypatch), **a)


def _sized(monkeypatch):
    """A windowed workspace whose sizes come from the real library's formulas."""
    monkeypatch.setattr(H, "hpa_taskmap_bytes", lambda b, c: 4096)
    monkeypatch.setattr(H, "hpa_max_segments", lambda b, c: b + c - 1)
    monkeypatch.setattr(H, "hpa_arrivals_elems", lambda *a: 1024)
    return _workspace()


def test_store_at_refuses_what_the_kernel_would_read_past(lib):
    _store()
    assert lib.calls == ["hpa_store_kv_at"]
    scale = torch.ones(HKV)
    e4m3 = dict(k_pool=torch.zeros(P, HKV, 64, D, dtype=torch.uint8),
                v_pool=torch.zeros(P, HKV, 64, D, dtype=torch.uint8))
    _store(**e4m3, k_scale=scale, v_scale=scale)
    lib.calls.clear()
    for kw, text in ((dict(page_indptr=_i32(0, 1, 2)), "page_indptr"),
                     (dict(text_pos=_i32(0, 0)), "text_pos"), (dict(seq_lens=_i32(9)), "seq_lens"),
                     (dict(v_new=torch.zeros(B, 1, HKV, D, dtype=torch.bfloat16)), "v_new"),
                     (dict(k_new=torch.zeros(B, Q_LEN, HKV, 64, dtype=torch.bfloat16),
                           v_new=torch.zeros(B, Q_LEN, HKV, 64, dtype=torch.bfloat16)),
                      "head dim"),
                     (dict(v_pool=torch.zeros(P - 1, HKV, 64, D, dtype=torch.bfloat16)), "match"),
                     (dict(v_pool=torch.zeros(P, HKV, 64, D, dtype=torch.uint8)), "v_pool"),
                     (dict(k_pool=torch.zeros(P, HKV, 64, D), v_pool=torch.zeros(P, HKV, 64, D)),
                      "dtype"),
                     (dict(cos_sin=torch.zeros(50, D // 2)), "cos_sin"),
                     (dict(norm_w=torch.zeros(D - 1)), "norm_w"),
                     (dict(status=torch.zeros(1, dtype=torch.int64)), "status"),
                     (dict(e4m3, k_scale=scale, v_scale=scale[:1]), "scale"),
                     (dict(e4m3, k_scale=scale.double(), v_scale=scale), "scale"),
                     (dict(e4m3), "scale")):
        with pytest.raises(pkg.HpaError, match=text):
            _store(**kw)
    assert not lib.calls


def test_windowed_step_refuses_a_short_page_table(lib, monkeypatch):
    _step(monkeypatch)
    assert lib.calls == ["hpa_plan_window", "hpa_decode_attn_window", "hpa_combine"]
    lib.calls.clear()
    with pytest.raises(pkg.HpaError, match="page_indptr"):
        _step(monkeypatch, page_indptr=_i32(0, 1, 2))
    assert "hpa_decode_attn_window" not in lib.calls
    ws = _sized(monkeypatch)
    with pytest.raises(pkg.HpaError, match="page_indptr"):
        pkg.hpa_decode_attn_window(torch.zeros(B, Q_LEN, HQ, D, dtype=torch.bfloat16),
                                   torch.zeros(P, HKV, 64, D, dtype=torch.bfloat16),
                                   torch.zeros(P, HKV, 64, D, dtype=torch.bfloat16),
                                   _i32(0, 1, 2), _i32(0, 1), ws.taskmap, 4, ws.partial_o,
                                   ws.partial_lse)
    assert "hpa_decode_attn_window" not in lib.calls


def test_tensors_of_another_device_are_refused(lib, monkeypatch):
    """Two devices, the current one not that of the tensors (host tensors have device -1)."""
    ws = _sized(monkeypatch)
    monkeypatch.setattr(H, "_n_devices", 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    lib.calls.clear()
    for call in (_store, lambda: ws.plan(_i32(9, 9, 9)), lambda: _step(monkeypatch, ws=ws),
                 lambda: pkg.hpa_plan_window(_i32(9), 1, 5, 0, 64, 2, _i32(*[0] * 400))):
        with pytest.raises(pkg.HpaError, match="current device"):
            call()
    assert not lib.calls
