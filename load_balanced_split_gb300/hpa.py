"""Python binding of libhpa (ctypes): the C entry points under the same names.

Argument marshalling only -- every step of the path runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors; shapes are taken from them and
checked by the library, which returns an error code (raised here as
HpaError) before launching anything on bad input.  There is no CPU path: if
the shared library is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

from . import build as _build

KV_BF16, KV_E4M3 = 0, 1
STATUS_BITS = {1: "BAD_SEQLEN", 2: "MISMATCH", 4: "BAD_PAGE", 8: "TIMEOUT", 16: "OVERFLOW",
               32: "BAD_MAP", 64: "BAD_BUDGET"}
HEADER_WORDS = 16

_lock = threading.Lock()
_lib = None


class HpaError(RuntimeError):
    pass


def lib():
    """Load libhpa.so (building it first if it is missing or older than its sources)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if _build._stale():
                try:
                    path = _build.build()
                except Exception as e:  # no nvcc, or a compile error: fail loudly
                    raise HpaError("libhpa.so is not built and cannot be built: %s" % e)
            L = ctypes.CDLL(path)
            P, I32, I64, SZ, F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                  ctypes.c_size_t, ctypes.c_float)
            sig = {
                "hpa_taskmap_bytes": ([I32, I32], SZ),
                "hpa_max_segments": ([I32, I32], I32),
                "hpa_static_num_ctas": ([I32, I32], I32),
                "hpa_static_taskmap_bytes": ([I32, I32], SZ),
                "hpa_default_num_ctas": ([I32, I32, I32, I32], I32),
                "hpa_plan": ([P, I32, I32, I32, P, SZ, P], ctypes.c_int),
                "hpa_plan_static": ([P, I32, I32, I32, P, SZ, P], ctypes.c_int),
                "hpa_plan_weighted": ([P, I32, I32, I32, P, SZ, P], ctypes.c_int),
                "hpa_decode_attn": ([P, P, P, I32, P, P, I64, P, P, I32, I32, I32, I32, I32,
                                     I32, F, P, I32, P, P, P], ctypes.c_int),
                "hpa_decode_attn_tc": ([P, P, P, I32, P, P, I64, P, P, I32, I32, I32, I32, I32,
                                        I32, F, P, I32, P, P, P], ctypes.c_int),
                "hpa_default_num_ctas_tc": ([I32, I32, I32, I32], I32),
                "hpa_decode_attn_mma": ([P, P, P, I32, P, P, I64, P, P, I32, I32, I32, I32, I32,
                                         I32, F, P, I32, P, P, P], ctypes.c_int),
                "hpa_default_num_ctas_mma": ([I32, I32, I32, I32], I32),
                "hpa_decode_attn_allheads": ([P, P, P, I32, P, P, I64, P, P, I32, I32, I32, I32,
                                              I32, I32, F, P, I32, P, P, P, P], ctypes.c_int),
                "hpa_default_num_ctas_allheads": ([I32, I32, I32, I32], I32),
                "hpa_decode_attn_traced": ([P, P, P, I32, P, P, I64, P, P, I32, I32, I32, I32,
                                            I32, I32, F, P, I32, P, P, P, P], ctypes.c_int),
                "hpa_combine": ([P, P, P, I32, I32, I32, I32, I32, P, P, P], ctypes.c_int),
                "hpa_arrivals_elems": ([I32, I32, I32, I32], SZ),
                "hpa_decode_attn_fused": ([P, P, P, I32, P, P, I64, P, P, I32, I32, I32, I32,
                                           I32, I32, F, P, I32, P, P, P, P, P, P],
                                          ctypes.c_int),
                "hpa_selftest_wait_timeout": ([P, I64, P], ctypes.c_int),
                "hpa_decode_attn_combine_noalloc": ([P, P, P, I32, P, P, I64, P, P, I32, I32,
                                                     I32, I32, I32, I32, F, P, I32, P, P, P],
                                                    ctypes.c_int),
                "hpa_store_kv": ([P, P, P, P, P, I64, I32, P, I32, P, F, I32, I32, P, P, P, P,
                                  I32, I32, I32, I32, P, P], ctypes.c_int),
                "hpa_plan_window": ([P, I32, I32, I32, I32, I32, I32, P, SZ, P], ctypes.c_int),
                "hpa_decode_attn_window": ([P, P, P, I32, P, P, I64, P, P, I32, I32, I32, I32,
                                            I32, I32, F, P, I32, P, P, P], ctypes.c_int),
                "hpa_default_num_ctas_window": ([I32, I32, I32, I32], I32),
                "hpa_store_kv_at": ([P, P, P, P, P, P, I64, I32, P, I32, P, F, I32, I32, P, P, P,
                                     P, I32, I32, I32, I32, P, P], ctypes.c_int),
                "hpa_key_weights": ([P, P, P, I32, P, I64, P, P, I32, I32, I32, I32, I32, I32, F,
                                     F, P, I32, P, P, P], ctypes.c_int),
                "hpa_evict_select": ([P, P, P, P, I64, I32, P, I32, I32, I32, I32, P, I64, P, P,
                                      P], ctypes.c_int),
                "hpa_evict_compact": ([P, P, I32, P, I64, P, P, P, P, I32, P, I64, P, I32, I32,
                                       I32, P, P], ctypes.c_int),
                "hpa_evict": ([P, P, I32, P, I64, P, P, P, P, P, I32, P, I32, I32, I32, I32, I32, P,
                               I64, P, P, P], ctypes.c_int),
                "hpa_error_string": ([ctypes.c_int], ctypes.c_char_p),
                "hpa_last_cuda_error": ([], ctypes.c_int),
            }
            for name, (args, res) in sig.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        L = lib()
        msg = L.hpa_error_string(rc).decode()
        if rc == -5:
            msg += " (cudaError %d)" % L.hpa_last_cuda_error()
        raise HpaError("%s failed: %s (%d)" % (what, msg, rc))


def _stream(stream):
    """The stream's handle; a torch stream, a handle, or None for torch's current stream (read
    without the Stream object of torch.cuda.current_stream(), which takes longer than a launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return getattr(stream, "cuda_stream", stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dev(t, name, dtype=None):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
        raise HpaError("%s must be a contiguous CUDA tensor" % name)
    if dtype is not None and t.dtype is not dtype:
        raise HpaError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


# ----------------------------------------------------------------------------- sizes
def hpa_taskmap_bytes(B: int, num_ctas: int) -> int:
    return int(lib().hpa_taskmap_bytes(B, num_ctas))


def hpa_max_segments(B: int, num_ctas: int) -> int:
    return int(lib().hpa_max_segments(B, num_ctas))


def hpa_static_num_ctas(B: int, splits: int) -> int:
    return int(lib().hpa_static_num_ctas(B, splits))


def hpa_static_taskmap_bytes(B: int, splits: int) -> int:
    return int(lib().hpa_static_taskmap_bytes(B, splits))


def hpa_default_num_ctas(Hkv: int, q_len: int, kv_dtype: int, Hq: int = 64) -> int:
    c = int(lib().hpa_default_num_ctas(Hq, Hkv, q_len, kv_dtype))
    if c <= 0:
        raise HpaError("hpa_default_num_ctas failed (cudaError %d)" % lib().hpa_last_cuda_error())
    return c


def hpa_default_num_ctas_mma(Hkv: int, q_len: int, kv_dtype: int, Hq: int = 64) -> int:
    c = int(lib().hpa_default_num_ctas_mma(Hq, Hkv, q_len, kv_dtype))
    if c <= 0:
        raise HpaError("hpa_default_num_ctas_mma failed (cudaError %d)" %
                       lib().hpa_last_cuda_error())
    return c


def hpa_default_num_ctas_tc(Hkv: int, q_len: int, kv_dtype: int, Hq: int = 64) -> int:
    c = int(lib().hpa_default_num_ctas_tc(Hq, Hkv, q_len, kv_dtype))
    if c <= 0:
        raise HpaError("hpa_default_num_ctas_tc failed (cudaError %d)" %
                       lib().hpa_last_cuda_error())
    return c


def hpa_default_num_ctas_allheads(Hkv: int, q_len: int, kv_dtype: int, Hq: int = 64) -> int:
    c = int(lib().hpa_default_num_ctas_allheads(Hq, Hkv, q_len, kv_dtype))
    if c <= 0:
        raise HpaError("hpa_default_num_ctas_allheads failed (cudaError %d)" %
                       lib().hpa_last_cuda_error())
    return c


def hpa_default_num_ctas_window(Hkv: int, q_len: int, kv_dtype: int, Hq: int = 64) -> int:
    c = int(lib().hpa_default_num_ctas_window(Hq, Hkv, q_len, kv_dtype))
    if c <= 0:
        raise HpaError("hpa_default_num_ctas_window failed (cudaError %d)" %
                       lib().hpa_last_cuda_error())
    return c


# ----------------------------------------------------------------------------- the three calls
def hpa_plan(seq_lens, tile: int, num_ctas: int, taskmap, stream=None):
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(taskmap, "taskmap")
    _check(lib().hpa_plan(_ptr(seq_lens), seq_lens.numel(), tile, num_ctas, _ptr(taskmap),
                          taskmap.numel() * taskmap.element_size(), _stream(stream)), "hpa_plan")


def hpa_plan_weighted(seq_lens, tile: int, num_ctas: int, taskmap, stream=None):
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(taskmap, "taskmap")
    _check(lib().hpa_plan_weighted(_ptr(seq_lens), seq_lens.numel(), tile, num_ctas,
                                   _ptr(taskmap), taskmap.numel() * taskmap.element_size(),
                                   _stream(stream)), "hpa_plan_weighted")


def hpa_plan_static(seq_lens, tile: int, splits: int, taskmap, stream=None):
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(taskmap, "taskmap")
    _check(lib().hpa_plan_static(_ptr(seq_lens), seq_lens.numel(), tile, splits, _ptr(taskmap),
                                 taskmap.numel() * taskmap.element_size(), _stream(stream)),
           "hpa_plan_static")


def hpa_plan_window(seq_lens, q_len: int, window: int, sinks: int, tile: int, num_ctas: int,
                    taskmap, stream=None):
    """The plan for hpa_decode_attn_window: token at position a sees key i <= a when
    i > a - window or i < sinks."""
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(taskmap, "taskmap")
    _one_device(seq_lens, taskmap)
    _check(lib().hpa_plan_window(_ptr(seq_lens), seq_lens.numel(), q_len, window, sinks, tile,
                                 num_ctas, _ptr(taskmap),
                                 taskmap.numel() * taskmap.element_size(), _stream(stream)),
           "hpa_plan_window")


def _attn_args(q, k_pool, v_pool, page_indptr, page_indices, taskmap, k_scale, v_scale):
    """Checks shared by every attention call; returns (kv, B, q_len, Hq, d, P, Hkv, page)."""
    _dev(q, "q", torch.bfloat16)
    _dev(k_pool, "k_pool")
    _dev(v_pool, "v_pool")
    if k_pool.dtype == torch.bfloat16:
        kv = KV_BF16
    elif k_pool.dtype in (torch.uint8, torch.float8_e4m3fn):
        kv = KV_E4M3
        _dev(k_scale, "k_scale", torch.float32)
        _dev(v_scale, "v_scale", torch.float32)
    else:
        raise HpaError("unsupported KV dtype %s" % k_pool.dtype)
    if v_pool.dtype != k_pool.dtype or v_pool.shape != k_pool.shape:
        raise HpaError("k_pool and v_pool must match")
    for t, n in ((page_indptr, "page_indptr"), (page_indices, "page_indices")):
        _dev(t, n, torch.int32)
    _dev(taskmap, "taskmap")
    if q.dim() != 4 or k_pool.dim() != 4:
        raise HpaError("q must be [B][q_len][Hq][d] and the pools [P][Hkv][page][d]")
    B, q_len, Hq, d = q.shape
    P, Hkv, page, d2 = k_pool.shape
    if d2 != d:
        raise HpaError("head dim mismatch")
    if page_indptr.numel() < B + 1:
        raise HpaError("page_indptr must have B + 1 = %d entries" % (B + 1))
    if kv == KV_E4M3 and (k_scale.numel() < Hkv or v_scale.numel() < Hkv):
        raise HpaError("k_scale / v_scale need one fp32 value per KV head")
    return kv, B, q_len, Hq, d, P, Hkv, page


def _partials(partial_o, partial_lse, B, num_ctas, q_len, Hq, d):
    _dev(partial_o, "partial_o", torch.float32)
    _dev(partial_lse, "partial_lse", torch.float32)
    need = (B + num_ctas - 1) * q_len * Hq
    if partial_lse.numel() < need or partial_o.numel() < need * d:
        raise HpaError("partial buffers too small: need (B + num_ctas - 1) segments")


def _outputs(out, out_lse, B, q_len, Hq, d):
    _dev(out, "out", torch.bfloat16)
    if out.shape != (B, q_len, Hq, d):
        raise HpaError("out must have q's shape %s, got %s" % ((B, q_len, Hq, d),
                                                               tuple(out.shape)))
    if out_lse is not None:
        _dev(out_lse, "out_lse", torch.float32)
        if out_lse.shape != (B, q_len, Hq):
            raise HpaError("out_lse must have shape %s" % ((B, q_len, Hq),))


def hpa_decode_attn(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas: int,
                    partial_o, partial_lse, k_scale=None, v_scale=None,
                    sm_scale: float | None = None, stream=None, tc: bool = False,
                    mma: bool = False, window: bool = False):
    """q bf16 [B][q_len][Hq][d]; k/v pools bf16 or uint8 (E4M3) [P][Hkv][page][d].

    hpa_decode_attn picks the kernel by query rows per KV head (mma.sync up to 16,
    tcgen05 above); tc=True calls hpa_decode_attn_tc, mma=True hpa_decode_attn_mma and
    window=True hpa_decode_attn_window with the same arguments."""
    args = _attn_args(q, k_pool, v_pool, page_indptr, page_indices, taskmap, k_scale, v_scale)
    _, B, q_len, Hq, d, _, _, _ = args
    _partials(partial_o, partial_lse, B, num_ctas, q_len, Hq, d)
    _attn_call(args, q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas, partial_o,
               partial_lse, k_scale, v_scale, sm_scale, _stream(stream), tc, mma, window)


def _attn_call(args, q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas, partial_o,
               partial_lse, k_scale, v_scale, sm_scale, stream, tc, mma, window):
    """The attention call of the kernel asked for, on checked arguments."""
    kv, B, q_len, Hq, d, P, Hkv, page = args
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    name = ("hpa_decode_attn_tc" if tc else "hpa_decode_attn_mma" if mma else
            "hpa_decode_attn_window" if window else "hpa_decode_attn")
    rc = getattr(lib(), name)(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), kv, _ptr(k_scale), _ptr(v_scale), P,
        _ptr(page_indptr), _ptr(page_indices), page, B, q_len, Hq, Hkv, d, sm_scale,
        _ptr(taskmap), num_ctas, _ptr(partial_o), _ptr(partial_lse), stream)
    if rc != 0:
        _check(rc, name)


def hpa_decode_attn_mma(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas: int,
                        partial_o, partial_lse, k_scale=None, v_scale=None,
                        sm_scale: float | None = None, stream=None):
    """hpa_decode_attn computed by the mma.sync kernel at any query-row count."""
    hpa_decode_attn(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas, partial_o,
                    partial_lse, k_scale, v_scale, sm_scale, stream, mma=True)


def hpa_decode_attn_tc(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas: int,
                       partial_o, partial_lse, k_scale=None, v_scale=None,
                       sm_scale: float | None = None, stream=None):
    """hpa_decode_attn computed on the tcgen05 tensor cores (one pass for up to 64 rows)."""
    hpa_decode_attn(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas, partial_o,
                    partial_lse, k_scale, v_scale, sm_scale, stream, tc=True)


def hpa_decode_attn_window(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas: int,
                           partial_o, partial_lse, k_scale=None, v_scale=None,
                           sm_scale: float | None = None, stream=None):
    """hpa_decode_attn over a map of hpa_plan_window (sliding window and sink tokens)."""
    _one_device(q, k_pool, v_pool, page_indptr, page_indices, taskmap, partial_o, partial_lse,
                k_scale, v_scale)
    hpa_decode_attn(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas, partial_o,
                    partial_lse, k_scale, v_scale, sm_scale, stream, window=True)


def hpa_decode_attn_allheads(q, k_pool, v_pool, page_indptr, page_indices, taskmap,
                             num_ctas: int, partial_o, partial_lse, k_scale=None, v_scale=None,
                             sm_scale: float | None = None, trace=None, stream=None):
    """hpa_decode_attn with every KV head walked inside the CTA of a partition (grid over
    partitions only); num_ctas counts partitions of the whole grid.  trace: optional int64
    [4 * num_ctas * row groups] per-CTA timestamps."""
    kv, B, q_len, Hq, d, P, Hkv, page = _attn_args(q, k_pool, v_pool, page_indptr,
                                                   page_indices, taskmap, k_scale, v_scale)
    _partials(partial_o, partial_lse, B, num_ctas, q_len, Hq, d)
    if trace is not None:
        _dev(trace, "trace", torch.int64)
        if trace.numel() < 4 * num_ctas * ((Hq // Hkv * q_len + 15) // 16):
            raise HpaError("trace buffer too small")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    _check(lib().hpa_decode_attn_allheads(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), kv, _ptr(k_scale), _ptr(v_scale), P,
        _ptr(page_indptr), _ptr(page_indices), page, B, q_len, Hq, Hkv, d, float(sm_scale),
        _ptr(taskmap), num_ctas, _ptr(partial_o), _ptr(partial_lse), _ptr(trace),
        _stream(stream)), "hpa_decode_attn_allheads")


def hpa_decode_attn_traced(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas: int,
                           partial_o, partial_lse, trace, k_scale=None, v_scale=None,
                           sm_scale: float | None = None, stream=None):
    """hpa_decode_attn plus per-CTA timestamps: trace is int64 [num_ctas * Hkv * 4] on device."""
    kv, B, q_len, Hq, d, P, Hkv, page = _attn_args(q, k_pool, v_pool, page_indptr,
                                                   page_indices, taskmap, k_scale, v_scale)
    _partials(partial_o, partial_lse, B, num_ctas, q_len, Hq, d)
    _dev(trace, "trace", torch.int64)
    groups = (Hq // Hkv * q_len + 15) // 16
    if trace.numel() < 4 * num_ctas * Hkv * groups:
        raise HpaError("trace buffer too small")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    _check(lib().hpa_decode_attn_traced(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), kv, _ptr(k_scale), _ptr(v_scale), P,
        _ptr(page_indptr), _ptr(page_indices), page, B, q_len, Hq, Hkv, d, float(sm_scale),
        _ptr(taskmap), num_ctas, _ptr(partial_o), _ptr(partial_lse), _ptr(trace),
        _stream(stream)), "hpa_decode_attn_traced")


def trace_summary(trace, num_ctas: int, Hkv: int, groups: int = 1) -> dict:
    """SM busy and tail figures from a hpa_decode_attn_traced buffer (host-side arithmetic)."""
    import numpy as np
    t = trace.view(-1, 4).cpu().numpy().astype(np.int64)[:num_ctas * Hkv * groups]
    entry, go, end, info = t[:, 0], t[:, 1], t[:, 2], t[:, 3]
    sm = info & 0xffffffff
    busy = t[(info >> 32) > 0]
    t0 = int(entry.min())
    span = int(end.max()) - t0
    ends = np.sort(busy[:, 2]) if len(busy) else np.sort(end)
    per_sm = {}
    for s_, a, b_ in zip(sm, go, end):
        per_sm.setdefault(int(s_), []).append((int(a), int(b_)))
    occ = []
    for iv in per_sm.values():
        iv.sort()
        tot, cur_a, cur_b = 0, iv[0][0], iv[0][1]
        for a, b_ in iv[1:]:
            if a > cur_b:
                tot += cur_b - cur_a
                cur_a, cur_b = a, b_
            else:
                cur_b = max(cur_b, b_)
        occ.append(tot + cur_b - cur_a)
    return {"span_us": span / 1e3,
            "first_go_us": (int(go.min()) - t0) / 1e3,
            "median_cta_end_us": (float(np.median(ends)) - t0) / 1e3,
            "last_cta_tail_us": (float(ends[-1]) - float(np.median(ends))) / 1e3,
            "sm_busy_frac": float(np.mean(occ)) / span if span > 0 else 0.0,
            "sms_used": len(per_sm)}


def hpa_arrivals_elems(B: int, Hq: int, Hkv: int, q_len: int) -> int:
    return int(lib().hpa_arrivals_elems(B, Hq, Hkv, q_len))


def hpa_decode_attn_fused(q, k_pool, v_pool, page_indptr, page_indices, taskmap, num_ctas: int,
                          partial_o, partial_lse, out, arrivals, out_lse=None, k_scale=None,
                          v_scale=None, sm_scale: float | None = None, stream=None):
    """Attention with the combine folded in; arrivals: int32, hpa_arrivals_elems(B, Hq, Hkv,
    q_len) elements, zero between calls."""
    kv, B, q_len, Hq, d, P, Hkv, page = _attn_args(q, k_pool, v_pool, page_indptr,
                                                   page_indices, taskmap, k_scale, v_scale)
    _partials(partial_o, partial_lse, B, num_ctas, q_len, Hq, d)
    _outputs(out, out_lse, B, q_len, Hq, d)
    _dev(arrivals, "arrivals", torch.int32)
    if arrivals.numel() < hpa_arrivals_elems(B, Hq, Hkv, q_len):
        raise HpaError("arrivals has the wrong size")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    _check(lib().hpa_decode_attn_fused(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), kv, _ptr(k_scale), _ptr(v_scale), P,
        _ptr(page_indptr), _ptr(page_indices), page, B, q_len, Hq, Hkv, d, float(sm_scale),
        _ptr(taskmap), num_ctas, _ptr(partial_o), _ptr(partial_lse), _ptr(out), _ptr(out_lse),
        _ptr(arrivals), _stream(stream)), "hpa_decode_attn_fused")


def hpa_combine(partial_o, partial_lse, taskmap, num_ctas: int, out, out_lse=None, stream=None):
    """out bf16 [B][q_len][Hq][d]; out_lse fp32 [B][q_len][Hq] or None."""
    _dev(partial_o, "partial_o", torch.float32)
    _dev(partial_lse, "partial_lse", torch.float32)
    _dev(taskmap, "taskmap")
    _dev(out, "out", torch.bfloat16)
    if out.dim() != 4:
        raise HpaError("out must be [B][q_len][Hq][d]")
    B, q_len, Hq, d = out.shape
    _outputs(out, out_lse, B, q_len, Hq, d)
    _partials(partial_o, partial_lse, B, num_ctas, q_len, Hq, d)
    _combine_call(partial_o, partial_lse, taskmap, num_ctas, out, out_lse, B, q_len, Hq, d,
                  _stream(stream))


def _combine_call(partial_o, partial_lse, taskmap, num_ctas, out, out_lse, B, q_len, Hq, d,
                  stream):
    """hpa_combine on checked arguments."""
    rc = lib().hpa_combine(_ptr(partial_o), _ptr(partial_lse), _ptr(taskmap), B, num_ctas, q_len,
                           Hq, d, _ptr(out), _ptr(out_lse), stream)
    if rc != 0:
        _check(rc, "hpa_combine")


def hpa_selftest_wait_timeout(status, limit_ns: int, stream=None):
    """Run the bounded-wait diagnostic; status: int32 CUDA tensor of >= 1 element."""
    _dev(status, "status", torch.int32)
    _check(lib().hpa_selftest_wait_timeout(_ptr(status), int(limit_ns), _stream(stream)),
           "hpa_selftest_wait_timeout")


def hpa_decode_attn_combine_noalloc(q, k_pool, v_pool, page_indptr, page_indices, taskmap,
                                    num_ctas: int, out, out_lse=None, k_scale=None,
                                    v_scale=None, sm_scale: float | None = None, stream=None):
    """Attention + combine with the split partials in the library's fixed device array.

    For callers that cannot allocate device memory during a decode step (a
    plugin inside a runtime that owns the memory pool, a serving loop that
    must not call cudaMalloc/cudaFree).  Calls that overlap on the GPU share
    that array and race; serialise them.
    """
    kv, B, q_len, Hq, d, P, Hkv, page = _attn_args(q, k_pool, v_pool, page_indptr,
                                                   page_indices, taskmap, k_scale, v_scale)
    _outputs(out, out_lse, B, q_len, Hq, d)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    _check(lib().hpa_decode_attn_combine_noalloc(
        _ptr(q), _ptr(k_pool), _ptr(v_pool), kv, _ptr(k_scale), _ptr(v_scale), P,
        _ptr(page_indptr), _ptr(page_indices), page, B, q_len, Hq, Hkv, d, float(sm_scale),
        _ptr(taskmap), num_ctas, _ptr(out), _ptr(out_lse), _stream(stream)),
        "hpa_decode_attn_combine_noalloc")


def _store_kv(name, k_new, v_new, seq_lens, text_pos, page_indptr, page_indices, cos_sin, norm_w,
              k_pool, v_pool, eps, use_hadamard, k_scale, v_scale, status, stream):
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _dev(t, n, torch.bfloat16)
    _dev(cos_sin, "cos_sin", torch.float32)
    _dev(norm_w, "norm_w", torch.float32)
    for t, n in ((seq_lens, "seq_lens"), (page_indptr, "page_indptr"),
                 (page_indices, "page_indices")):
        _dev(t, n, torch.int32)
    kv, P, Hkv2, page, _ = _pools(k_pool, v_pool)
    if k_new.dim() != 4 or v_new.shape != k_new.shape:
        raise HpaError("k_new and v_new must match, [B][q_len][Hkv][d]")
    B, q_len, Hkv, d = k_new.shape
    if Hkv2 != Hkv or k_pool.shape[3] != d:
        raise HpaError("KV head count or head dim mismatch")
    if page_indptr.numel() < B + 1 or seq_lens.numel() < B:
        raise HpaError("page_indptr needs B + 1 = %d entries and seq_lens B" % (B + 1))
    if cos_sin.dim() < 2 or cos_sin.numel() < cos_sin.shape[0] * d or norm_w.numel() < d:
        raise HpaError("cos_sin must be [max_pos][d] and norm_w [d]")
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if kv == KV_E4M3 and _dev(t, n, torch.float32).numel() < Hkv:
            raise HpaError("%s needs one fp32 value per KV head" % n)
    if status is not None:
        _dev(status, "status", torch.int32)
    at = ()
    if name == "hpa_store_kv_at":
        _dev(text_pos, "text_pos", torch.int32)
        if text_pos.numel() != B or seq_lens.numel() != B:
            raise HpaError("text_pos and seq_lens need one value per request")
        _one_device(k_new, v_new, seq_lens, text_pos, page_indptr, page_indices, cos_sin, norm_w,
                    k_pool, v_pool, k_scale, v_scale, status)
        at = (_ptr(text_pos),)
    _check(getattr(lib(), name)(
        _ptr(k_new), _ptr(v_new), _ptr(seq_lens), *at, _ptr(page_indptr), _ptr(page_indices), P,
        page, _ptr(cos_sin), cos_sin.shape[0], _ptr(norm_w), float(eps), int(use_hadamard), kv,
        _ptr(k_scale), _ptr(v_scale), _ptr(k_pool), _ptr(v_pool), B, q_len, Hkv, d,
        _ptr(status), _stream(stream)), name)


def hpa_store_kv(k_new, v_new, seq_lens, page_indptr, page_indices, cos_sin, norm_w, k_pool,
                 v_pool, eps: float = 1e-6, use_hadamard: bool = True, k_scale=None,
                 v_scale=None, status=None, stream=None):
    """Fused RoPE + RMSNorm + Hadamard + quantise + paged store of the new tokens' K/V.

    k_new, v_new: bf16 [B][q_len][Hkv][d]; cos_sin: fp32 [max_pos][d]; norm_w: fp32 [d];
    pools: bf16 or uint8 (E4M3) [P][Hkv][page][d] (E4M3 needs k_scale / v_scale)."""
    _store_kv("hpa_store_kv", k_new, v_new, seq_lens, None, page_indptr, page_indices, cos_sin,
              norm_w, k_pool, v_pool, eps, use_hadamard, k_scale, v_scale, status, stream)


def hpa_store_kv_at(k_new, v_new, seq_lens, text_pos, page_indptr, page_indices, cos_sin, norm_w,
                    k_pool, v_pool, eps: float = 1e-6, use_hadamard: bool = True, k_scale=None,
                    v_scale=None, status=None, stream=None):
    """hpa_store_kv for a cache that evicts: seq_lens place the new tokens in the cache, and
    text_pos (int32 [B], the text position of each request's first new token) rotates them."""
    _store_kv("hpa_store_kv_at", k_new, v_new, seq_lens, text_pos, page_indptr, page_indices,
              cos_sin, norm_w, k_pool, v_pool, eps, use_hadamard, k_scale, v_scale, status, stream)


# ----------------------------------------------------------------------------- bounded cache
_n_devices = 0


def _one_device(*tensors):
    """The library launches on the current device: every tensor has to live there."""
    global _n_devices
    if not _n_devices:
        _n_devices = torch.cuda.device_count()
    if _n_devices == 1:
        return
    here = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise HpaError("tensors must be on the current device (cuda:%d), got %s" %
                           (here, t.device))


def _acc_pool(t, name, k_pool):
    _dev(t, name, torch.float32)
    if t.shape != k_pool.shape[:3]:
        raise HpaError("%s must have shape %s, one weight per cached key, got %s" %
                       (name, tuple(k_pool.shape[:3]), tuple(t.shape)))


def _page_table(indptr, indices, B, what="page"):
    _dev(indptr, what + "_indptr", torch.int32)
    _dev(indices, what + "_indices", torch.int32)
    if indptr.numel() != B + 1:
        raise HpaError("%s_indptr must have B + 1 = %d entries" % (what, B + 1))


def _dst_table(indptr, indices, B):
    if (indptr is None) != (indices is None):
        raise HpaError("dst_indptr and dst_indices go together")
    if indptr is not None:
        _page_table(indptr, indices, B, "dst")


def _pools(k_pool, v_pool):
    """(kv, P, Hkv, page, d) of the two pools of one cache."""
    _dev(k_pool, "k_pool")
    _dev(v_pool, "v_pool", k_pool.dtype)
    if k_pool.dim() != 4 or v_pool.shape != k_pool.shape:
        raise HpaError("k_pool and v_pool must match, [P][Hkv][page][d]")
    if k_pool.dtype not in (torch.bfloat16, torch.uint8, torch.float8_e4m3fn):
        raise HpaError("unsupported KV dtype %s" % k_pool.dtype)
    return (KV_BF16 if k_pool.dtype == torch.bfloat16 else KV_E4M3, *k_pool.shape)


def hpa_key_weights(q, lse, k_pool, page_indptr, page_indices, taskmap, num_ctas: int, acc,
                    out=None, k_scale=None, decay: float = 1.0, sm_scale: float | None = None,
                    stream=None):
    """Adds one attention step's weights to the accumulators of the cached keys.

    lse: the step's out_lse, fp32 [B][q_len][Hq]; acc: fp32 [P][Hkv][page], updated in
    place, or read only when `out` (same shape) is given, or None for zero (then `out` is
    required); taskmap: the map of the attention step (any plan, window maps included)."""
    _dev(q, "q", torch.bfloat16)
    if q.dim() != 4 or k_pool.dim() != 4:
        raise HpaError("q must be [B][q_len][Hq][d] and the pool [P][Hkv][page][d]")
    _dev(k_pool, "k_pool")
    B, q_len, Hq, d = q.shape
    P, Hkv, page, d2 = k_pool.shape
    if d2 != d:
        raise HpaError("head dim mismatch")
    if k_pool.dtype == torch.bfloat16:
        kv = KV_BF16
    elif k_pool.dtype in (torch.uint8, torch.float8_e4m3fn):
        kv = KV_E4M3
        _dev(k_scale, "k_scale", torch.float32)
        if k_scale.numel() < Hkv:
            raise HpaError("k_scale needs one fp32 value per KV head")
    else:
        raise HpaError("unsupported KV dtype %s" % k_pool.dtype)
    _dev(lse, "lse", torch.float32)
    if lse.shape != (B, q_len, Hq):
        raise HpaError("lse must have shape %s" % ((B, q_len, Hq),))
    out = acc if out is None else out
    for t, n in ((acc, "acc"), (out, "out")):
        if t is not None or n == "out":
            _acc_pool(t, n, k_pool)
    _page_table(page_indptr, page_indices, B)
    _dev(taskmap, "taskmap")
    # int32 words of the smallest map of this shape, a static one: num_ctas segment rows
    if taskmap.numel() * taskmap.element_size() < 4 * (((23 + 3 * B + 2 * num_ctas) & ~3) +
                                                       4 * num_ctas):
        raise HpaError("taskmap is too small for %d requests over %d partitions" % (B, num_ctas))
    _one_device(q, lse, k_pool, k_scale, acc, out, page_indptr, page_indices, taskmap)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(d)
    _check(lib().hpa_key_weights(
        _ptr(q), _ptr(lse), _ptr(k_pool), kv, _ptr(k_scale), P, _ptr(page_indptr),
        _ptr(page_indices), page, B, q_len, Hq, Hkv, d, float(sm_scale), float(decay),
        _ptr(taskmap), num_ctas, _ptr(acc), _ptr(out), _stream(stream)), "hpa_key_weights")


def _kept(kept, new_lens, B, Hkv):
    _dev(kept, "kept", torch.int32)
    _dev(new_lens, "new_lens", torch.int32)
    shape = kept.shape
    if len(shape) != 3 or shape[0] != B or shape[1] != Hkv or shape[2] < 1:
        raise HpaError("kept must be int32 [B][Hkv][at least the largest budget]")
    if new_lens.numel() != B:
        raise HpaError("new_lens needs one value per request")


def hpa_evict_select(acc, seq_lens, page_indptr, page_indices, budgets, sinks: int, recent: int,
                     kept, new_lens, status=None, stream=None):
    """The keys every KV head keeps, ascending, in kept [B][Hkv][stride] (int32), and how many
    in new_lens [B]: the first `sinks`, the last `recent` and the heaviest of the rest up to
    budgets[r], or all of a request within its budget."""
    _dev(acc, "acc", torch.float32)
    if acc.dim() != 3:
        raise HpaError("acc must be [P][Hkv][page]")
    P, Hkv, page = acc.shape
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(budgets, "budgets", torch.int32)
    B = seq_lens.numel()
    if budgets.numel() != B:
        raise HpaError("budgets needs one value per request")
    _page_table(page_indptr, page_indices, B)
    _kept(kept, new_lens, B, Hkv)
    if status is not None:
        _dev(status, "status", torch.int32)
    _one_device(acc, seq_lens, budgets, page_indptr, page_indices, kept, new_lens, status)
    _check(lib().hpa_evict_select(
        _ptr(acc), _ptr(seq_lens), _ptr(page_indptr), _ptr(page_indices), P, page, _ptr(budgets),
        sinks, recent, B, Hkv, _ptr(kept), kept.shape[2], _ptr(new_lens), _ptr(status),
        _stream(stream)), "hpa_evict_select")


def hpa_evict_compact(k_pool, v_pool, page_indptr, page_indices, kept, new_lens, acc=None,
                      dst_indptr=None, dst_indices=None, status=None, stream=None):
    """Moves the kept rows of K, V and acc to the front of each request's own pages, or to the
    pages that dst_indptr / dst_indices list (the old cache then stays as it was)."""
    kv, P, Hkv, page, d = _pools(k_pool, v_pool)
    B = page_indptr.numel() - 1
    _page_table(page_indptr, page_indices, B)
    _kept(kept, new_lens, B, Hkv)
    if acc is not None:
        _acc_pool(acc, "acc", k_pool)
    _dst_table(dst_indptr, dst_indices, B)
    if status is not None:
        _dev(status, "status", torch.int32)
    _one_device(k_pool, v_pool, page_indptr, page_indices, kept, new_lens, acc, dst_indptr,
                dst_indices, status)
    _check(lib().hpa_evict_compact(
        _ptr(k_pool), _ptr(v_pool), kv, _ptr(acc), P, _ptr(page_indptr), _ptr(page_indices),
        _ptr(dst_indptr), _ptr(dst_indices), page, _ptr(kept), kept.shape[2], _ptr(new_lens), B,
        Hkv, d, _ptr(status), _stream(stream)), "hpa_evict_compact")


def hpa_evict(acc, k_pool, v_pool, seq_lens, page_indptr, page_indices, budgets, sinks: int,
              recent: int, kept, new_lens, dst_indptr=None, dst_indices=None, status=None,
              stream=None):
    """hpa_evict_select, then hpa_evict_compact of K, V and acc; the cache then has new_lens[r]
    keys per request (-1: a request that `status` reports, for a bad destination list as well;
    nothing of it is moved)."""
    kv, P, Hkv, page, d = _pools(k_pool, v_pool)
    _acc_pool(acc, "acc", k_pool)
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(budgets, "budgets", torch.int32)
    B = seq_lens.numel()
    if budgets.numel() != B:
        raise HpaError("budgets needs one value per request")
    _page_table(page_indptr, page_indices, B)
    _dst_table(dst_indptr, dst_indices, B)
    _kept(kept, new_lens, B, Hkv)
    if status is not None:
        _dev(status, "status", torch.int32)
    _one_device(k_pool, v_pool, acc, seq_lens, budgets, page_indptr, page_indices, kept, new_lens,
                dst_indptr, dst_indices, status)
    _check(lib().hpa_evict(
        _ptr(k_pool), _ptr(v_pool), kv, _ptr(acc), P, _ptr(seq_lens), _ptr(page_indptr),
        _ptr(page_indices), _ptr(dst_indptr), _ptr(dst_indices), page, _ptr(budgets), sinks,
        recent, B, Hkv, d, _ptr(kept), kept.shape[2], _ptr(new_lens), _ptr(status),
        _stream(stream)), "hpa_evict")


# ----------------------------------------------------------------------------- workspace helper
class Workspace:
    """Device buffers for one decode step: task map and split partials.

    Sized once for (B, num_ctas, q_len, Hq, d) -- dynamic map by default, or
    the static comparator with `splits`.  Allocation is done with torch; the
    library itself never allocates.  num_ctas (partitions per KV head) is
    normally hpa_default_num_ctas(...), which follows hpa_decode_attn's kernel
    choice (mma.sync up to 16 query rows per KV head, tcgen05 above);
    hpa_default_num_ctas_mma / _tc size for a forced kernel.  Either kernel
    accepts any partition count.  With `window` (keys) and `sinks` the steps run
    sliding-window attention: hpa_plan_window and hpa_decode_attn_window, sized by
    hpa_default_num_ctas_window.
    """

    def __init__(self, B, q_len, Hq, d, num_ctas=None, splits=None, device="cuda", Hkv=8,
                 weighted=False, window=None, sinks=0):
        if window is not None and (splits is not None or weighted):
            raise HpaError("a window has the dynamic plan alone")
        if window is None and sinks:
            raise HpaError("sinks come with a window")
        if splits is not None:
            self.num_ctas = hpa_static_num_ctas(B, splits)
            nbytes = hpa_static_taskmap_bytes(B, splits)
        else:
            self.num_ctas = num_ctas
            nbytes = hpa_taskmap_bytes(B, num_ctas)
        cap = hpa_max_segments(B, self.num_ctas)   # partial rows, valid for either map
        if nbytes == 0 or cap == 0:
            raise HpaError("workspace size query failed")
        self.splits = splits
        self.weighted = weighted
        self.window, self.sinks, self.q_len = window, sinks, q_len
        self.capacity = cap
        self.taskmap = torch.zeros((nbytes + 3) // 4, dtype=torch.int32, device=device)
        self.partial_o = torch.empty(cap * q_len * Hq * d, dtype=torch.float32, device=device)
        self.partial_lse = torch.empty(cap * q_len * Hq, dtype=torch.float32, device=device)
        self.arrivals = torch.zeros(hpa_arrivals_elems(B, Hq, Hkv, q_len), dtype=torch.int32,
                                    device=device)  # fused combine

    def plan(self, seq_lens, tile=None, stream=None):
        """tile: keys per tile, by default 512, or one page of 64 with a window."""
        if tile is None:
            tile = 512 if self.window is None else 64
        if self.window is not None:
            hpa_plan_window(seq_lens, self.q_len, self.window, self.sinks, tile, self.num_ctas,
                            self.taskmap, stream)
        elif self.splits is not None:
            hpa_plan_static(seq_lens, tile, self.splits, self.taskmap, stream)
        elif self.weighted:
            hpa_plan_weighted(seq_lens, tile, self.num_ctas, self.taskmap, stream)
        else:
            hpa_plan(seq_lens, tile, self.num_ctas, self.taskmap, stream)

    def status(self) -> int:
        """Status word of the map (synchronises the current stream)."""
        return int(self.taskmap[6].item())


def decode_step(ws: Workspace, q, k_pool, v_pool, seq_lens, page_indptr, page_indices, out,
                out_lse=None, k_scale=None, v_scale=None, tile=None, plan=True, stream=None,
                fused=False, tc=False, sm_scale: float | None = None, allheads=False,
                mma=False, acc=None, decay: float = 1.0):
    """plan (optional) -> split-KV attention -> combine, all enqueued on one stream.

    fused=True runs the attention kernel with the combine folded in (one launch);
    The attention call is hpa_decode_attn, which picks its kernel by query rows per KV
    head (size the workspace with hpa_default_num_ctas); tc=True forces the tcgen05
    kernel (hpa_default_num_ctas_tc), mma=True the mma.sync kernel
    (hpa_default_num_ctas_mma), allheads=True the mma.sync variant with every KV head
    inside the CTA (hpa_default_num_ctas_allheads); sm_scale defaults to 1/sqrt(d).  A
    workspace with a window runs hpa_decode_attn_window (and none of the variants above).
    acc: accumulators of the cached keys ([P][Hkv][page] fp32), which the step's weights
    are added to in place after a decay (hpa_key_weights); needs out_lse."""
    if fused and tc:
        raise HpaError("the tcgen05 kernel has no fused-combine variant")
    if allheads and (fused or tc):
        raise HpaError("the all-heads variant has no fused or tcgen05 form")
    if ws.window is not None and (fused or tc or allheads or mma):
        raise HpaError("a window has one attention kernel")
    if acc is not None and out_lse is None:
        raise HpaError("accumulating key weights needs out_lse")
    if acc is not None and allheads:
        raise HpaError("hpa_key_weights needs a map per KV head, which the all-heads one is not")
    stream = _stream(stream)
    if plan:
        ws.plan(seq_lens, tile, stream)
    if fused:
        hpa_decode_attn_fused(q, k_pool, v_pool, page_indptr, page_indices, ws.taskmap,
                              ws.num_ctas, ws.partial_o, ws.partial_lse, out, ws.arrivals,
                              out_lse, k_scale, v_scale, sm_scale=sm_scale, stream=stream)
    elif allheads:
        hpa_decode_attn_allheads(q, k_pool, v_pool, page_indptr, page_indices, ws.taskmap,
                                 ws.num_ctas, ws.partial_o, ws.partial_lse, k_scale, v_scale,
                                 sm_scale=sm_scale, stream=stream)
        hpa_combine(ws.partial_o, ws.partial_lse, ws.taskmap, ws.num_ctas, out, out_lse, stream)
    else:  # both calls after one round of checks
        if ws.window is not None:
            _one_device(q, k_pool, v_pool, seq_lens, page_indptr, page_indices, out, out_lse,
                        k_scale, v_scale, ws.taskmap)
        args = _attn_args(q, k_pool, v_pool, page_indptr, page_indices, ws.taskmap, k_scale,
                          v_scale)
        _, B, q_len, Hq, d, _, _, _ = args
        _partials(ws.partial_o, ws.partial_lse, B, ws.num_ctas, q_len, Hq, d)
        _outputs(out, out_lse, B, q_len, Hq, d)
        _attn_call(args, q, k_pool, v_pool, page_indptr, page_indices, ws.taskmap, ws.num_ctas,
                   ws.partial_o, ws.partial_lse, k_scale, v_scale, sm_scale, stream, tc, mma,
                   ws.window is not None)
        _combine_call(ws.partial_o, ws.partial_lse, ws.taskmap, ws.num_ctas, out, out_lse, B,
                      q_len, Hq, d, stream)
    if acc is not None:
        hpa_key_weights(q, out_lse, k_pool, page_indptr, page_indices, ws.taskmap, ws.num_ctas,
                        acc, k_scale=k_scale, decay=decay, sm_scale=sm_scale, stream=stream)


def evict_step(acc, k_pool, v_pool, seq_lens, page_indptr, page_indices, budgets, sinks: int,
               recent: int, kept, new_lens, dst_indptr=None, dst_indices=None, status=None,
               stream=None):
    """What follows a decode_step once caches have outgrown their budgets: selection and the
    move of K, V and the accumulated weights, enqueued on one stream (hpa_evict)."""
    hpa_evict(acc, k_pool, v_pool, seq_lens, page_indptr, page_indices, budgets, sinks, recent,
              kept, new_lens, dst_indptr, dst_indices, status, stream)
