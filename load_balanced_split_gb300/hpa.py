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

KV_BF16, KV_E4M3, KV_E2M1 = 0, 1, 2
E2M1_PAGE_BYTES = 4608   # one page and KV head of a 4-bit pool: 64 x 64 of codes, 64 x 8 scales
STATUS_BITS = {1: "BAD_SEQLEN", 2: "MISMATCH", 4: "BAD_PAGE", 8: "TIMEOUT", 16: "OVERFLOW",
               32: "BAD_MAP", 64: "BAD_BUDGET", 128: "NO_PAGES"}
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
                "hpa_store_qkv": ([P, I64, P, I64, P, I64, I32, I32, I32, I32, P, P, P, I32, I32,
                                   P, P, F, I32, P, I64, I32, P, P, P, P, I64, I32, P, P],
                                  ctypes.c_int),
                "hpa_assign_pages_workspace": ([I32, I32], SZ),
                "hpa_assign_pages": ([P, P, P, P, I32, I32, P, I32, P, P, P, P, P, I32, I32, P, P,
                                      I32, P, P, I32, P, SZ, P, P], ctypes.c_int),
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


def _devs(dtype, names, tensors):
    """_dev for several tensors of one type (None is passed over), at less host time each."""
    try:
        for t in tensors:
            if t is not None and not (t.is_cuda and t.dtype is dtype and t.is_contiguous()):
                break
        else:
            return
    except AttributeError:
        pass
    for t, name in zip(tensors, names.split()):
        if t is not None:
            _dev(t, name, dtype)


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


def _is_e2m1(pool):
    """Whether a pool is one of 4-bit pages, uint8 [P][Hkv][E2M1_PAGE_BYTES]."""
    return pool.dim() == 3 and pool.dtype is torch.uint8 and pool.shape[2] == E2M1_PAGE_BYTES


def _attn_args(q, k_pool, v_pool, page_indptr, page_indices, taskmap, k_scale, v_scale):
    """Checks shared by every attention call; returns (kv, B, q_len, Hq, d, P, Hkv, page)."""
    _dev(q, "q", torch.bfloat16)
    _dev(k_pool, "k_pool")
    _dev(v_pool, "v_pool")
    e2m1 = _is_e2m1(k_pool)
    if k_pool.dtype == torch.bfloat16:
        kv = KV_BF16
    elif k_pool.dtype in (torch.uint8, torch.float8_e4m3fn):
        kv = KV_E2M1 if e2m1 else KV_E4M3
        _dev(k_scale, "k_scale", torch.float32)
        _dev(v_scale, "v_scale", torch.float32)
    else:
        raise HpaError("unsupported KV dtype %s" % k_pool.dtype)
    if v_pool.dtype != k_pool.dtype or v_pool.shape != k_pool.shape:
        raise HpaError("k_pool and v_pool must match")
    for t, n in ((page_indptr, "page_indptr"), (page_indices, "page_indices")):
        _dev(t, n, torch.int32)
    _dev(taskmap, "taskmap")
    if q.dim() != 4 or (k_pool.dim() != 4 and not e2m1):
        raise HpaError("q must be [B][q_len][Hq][d] and the pools [P][Hkv][page][d] "
                       "(4-bit pools: uint8 [P][Hkv][%d])" % E2M1_PAGE_BYTES)
    B, q_len, Hq, d = q.shape
    P, Hkv, page, d2 = (*k_pool.shape[:2], 64, 128) if e2m1 else k_pool.shape
    if d2 != d:
        raise HpaError("head dim mismatch")
    if page_indptr.numel() < B + 1:
        raise HpaError("page_indptr must have B + 1 = %d entries" % (B + 1))
    if e2m1:
        _one_device(q, k_pool, v_pool, page_indptr, page_indices, taskmap, k_scale, v_scale)
    if kv != KV_BF16 and (k_scale.numel() < Hkv or v_scale.numel() < Hkv):
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
    """q bf16 [B][q_len][Hq][d]; k/v pools bf16 or uint8 (E4M3) [P][Hkv][page][d], or 4-bit
    (E2M1 with block scales) uint8 [P][Hkv][E2M1_PAGE_BYTES].

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


def _heads(t, name, n):
    """Checks a bf16 [n][heads][128] tensor whose tokens may lie apart; (heads, token stride)."""
    try:
        if t.is_cuda and t.dtype is torch.bfloat16:
            tokens, heads, d = t.shape
            s0, s1, s2 = t.stride()
            if tokens == n and d == 128 and s2 == 1 and s1 == 128 and s0 >= heads * 128:
                if s0 % 8 == 0 or n <= 1:
                    return heads, s0 if n > 1 else heads * 128
    except (AttributeError, ValueError):
        pass
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise HpaError("%s must be a CUDA tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise HpaError("%s must be %s, got %s" % (name, torch.bfloat16, t.dtype))
    if t.dim() != 3 or t.shape[0] != n or t.shape[2] != 128:
        raise HpaError("%s must be [%d tokens][heads][128], got %s" % (name, n, tuple(t.shape)))
    heads, st = t.shape[1], t.stride()
    if n and heads and (st[2] != 1 or (heads > 1 and st[1] != 128) or
                        (n > 1 and (st[0] < heads * 128 or st[0] % 8))):
        raise HpaError("%s: a token's heads must be contiguous, tokens a multiple of 8 elements "
                       "apart, got strides %s" % (name, st))
    return heads, st[0] if n > 1 else heads * 128


def hpa_store_qkv(q, k, v, positions, slots, cos_sin, k_pool=None, v_pool=None, q_out=None,
                  q_norm=None, k_norm=None, eps: float = 1e-6, norm_after: bool = False,
                  interleaved: bool = False, use_hadamard: bool = False, k_scale=None,
                  v_scale=None, status=None, stream=None, num_pages=None):
    """Per-head RMSNorm, rotation, optional Hadamard transform and paged store of tokens'
    projections, and their queries, in one pass.

    q bf16 [n][Hq][128] (or None), k and v [n][Hkv][128] (or both None): tokens may be strided,
    as the parts of a packed projection are; positions int32 [n], slots int64 [n] (-1: no token),
    as hpa_assign_pages writes them; cos_sin fp32 [max_pos][rot_dim] (None: no rotation).  q_out:
    like q, by default q itself (in place).  Pools bf16 or uint8 (E4M3) [P][Hkv][64][128] or 4-bit
    uint8 [P][Hkv][E2M1_PAGE_BYTES]; without them num_pages bounds the slots."""
    if q is None and k is None:
        raise HpaError("neither queries nor keys and values")
    if (k is None) != (v is None):
        raise HpaError("k and v go together")
    _dev(slots, "slots", torch.int64)
    _dev(positions, "positions", torch.int32)
    _devs(torch.float32, "cos_sin q_norm k_norm k_scale v_scale",
          (cos_sin, q_norm, k_norm, k_scale, v_scale))
    n = positions.numel()
    if slots.numel() != n:
        raise HpaError("positions and slots need one value per token")
    Hq = Hkv = kv = 0
    sq = sk = sv = so = 0
    if q is not None:
        Hq, sq = _heads(q, "q", n)
        q_out = q if q_out is None else q_out
        heads, so = _heads(q_out, "q_out", n)
        if heads != Hq:
            raise HpaError("q_out must have q's shape")
    if k is not None:
        Hkv, sk = _heads(k, "k", n)
        heads, sv = _heads(v, "v", n)
        if heads != Hkv:
            raise HpaError("k and v must have the same heads")
        if k_pool is None or v_pool is None:
            raise HpaError("k and v need their pools")
        if _is_e2m1(k_pool):
            kv, num_pages = KV_E2M1, k_pool.shape[0]
            _dev(k_pool, "k_pool")
            _dev(v_pool, "v_pool", torch.uint8)
            if v_pool.shape != k_pool.shape:
                raise HpaError("k_pool and v_pool must match")
            if k_pool.shape[1] != Hkv:
                raise HpaError("KV head count mismatch")
        else:
            kv, num_pages, heads, page, d = _pools(k_pool, v_pool)
            if heads != Hkv or page != 64 or d != 128:
                raise HpaError("the pools must be [P][%d][64][128]" % Hkv)
        if kv != KV_BF16:
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if (t if t is not None else _dev(t, name)).numel() < Hkv:
                    raise HpaError("%s needs one fp32 value per KV head" % name)
    elif num_pages is None:
        raise HpaError("without pools num_pages has to say how many there are")
    rot = max_pos = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise HpaError("cos_sin must be [max_pos][rot_dim]")
        max_pos, rot = cos_sin.shape
        if rot == 0:
            raise HpaError("cos_sin must be [max_pos][rot_dim] (None: no rotation)")
    if ((q_norm is not None and q_norm.numel() != 128) or
            (k_norm is not None and k_norm.numel() != 128)):
        raise HpaError("q_norm and k_norm must be [128]")
    if status is not None:
        _dev(status, "status", torch.int32)
    _one_device(q, k, v, positions, slots, cos_sin, k_pool, v_pool, q_out, q_norm, k_norm, k_scale,
                v_scale, status)
    if n == 0:                    # tensors without elements have no address to pass on
        return
    flags = (1 if norm_after else 0) + (2 if interleaved else 0) + (4 if use_hadamard else 0)
    rc = lib().hpa_store_qkv(
        _ptr(q), sq, _ptr(k), sk, _ptr(v), sv, n, Hq, Hkv, 128, _ptr(positions), _ptr(slots),
        _ptr(cos_sin), max_pos, rot, _ptr(q_norm), _ptr(k_norm), eps, flags, _ptr(q_out), so, kv,
        _ptr(k_scale), _ptr(v_scale), _ptr(k_pool), _ptr(v_pool), num_pages, 64, _ptr(status),
        _stream(stream))
    if rc != 0:
        _check(rc, "hpa_store_qkv")


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


# ----------------------------------------------------------------------------- page tables
def hpa_assign_pages_workspace(B: int, num_rows: int) -> int:
    return int(lib().hpa_assign_pages_workspace(B, num_rows))


def hpa_assign_pages(seq_lens, new_tokens, table, held, free_pages, free_count, page_indptr,
                     page_indices, slots, positions, workspace, rows=None, pos_offset=None,
                     held_out=None, free_count_out=None, status=None, stream=None):
    """One step of a paged cache's tables, on the device: the pages that seq_lens (int32 [B], 0
    for an ended session) ask for are taken from the free stack or given back, and the batch's
    page_indptr [B+1] and page_indices and the slots (int64) and positions (int32) of its
    new_tokens (int32 [B], or None with slots and positions None) are written.

    State: table int32 [num_rows][max pages], held int32 [num_rows], free_pages int32
    [num_pages], free_count int32 [1]; updated in place, or held and free_count into held_out and
    free_count_out.  rows (int32 [B]): the table row of each request, by default 0 .. B - 1."""
    held_out = held if held_out is None else held_out
    free_count_out = free_count if free_count_out is None else free_count_out
    for t, name in ((seq_lens, "seq_lens"), (table, "table"), (held, "held"),
                    (free_pages, "free_pages"), (free_count, "free_count"),
                    (page_indptr, "page_indptr"), (page_indices, "page_indices")):
        if t is None:
            raise HpaError("%s must be a contiguous CUDA tensor" % name)
    _devs(torch.int32, "seq_lens table held held_out free_pages free_count free_count_out "
          "page_indptr page_indices new_tokens positions rows pos_offset status",
          (seq_lens, table, held, held_out, free_pages, free_count, free_count_out, page_indptr,
           page_indices, new_tokens, positions, rows, pos_offset, status))
    _dev(workspace, "workspace")
    B = seq_lens.numel()
    if table.dim() != 2:
        raise HpaError("table must be int32 [num_rows][max pages]")
    num_rows, stride = table.shape
    if held.numel() != num_rows or held_out.numel() != num_rows:
        raise HpaError("held and held_out need one count for each of %d rows" % num_rows)
    if free_count.numel() != 1 or free_count_out.numel() != 1:
        raise HpaError("free_count and free_count_out are one number each")
    if page_indptr.numel() != B + 1:
        raise HpaError("page_indptr must have B + 1 = %d entries" % (B + 1))
    if rows is None:
        if B > num_rows:
            raise HpaError("%d requests without rows in a table of %d rows" % (B, num_rows))
    elif rows.numel() != B:
        raise HpaError("rows needs one value per request")
    if pos_offset is not None and pos_offset.numel() != B:
        raise HpaError("pos_offset needs one value per request")
    tokens = 0
    if new_tokens is not None and slots is not None and positions is not None:
        _dev(slots, "slots", torch.int64)
        tokens = slots.numel()
        if new_tokens.numel() != B or positions.numel() != tokens:
            raise HpaError("new_tokens needs one value per request, positions one per slot")
    elif not (new_tokens is None and slots is None and positions is None):
        raise HpaError("new_tokens, slots and positions go together")
    _one_device(seq_lens, new_tokens, table, held, held_out, free_pages, free_count,
                free_count_out, page_indptr, page_indices, slots, positions, workspace, rows,
                pos_offset, status)
    rc = lib().hpa_assign_pages(
        seq_lens.data_ptr(), _ptr(new_tokens), _ptr(rows), _ptr(pos_offset), B, num_rows,
        table.data_ptr(), stride, held.data_ptr(), held_out.data_ptr(), free_pages.data_ptr(),
        free_count.data_ptr(), free_count_out.data_ptr(), free_pages.numel(), 64,
        page_indptr.data_ptr(), page_indices.data_ptr(), page_indices.numel(), _ptr(slots),
        _ptr(positions), tokens, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream))
    if rc != 0:
        _check(rc, "hpa_assign_pages")


class PageTable:
    """The page tables of a pool of num_pages pages and what hpa_assign_pages writes for a step.

    num_rows sessions of up to max_pages pages each; steps of up to max_batch requests and
    max_tokens new tokens.  After assign(...), page_indptr and page_indices are the batch's lists,
    and slots and positions hold its new tokens (slot -1 behind the last); `status` gathers the
    bits of steps that could not serve a request (HPA_STATUS_NO_PAGES and others)."""

    def __init__(self, num_pages, num_rows, max_pages, max_batch=None, max_tokens=None,
                 device="cuda"):
        max_batch = num_rows if max_batch is None else max_batch
        max_tokens = max_batch if max_tokens is None else max_tokens

        def i32(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=device)
        nbytes = hpa_assign_pages_workspace(max_batch, num_rows)
        if nbytes == 0 or num_pages < 1 or max_pages < 1 or max_tokens < 0:
            raise HpaError("page table sizes out of range")
        self.table, self.held = i32(num_rows, max_pages), i32(num_rows)
        # page 0 on top
        self.free_pages = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.free_count = i32(1) + num_pages
        self._indptr = i32(max_batch + 1)
        self.page_indptr, self.page_indices = self._indptr, i32(num_pages)
        self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=device)
        self.positions = i32(max_tokens)
        self.workspace = i32((nbytes + 3) // 4)
        self.status = i32(1)

    def assign(self, seq_lens, new_tokens=None, rows=None, pos_offset=None, stream=None):
        B = seq_lens.numel()
        if B + 1 > self._indptr.numel():
            raise HpaError("a batch of %d requests, and room for %d"
                           % (B, self._indptr.numel() - 1))
        self.page_indptr = self._indptr[:B + 1]
        slots, positions = (None, None) if new_tokens is None else (self.slots, self.positions)
        hpa_assign_pages(seq_lens, new_tokens, self.table, self.held, self.free_pages,
                         self.free_count, self.page_indptr, self.page_indices, slots, positions,
                         self.workspace, rows=rows, pos_offset=pos_offset, status=self.status,
                         stream=stream)


# ----------------------------------------------------------------------------- workspace helper
def _default_tile(window, e2m1):
    """Keys per tile of a plan: 256 of 4-bit pages give small batches more to share out (one
    request of 900 keys 12.8 -> 11.6 us, of 100000 33.9 -> 32.5) and change large ones little."""
    return 64 if window is not None else 256 if e2m1 else 512


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
    hpa_default_num_ctas_window.  kv_dtype: the cache's type, where it is KV_E2M1; plan then
    takes as many keys a tile as decode_step does for 4-bit pages, so that a map planned once
    for many layers is the one that each of them would plan.
    """

    def __init__(self, B, q_len, Hq, d, num_ctas=None, splits=None, device="cuda", Hkv=8,
                 weighted=False, window=None, sinks=0, kv_dtype=None):
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
        self.kv_dtype = kv_dtype
        self.window, self.sinks, self.q_len = window, sinks, q_len
        self.capacity = cap
        self.taskmap = torch.zeros((nbytes + 3) // 4, dtype=torch.int32, device=device)
        self.partial_o = torch.empty(cap * q_len * Hq * d, dtype=torch.float32, device=device)
        self.partial_lse = torch.empty(cap * q_len * Hq, dtype=torch.float32, device=device)
        self.arrivals = torch.zeros(hpa_arrivals_elems(B, Hq, Hkv, q_len), dtype=torch.int32,
                                    device=device)  # fused combine

    def plan(self, seq_lens, tile=None, stream=None):
        """tile: keys per tile, by default 512 (256 of 4-bit pages), or one page of 64 with a
        window."""
        if tile is None:
            tile = _default_tile(self.window, self.kv_dtype == KV_E2M1)
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
    if acc is not None and _is_e2m1(k_pool):
        raise HpaError("hpa_key_weights has no 4-bit form")
    stream = _stream(stream)
    if plan:
        if tile is None:
            tile = _default_tile(ws.window, ws.kv_dtype == KV_E2M1 or _is_e2m1(k_pool))
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
