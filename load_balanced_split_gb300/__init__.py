"""Load-balanced split-KV GQA decode attention for GB300 (sm_103a).

The compute path is the C-ABI library libhpa (include/hpa.h, sources in
csrc/); `hpa` is its ctypes binding.  Nothing here computes on the CPU.
"""
from .hpa import (E2M1_PAGE_BYTES, KV_BF16, KV_E2M1, KV_E4M3, HpaError,  # noqa: F401
                  PageTable, Workspace, decode_step, evict_step, hpa_assign_pages,
                  hpa_assign_pages_workspace, hpa_store_qkv,
                  hpa_decode_attn_window, hpa_default_num_ctas_window, hpa_evict, hpa_evict_compact,
                  hpa_evict_select, hpa_key_weights, hpa_plan_window, hpa_store_kv_at,
                  hpa_arrivals_elems, hpa_combine, hpa_decode_attn, hpa_decode_attn_allheads,
                  hpa_decode_attn_combine_noalloc, hpa_default_num_ctas_allheads,
                  hpa_decode_attn_mma, hpa_default_num_ctas_mma,
                  hpa_decode_attn_fused, hpa_decode_attn_tc, hpa_default_num_ctas_tc,
                  hpa_decode_attn_traced, hpa_default_num_ctas, hpa_max_segments, hpa_plan,
                  hpa_plan_static, hpa_plan_weighted, hpa_selftest_wait_timeout, hpa_static_num_ctas,
                  hpa_static_taskmap_bytes, hpa_store_kv, hpa_taskmap_bytes, lib,
                  trace_summary)
