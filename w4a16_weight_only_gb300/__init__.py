"""AWQ W4A16 weight-only linear for GB300 (sm_103a).

The computation lives in ``libawq_gb300.so`` (C ABI in ``include/awq.h``, CUDA sources
in ``csrc/``).  This package only builds it (``build.py``) and marshals arguments
(``_binding.py``, ``_layer.py``, ``_step.py``); PyTorch supplies device memory and streams.
"""
from ._binding import (AwqError, AwqLinear, PATHS, awq_dequant, awq_dequant_w8, awq_gemm, awq_gemm_grouped,
                       awq_gemm_packed, awq_gemm_packed_grouped, awq_gemm_packed_noalloc,
                       awq_gemm_packed_workspace_size, awq_repack, awq_repack_experts, awq_repack_size,
                       awq_gemm_w8, awq_quantize_rtn,
                       device_status,
                       last_error, load_library, runtime_available, select_path,
                       selftest_attention_give_up, selftest_wait_timeout)
from ._layer import (awq_attention_shared, awq_attention_shared_workspace_size, awq_moe_combine, awq_moe_dispatch,
                     awq_moe_dispatch_workspace_size, awq_moe_route, awq_rope, awq_rope_append, awq_rope_table)
from ._step import (awq_attention_kv4, awq_attention_kv4_workspace_size, awq_kv4_page_bytes, awq_kv4_read, awq_moe_layer,
                    awq_moe_layer_workspace_size, awq_residual_norm, awq_rope_append_kv4)

__all__ = ["AwqError", "AwqLinear", "PATHS", "awq_dequant", "awq_dequant_w8", "awq_gemm", "awq_gemm_grouped",
           "awq_gemm_packed", "awq_gemm_packed_grouped", "awq_gemm_packed_noalloc",
           "awq_gemm_packed_workspace_size", "awq_repack", "awq_repack_experts", "awq_repack_size",
           "awq_gemm_w8", "awq_quantize_rtn",
           "device_status",
           "last_error",
           "load_library", "runtime_available", "select_path", "selftest_attention_give_up",
           "selftest_wait_timeout",
           "awq_rope_table", "awq_rope", "awq_rope_append", "awq_attention_shared",
           "awq_attention_shared_workspace_size", "awq_moe_route", "awq_moe_dispatch",
           "awq_moe_dispatch_workspace_size", "awq_moe_combine",
           "awq_kv4_page_bytes", "awq_rope_append_kv4", "awq_kv4_read", "awq_attention_kv4",
           "awq_attention_kv4_workspace_size", "awq_residual_norm", "awq_moe_layer", "awq_moe_layer_workspace_size"]
