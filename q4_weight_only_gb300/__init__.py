"""Q4_0 weight-only matmul for one NVIDIA GB300 (sm_103a), and the operators
a served decoder layer runs around it.

The compute lives in libq4_0.so (hand-written CUDA: a decode GEMV, a tcgen05
tensor-core GEMM, a quantizer, a paged cache's append and attention, in
bfloat16 or in 4 bits, and token log probabilities); this package is its thin
Python binding.  Build it with ``q4_weight_only_gb300.build.build()``.
"""
from ._lib import (ERR_CUDA, ERR_DEVICE_INDEX, ERR_DEVICE_TIMEOUT, ERR_INVALID_ARG, ERR_UNSUPPORTED,
                   ERR_WORKSPACE, OK, Y_BF16, Y_F32, Q4Error, device_error, gemm, gemm_plan, gemv, gemv_alloc, lib, matmul,
                   matmul_alloc, matmul_grouped, grouped_launches, matmul_host, host_workspace_bytes, quantize, selftest_wait_timeout, status_string, version,
                   weight_bytes)
from .serving import (MAX_TOP, KVCacheQ4, attention, attention_q4, attention_q4_workspace_bytes,
                      attention_workspace_bytes, kv_append, kv_append_q4, kv_cache_q4, kv_read_q4, token_logprobs)

__all__ = ["quantize", "matmul", "matmul_alloc", "matmul_grouped", "grouped_launches", "matmul_host", "host_workspace_bytes", "gemv", "gemv_alloc", "gemm", "gemm_plan", "weight_bytes", "device_error",
           "version", "status_string", "lib", "selftest_wait_timeout", "Q4Error", "OK", "ERR_INVALID_ARG",
           "ERR_UNSUPPORTED", "ERR_CUDA", "ERR_DEVICE_TIMEOUT", "ERR_WORKSPACE", "Y_F32", "Y_BF16", "ERR_DEVICE_INDEX",
           "kv_append", "attention", "attention_workspace_bytes", "token_logprobs", "MAX_TOP",
           "KVCacheQ4", "kv_cache_q4", "kv_append_q4", "kv_read_q4", "attention_q4", "attention_q4_workspace_bytes"]
