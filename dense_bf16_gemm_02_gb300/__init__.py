"""GB300-native dense BF16 GEMM (C = A·Bᵀ, bf16 in, fp32 accumulate, bf16 out),
with its fused-epilogue (bias, activation, residual) and FP8 forms and the
attention forward (MHA / GQA) built on the same tensor-core primitives; and the
operators of a low-precision serving step: microscaled 4-bit matrices
(``quantize_fp4``, ``dequantize_fp4``, ``gemm_fp4``) and a paged 8-bit key/value
cache (``Kv8Cache``, ``kv8_append``, ``attention_kv8``); and those of a batch that
shares its prompts: the pages that its sequences hold (``Kv8Pool``,
``kv8_arrange``, ``kv8_compact``, ``kv8_copy_pages``), the norm of each head's
query and key with the rotation by its position (``qk_norm_rope``), and the
attention that reads shared pages once (``attention_kv8_shared``).

The compute path is the CUDA library built from ``csrc/`` for sm_103a and
reached through the C-ABI of ``include/hk_gemm.h``; this package is its
Python binding.
"""
from .hk_gemm import (HK_ACT_GELU, HK_ACT_NONE, HK_ACT_RELU, HK_ACT_SILU, HK_ERR_INVALID_ARG, HK_ERR_MISALIGNED,
                      HK_ERR_TIMEOUT, HK_ERR_UNSUPPORTED_DEVICE, HK_ERR_WORKSPACE, HK_FLAG_FAULT_DROP_ARRIVE,
                      HK_FLAG_NO_TAIL_SPLIT, HK_INPUT_BF16, HK_INPUT_E4M3, HK_OK, HKError, Plan, attention, gemm,
                      hk_attention_fwd, hk_attention_fwd_ex, hk_gemm_bf16, hk_gemm_bf16_epilogue, hk_gemm_bf16_fused,
                      hk_gemm_bf16_noalloc, hk_gemm_fp8_e4m3, hk_gemm_last_device_status, hk_gemm_last_error_string,
                      hk_gemm_mxfp8, hk_gemm_mxfp8_ex, hk_gemm_mxfp8_workspace_size, hk_status_string, load,
                      HK_FP4_MXFP4, HK_FP4_NVFP4, HK_KV8_FAULT_DROP_ARRIVE, HK_KV8_FEW_ROWS, HK_KV8_MANY_ROWS,
                      HK_TYPE_BF16, HK_TYPE_FP16, HK_TYPE_FP32, hk_fp4_dequantize,
                      hk_attention_kv8, hk_attention_kv8_workspace_size, hk_fp4_quantize, hk_fp4_scales_size,
                      hk_gemm_fp4, hk_gemm_fp4_ex, hk_kv8_append, hk_kv8_arrange, hk_kv8_arrange_workspace_size,
                      hk_kv8_cache, hk_kv8_compact, hk_kv8_compact_workspace_size, hk_kv8_copy_pages, hk_kv8_pool,
                      hk_qk_norm_rope, hk_attention_kv8_shared, hk_attention_kv8_shared_workspace_size)

_LOW_PRECISION = ("Fp4Matrix", "quantize_fp4", "dequantize_fp4", "gemm_fp4", "Kv8Cache", "kv8_append", "attention_kv8")
_SERVING = ("attention_kv8_shared", "Kv8Pool", "kv8_arrange", "kv8_compact", "kv8_copy_pages", "qk_norm_rope")


def __getattr__(name):
    # the modules that import torch load with the first use of one of their names
    if name in _LOW_PRECISION:
        from . import low_precision
        globals().update({n: getattr(low_precision, n) for n in _LOW_PRECISION})
        return globals()[name]
    if name in _SERVING:
        from . import serving
        globals().update({n: getattr(serving, n) for n in _SERVING})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


__all__ = ["attention", "gemm", "Plan", "HKError", "load",
           "hk_gemm_bf16", "hk_gemm_bf16_epilogue", "hk_gemm_bf16_fused", "hk_gemm_bf16_noalloc", "hk_gemm_fp8_e4m3",
           "hk_gemm_mxfp8", "hk_gemm_mxfp8_ex", "hk_gemm_mxfp8_workspace_size", "hk_attention_fwd",
           "hk_attention_fwd_ex", "hk_gemm_last_device_status", "hk_status_string", "hk_gemm_last_error_string",
           "HK_ACT_NONE", "HK_ACT_RELU", "HK_ACT_GELU", "HK_ACT_SILU", "HK_INPUT_BF16", "HK_INPUT_E4M3",
           "HK_OK", "HK_ERR_INVALID_ARG", "HK_ERR_MISALIGNED", "HK_ERR_TIMEOUT", "HK_ERR_WORKSPACE",
           "HK_ERR_UNSUPPORTED_DEVICE", "HK_FLAG_FAULT_DROP_ARRIVE", "HK_FLAG_NO_TAIL_SPLIT",
           "Fp4Matrix", "quantize_fp4", "dequantize_fp4", "gemm_fp4", "Kv8Cache", "kv8_append", "attention_kv8",
           "hk_kv8_cache", "hk_kv8_append", "hk_attention_kv8", "hk_attention_kv8_workspace_size",
           "hk_fp4_quantize", "hk_fp4_dequantize", "hk_fp4_scales_size", "hk_gemm_fp4", "hk_gemm_fp4_ex",
           "Kv8Pool", "kv8_arrange", "kv8_compact", "kv8_copy_pages", "qk_norm_rope", "hk_kv8_pool", "hk_kv8_arrange",
           "hk_kv8_arrange_workspace_size", "hk_kv8_compact", "hk_kv8_compact_workspace_size", "hk_kv8_copy_pages",
           "hk_qk_norm_rope", "attention_kv8_shared", "hk_attention_kv8_shared",
           "hk_attention_kv8_shared_workspace_size", "HK_FP4_MXFP4", "HK_FP4_NVFP4", "HK_KV8_FAULT_DROP_ARRIVE", "HK_KV8_FEW_ROWS", "HK_KV8_MANY_ROWS",
           "HK_TYPE_BF16", "HK_TYPE_FP16", "HK_TYPE_FP32"]
