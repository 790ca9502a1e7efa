"""GB300 (sm_103a) W8A8 / W4A8 quantized linear layer, with a quantized
key/value cache and the attention over it, the norm that feeds a layer its
codes, and the layer and the gated feed-forward block in 8-bit floats.

The compute lives in libw8a8.so (hand-written CUDA behind a C ABI declared in
include/w8a8.h); ``binding`` marshals torch tensors to it.  ``synth`` holds
the seeded input generators.
"""
from .binding import (KVCache, W8A8Error, fp8_feed_forward, fp8_feed_forward_workspace_bytes,
                      fp8_gated_gemm, fp8_gemm, fp8_linear, fp8_linear_workspace_bytes, kv_cache_attention, kv_cache_attention_workspace_bytes,
                      kv_cache_read, kv_cache_write, linear, linear_noalloc, load, pack_weight_int4, quantize_act_fp8, quantize_act_per_token,
                      quantize_act_per_token_h, quantize_weight_fp8, quantize_weight_int8,
                      rms_norm, rms_norm_quantize, w4a8_gemm,
                      w8a8_check_status, w8a8_gemm, w8a8_gemm_h, w8a8_gemm_i32,
                      w8a8_is_available, w8a8_linear_workspace_bytes, w8a8_mv,
                      w8a8_status_string, w8a8_test_set_fault, weight_only_gemm)

__all__ = ["KVCache", "fp8_feed_forward", "fp8_feed_forward_workspace_bytes", "fp8_gated_gemm", "fp8_gemm",
           "fp8_linear", "fp8_linear_workspace_bytes", "quantize_act_fp8", "quantize_weight_fp8", "rms_norm",
           "rms_norm_quantize", "kv_cache_attention", "kv_cache_attention_workspace_bytes", "kv_cache_read",
           "kv_cache_write", "W8A8Error", "linear", "linear_noalloc", "load", "pack_weight_int4", "quantize_act_per_token",
           "quantize_act_per_token_h", "w8a8_gemm_h", "quantize_weight_int8", "w4a8_gemm", "w8a8_check_status", "w8a8_gemm",
           "w8a8_gemm_i32", "w8a8_is_available", "w8a8_linear_workspace_bytes", "w8a8_mv",
           "w8a8_status_string", "w8a8_test_set_fault", "weight_only_gemm"]
