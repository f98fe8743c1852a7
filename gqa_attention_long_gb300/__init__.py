"""GB300-native (sm_103a) expert attention: the per-layer attention of a flow-matching action
expert over a long VLM KV cache (16 query heads, 8 KV heads, head width 128, 64 tokens).

The compute path is the C-ABI library ``libexpert_attn.so`` (hand-written CUDA kernels); this
package holds its ctypes binding, its build script and the seeded synthetic input generator.
"""
from ._lib import (  # noqa: F401
    EA_KV_BF16, EA_KV_FP8_E4M3, EA_OK, ExpertAttnError, LayerBuffers, alloc_workspace,
    expert_attn_layer, expert_attn_layers, expert_attn_layers_profiled, expert_attn_prologue,
    expert_attn_quantize_cache, expert_attn_quantize_cache_mxfp4, expert_attn_read_status,
    expert_attn_selftest_wait_timeout, expert_attn_set_splits,
    expert_attn_status_string, expert_attn_workspace_init, expert_attn_workspace_size,
    kernels_per_call, lib, make_args, split_parts, split_units,
    alloc_decoder_layer_workspace, expert_decoder_layer, expert_decoder_layer_workspace_size,
    expert_linear64, expert_linear64_workspace_size,
    DecodeBuffers, alloc_decode_workspace, make_decode_args, text_decode_attention,
    text_decode_workspace_init, text_decode_workspace_size,
    Mxfp4Cache, alloc_mxfp4_cache, Mxfp4Rows, make_rows_args, expert_attn_write_mxfp4, expert_attn_read_mxfp4,
    DecodeMxfp4Buffers, alloc_decode_mxfp4_workspace, make_decode_mxfp4_args, text_decode_attention_mxfp4,
    text_decode_mxfp4_workspace_size,
    LayerMxfp4Buffers, alloc_mxfp4_workspace, make_mxfp4_args, expert_attn_layers_mxfp4,
    expert_attn_mxfp4_workspace_size,
    Fp8Cache, alloc_fp8_cache, Fp8Rows, make_fp8_rows_args, expert_attn_write_fp8, expert_attn_read_fp8,
    DecodeFp8Buffers, alloc_decode_fp8_workspace, make_decode_fp8_args, text_decode_attention_fp8,
    text_decode_fp8_workspace_size,
    EvictFp8Buffers, alloc_evict_fp8_workspace, make_evict_fp8_args, expert_attn_evict_fp8,
    expert_attn_evict_fp8_workspace_size,
)
