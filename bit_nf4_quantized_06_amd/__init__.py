"""MI355X (gfx950) library for the frozen-NF4 linear layer with a LoRA adapter.

The computation lives in libqlora_nf4.so (HIP kernels behind a C ABI, see
include/qlora_nf4.h); this package is its thin Python binding.
"""
from .api import (Fp8Weight, GatedSaved, Int8Weight, NF4Weight, qlora_adamw_step, qlora_adamw_step16,
                  qlora_dropout_mask, qlora_dropout_mask_bytes,
                  qlora_fp8_gated_fwd, qlora_fp8_gated_workspace, qlora_fp8_linear_fwd,
                  qlora_fp8_matmul, qlora_fp8_quantize, qlora_fp8_quantize_weight,
                  qlora_fp8_workspace, qlora_gated_linear_bwd, qlora_gated_linear_fwd,
                  qlora_gated_linear_workspace, qlora_grouped_linear_bwd, qlora_grouped_linear_fwd,
                  qlora_grouped_linear_workspace, qlora_int8_linear_fwd,
                  qlora_int8_matmul, qlora_int8_quantize, qlora_int8_workspace,
                  qlora_linear_bwd, qlora_linear_bwd_dropout, qlora_linear_fwd,
                  qlora_linear_fwd_dropout, qlora_linear_fwd_noalloc,
                  qlora_linear_workspace, qlora_linear_workspace_dropout,
                  qlora_nf4_dequantize, qlora_nf4_merge, qlora_nf4_quantize,
                  qlora_pre_dequant_min_tokens, qlora_set_pre_dequant_min_tokens)
from ._lib import QloraError

__all__ = ["Fp8Weight", "GatedSaved", "Int8Weight", "NF4Weight", "QloraError",
           "qlora_nf4_quantize", "qlora_nf4_dequantize", "qlora_nf4_merge", "qlora_linear_fwd", "qlora_linear_bwd", "qlora_linear_workspace",
           "qlora_adamw_step", "qlora_adamw_step16", "qlora_dropout_mask", "qlora_dropout_mask_bytes",
           "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout",
           "qlora_linear_workspace_dropout", "qlora_linear_fwd_noalloc",
           "qlora_set_pre_dequant_min_tokens", "qlora_pre_dequant_min_tokens",
           "qlora_int8_quantize", "qlora_int8_matmul", "qlora_int8_linear_fwd",
           "qlora_int8_workspace", "qlora_grouped_linear_fwd", "qlora_grouped_linear_bwd",
           "qlora_grouped_linear_workspace", "qlora_fp8_quantize", "qlora_fp8_quantize_weight",
           "qlora_fp8_workspace", "qlora_fp8_matmul", "qlora_fp8_linear_fwd",
           "qlora_fp8_gated_workspace", "qlora_fp8_gated_fwd",
           "qlora_gated_linear_fwd", "qlora_gated_linear_bwd", "qlora_gated_linear_workspace"]
