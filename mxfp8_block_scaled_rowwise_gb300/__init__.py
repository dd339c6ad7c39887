"""GB300 (sm_103a) MXFP8 MoE hot path: quantizer -> permute -> grouped GEMM, with bf16 expert
products and the AdamW step next to it.

The compute lives in the CUDA library ``libmxmoe.so`` (sources in ``csrc/``,
C ABI in ``include/mxmoe.h``); ``binding`` is its thin Python binding and
``synth`` holds the seeded input generators.  Importing the package loads
nothing; the first binding call loads the library and raises if it is missing.
"""
from . import binding, synth  # noqa: F401
from .binding import (MX_COLWISE, MX_ROWWISE, MxError, adamw_grad_norm, adamw_plan,  # noqa: F401
                      adamw_state_values, adamw_step, grouped_gemm_bf16_dgrad, grouped_gemm_bf16_fwd,
                      grouped_gemm_bf16_wgrad, moe_swiglu_bwd, moe_swiglu_fwd, grouped_gemm_mxfp8_dgrad,
                      grouped_gemm_mxfp8_fwd, grouped_gemm_mxfp8_wgrad, moe_gather_rows, moe_permute,
                      mxfp8_quantize)
