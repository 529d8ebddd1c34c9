"""MI355X-native bit-exact emulated FP8 scaled GEMM.

``scaled_mm`` / ``accumulate`` call the HIP library ``libemu_fp8gemm.so``
through its C ABI (``include/emu_fp8gemm.h``); so do the operators beside the
product (``include/emu_operators.h``; ``policy_step`` runs them together) and
those on codes with a scale for each block of 128
(``include/emu_block_operators.h``; ``expert_step``).
Importing this package does not load the library; the first call does, and
fails loudly if it is missing.
"""
from .api import (EmuError, accumulate, abi_version, library_path, scaled_mm,  # noqa: F401
                  workspace_bytes)
from .block_operators import (SwigluCodes, block_quant, block_scaled_mm, block_weight_grad,  # noqa: F401
                              grouped_block_scaled_mm, swiglu_block_backward, swiglu_block_quant)
from .operators import (TokenLogprobs, add_rms_norm_backward, add_rms_norm_quant, int8_scaled_mm,  # noqa: F401
                        token_logprobs, token_logprobs_backward)
