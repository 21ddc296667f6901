"""MI355X-native QLoRA hot path: NF4 + double-quantized frozen linear layer with
a bf16 LoRA adapter (forward, backward, batch-1 decode), the same layer on an
8-bit frozen weight, dropout of the adapter's input, the gated feed-forward
block, and adapters of many requests beside one weight.

The compute runs in libqlora.so (hand-written gfx950 HIP kernels behind a C
ABI, include/qlora.h); this package is its thin Python binding.  The library
is loaded on the first call and a missing build is an error.
"""

from .ops import (AdapterPool, Dropout, GemvJob, Int8Weight, QuantizedWeight, dequant, dropout, gated_bwd, gated_fwd,
                  gated_many_fwd, gemv, i8_dequant, i8_linear_bwd, i8_linear_fwd, i8_matmul, i8_quantize, linear_bwd,
                  linear_fwd, many_fwd, nf4_levels, quantize, sizes, workspace, workspace_bytes)

__all__ = ["AdapterPool", "Dropout", "GemvJob", "Int8Weight", "QuantizedWeight", "dequant", "dropout", "gated_bwd",
           "gated_fwd", "gated_many_fwd", "gemv", "i8_dequant", "i8_linear_bwd", "i8_linear_fwd", "i8_matmul",
           "i8_quantize", "linear_bwd", "linear_fwd", "many_fwd", "nf4_levels", "quantize", "sizes", "workspace",
           "workspace_bytes"]
__version__ = "0.1.0"
