"""One GPU's MoE-layer forward on MI355X (gfx950): router GEMM and static
top-k gating, counting-sort dispatch queues, grouped SwiGLU expert FFN on
bf16 MFMA, gate-weighted combine; the layer's backward on the same queues;
routing by scores with a balance bias and groups, the combine's gradient, and
the products by expert on their own, with their gradients, in 8-bit integers
and in 4-bit microscaled floats.

The kernels live in ``libmoe.so`` (C ABI in ``include/moe.h``); this package
only binds them to torch tensors and streams.
"""
from ._lib import MoeError, load  # noqa: F401
from .api import (  # noqa: F401
    backward, backward_weights, combine, combine_backward, dequantize_rows_mxfp4, dispatch, dispatch_no_alloc,
    expert_ffn, expert_ffn_fp8, forward, grouped_matmul, grouped_matmul_backward, grouped_matmul_int8,
    grouped_matmul_mxfp4, grouped_workspace_size, mfma_peak_tflops, problem, quantize_rows_fp8, quantize_rows_int8,
    quantize_rows_mxfp4, quantize_weights_fp8, route, route_scored, route_scored_backward,
    route_scored_workspace_size, stream_copy_gbs, workspace_size,
)
