"""MI355X (gfx950) MoE layer forward: route -> permute -> grouped GEMM FC1+SwiGLU ->
grouped GEMM FC2 -> weighted finalize, as hand-written HIP kernels behind the C
ABI in include/moe.h, with the row operators around the experts' products (norm, rows in
expert order, activation with an 8-bit checkpoint) and their gradients.  This package holds
the in-tree library (libmoe.so), its binding, a preallocating layer wrapper and the seeded
workloads."""
from .binding import (BF16, F32, FP8_E4M3, MXFP4, ROUTE_DEEPSEEKV3, ROUTE_DEFAULT,  # noqa: F401
                      ROUTE_RENORMALIZE, ROUTE_RENORMALIZE_NAIVE, MoeError, alloc_workspace,
                      dequantize_mxfp4, dispatch, dispatch_backward,
                      expert_ffn, expert_ffn_fp8, expert_ffn_fp8_fused, expert_ffn_fused,
                      expert_ffn_mxfp4, expert_ffn_noalloc,
                      finalize, finalize_backward, kernel_times, layer_few, layer_few_workspace, lib, permute,
                      quantize_fp8, quantize_mxfp4, rmsnorm, rmsnorm_backward, rmsnorm_backward_workspace, route,
                      route_backward, swiglu, swiglu_backward, timing_enable, workspace_size)
from .layer import MoELayer, layer_for_workload  # noqa: F401
