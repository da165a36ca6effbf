"""GB300-native tiled FP32 matrix multiply C = A.B (sm_103a CUDA, C ABI).

``sgemm(A, B)`` multiplies CUDA float32 tensors through the C-ABI library
``libsgemm_f32.so`` (built by ``dense_fp32_tiled_gb300.build.build()``);
``sgemm_f32(...)`` is the raw C call on device addresses.  ``sgemm_host(A, B)``
takes CPU tensors (``sgemm_f32_host``: copies overlapped with the product).  ``transpose(x)`` /
``transpose_f32(...)`` run the FP32 transpose, the pages' second workload.
``copy_timeouts()``, ``tc_timeouts()`` and ``wait_selftest(case)`` expose the
bounded waits' failure reporting; ``bank_stride_probe(stride)`` measures the
bank page's stride law on the GPU.

Around the product, the operators of a feed-forward layer (float32, bfloat16,
float16): ``linear(x, w, bias, residual, activation)`` and
``linear_backward``; ``expert_linear`` and ``expert_linear_backward``, the same
over rows sorted by expert; ``expert_sort``, ``expert_gather`` and
``expert_combine`` with their gradients, the tokens' way to their experts and
back.  Around those layers, with their gradients: ``expert_choose``, a router's
choice of experts; ``layer_norm``; ``linear_cross_entropy``, the loss of a product
with a vocabulary without its logits in memory.
"""
from ._binding import (SGEMM_OK, WAIT_SELFTESTS, SgemmError, bank_pattern_probe, bank_stride_probe, copy_timeouts, declared_functions, host_workspace_size,
                       load_library, sgemm, sgemm_f32, sgemm_f32_3xtf32, sgemm_f32_host, sgemm_host,
                       sgemm_f32_static_scratch, sgemm_f32_ws, sgemm_tc, smem_request, smem_shape, status_string,
                       tc_timeouts, tc_workspace_size, transpose, transpose_f32, transpose_smem_request,
                       transpose_status_string, wait_selftest, workspace_size, workspace_size_for,
                       ws_schedule)
from ._layers import (ACTIVATIONS, SCORINGS, expert_choose, expert_choose_backward, expert_combine,
                      expert_combine_backward, expert_gather, expert_gather_backward, expert_linear,
                      expert_linear_backward, expert_sort, layer_norm, layer_norm_backward, linear, linear_backward,
                      linear_cross_entropy, linear_cross_entropy_backward, linear_timeouts)

__all__ = ["ACTIVATIONS", "SCORINGS", "expert_choose", "expert_choose_backward", "layer_norm", "layer_norm_backward",
           "expert_combine", "expert_combine_backward", "expert_gather", "expert_gather_backward",
           "expert_linear", "expert_linear_backward", "expert_sort", "linear", "linear_backward", "linear_cross_entropy",
           "linear_cross_entropy_backward", "linear_timeouts",
           "SGEMM_OK", "WAIT_SELFTESTS", "SgemmError", "bank_pattern_probe", "bank_stride_probe", "copy_timeouts", "declared_functions", "host_workspace_size",
           "load_library", "sgemm", "sgemm_f32", "sgemm_f32_3xtf32", "sgemm_f32_host", "sgemm_host",
           "sgemm_tc", "tc_timeouts", "tc_workspace_size",
           "sgemm_f32_static_scratch", "sgemm_f32_ws", "smem_request", "smem_shape", "status_string",
           "transpose", "transpose_f32", "transpose_smem_request", "transpose_status_string", "wait_selftest",
           "workspace_size", "workspace_size_for", "ws_schedule"]
