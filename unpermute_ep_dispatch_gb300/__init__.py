"""GB300-native single-GPU MoE expert-parallel token permute / unpermute.

The path has four steps, each a hand-written CUDA kernel for sm_103a behind a
C ABI (``include/epd.h``, ``libepd.so``):

1. ``ep_dispatch_layout`` -- per-expert / per-rank / per-RDMA-node token counts
   and ``is_token_in_rank`` from ``topk_idx`` (plus each pair's rank inside its
   expert, kept in the caller's workspace);
2. ``ep_scan_offsets``    -- ``expert_start_loc``, the exclusive prefix sum of
   the expert counts;
3. ``ep_permute``         -- the ep_scatter copy into the expert-contiguous
   buffer, with ``m_indices`` and ``output_index``;
4. ``ep_unpermute``       -- the topk-weighted, fp32-accumulated combine.

Around them: ``ep_route`` makes the picks and weights from router logits,
``ep_expert_matmul`` is the experts' product (bf16 or e4m3 rows; bias, activation and
residual in its epilogue) between steps 3 and 4, and ``ep_route_backward``,
``ep_expert_matmul_dgrad``, ``ep_expert_matmul_wgrad`` and ``ep_unpermute_backward`` are the
gradients. Beside the experts in a block: ``ep_layer_norm`` and its gradient, ``ep_rotary``,
``ep_cache_append`` and ``ep_decode_attention`` over the paged cache.

``ep_dispatch_layout_offsets`` runs steps 1 and 2 in one launch and
``ep_dispatch`` steps 1 to 3 in one call (one kernel for a small batch).
The Python functions of the same names only marshal torch tensors into the C
calls; the library is loaded on first use and its absence is an error.
"""
from . import workloads  # noqa: F401  (CPU-only input generator)
from ._binding import (  # noqa: F401,E402
    EPD_BF16, EPD_ERR_CAPACITY, EPD_ERR_CUDA, EPD_ERR_INVALID_ARG, EPD_ERR_INVALID_EXPERT,
    EPD_ERR_NONFINITE, EPD_ERR_TIMEOUT, EPD_ERR_UNSUPPORTED, EPD_F32, EPD_FP8_E4M3, EPD_OK,
    EpdError, check_status,
    aligned_capacity, ep_dispatch, ep_dispatch_layout, ep_dispatch_layout_offsets,
    ep_dispatch_lowlatency, ep_expert_matmul, ep_expert_matmul_dgrad, ep_expert_matmul_wgrad,
    ep_permute,
    ep_permute_ex, ep_permute_lowlatency, ep_scan_offsets, ep_scan_offsets_aligned,
    ep_route, ep_route_backward, ep_unpermute, ep_unpermute_backward, epd_workspace_bytes,
    epd_workspace_init, load_library, new_status, new_workspace, status_string, version,
    ep_layer_norm, ep_layer_norm_backward, epd_norm_workspace_bytes, new_norm_workspace,
    ep_cache_append, ep_decode_attention, ep_rotary, epd_attention_workspace_bytes,
    new_attention_workspace, rotary_frequencies, rotary_steps,
)
