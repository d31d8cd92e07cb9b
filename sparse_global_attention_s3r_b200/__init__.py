"""B200 (sm_100a) sparse global attention of Speed3R, and the dense operators that stand beside it
in a multi-view transformer: a C-ABI CUDA library (libs3r.so, include/s3r.h and
include/s3r_view.h) and its thin torch binding.

    from sparse_global_attention_s3r_b200 import Config, sparse_attn_fwd
"""
from .api import (Config, HostPipeline, SparseAttention, SparseAttentionFunction, alloc_workspace,
                  bwd_workspace_bytes, cmp_attn_and_score, compress_kv, gate_combine,
                  read_device_status, sel_attn, sparse_attn_bwd, sparse_attn_fwd, topk_blocks,
                  workspace_bytes)
from .view import (QKNormConfig, QKNormGrads, QKNormRopeFunction, ViewAttentionFunction,
                   ViewConfig, qk_norm_rope, qk_norm_rope_bwd, view_attn_bwd, view_attn_fwd,
                   view_positions)

__all__ = ["Config", "HostPipeline", "SparseAttention", "SparseAttentionFunction",
           "alloc_workspace", "bwd_workspace_bytes", "cmp_attn_and_score", "compress_kv",
           "gate_combine", "read_device_status", "sel_attn", "sparse_attn_bwd", "sparse_attn_fwd",
           "topk_blocks", "workspace_bytes",
           "QKNormConfig", "QKNormGrads", "QKNormRopeFunction", "ViewAttentionFunction",
           "ViewConfig", "qk_norm_rope", "qk_norm_rope_bwd", "view_attn_bwd", "view_attn_fwd",
           "view_positions"]
