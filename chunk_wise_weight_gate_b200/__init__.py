"""In-Place Test-Time Training MLP layer forward for NVIDIA B200 (sm_100a).

The layer: a gated MLP whose down projection is a fast weight, updated chunk by
chunk with a clipped Hebbian delta from an LM-aligned target and reset at each
document start.  Around it: norms of queries and keys with the position rotation,
linear attention with a decay for each head, and the softmax cross entropy of a linear
head, each with its gradients.  All arithmetic runs in libipttt.so (hand-written
CUDA); this package only marshals arguments (ipttt.py, block_ops.py) and draws seeded
synthetic inputs (synth.py).
"""
from .block_ops import (CrossEntropyConfig, LinearAttentionConfig, QKNormRopeConfig, cross_entropy,
                        cross_entropy_backward, cross_entropy_workspace_size, linear_attention,
                        linear_attention_backward, linear_attention_step, linear_attention_workspace_size,
                        qk_norm_rope, qk_norm_rope_backward)
from .ipttt import (BF16, F32, IptttError, LayerConfig, StreamState, alloc_workspace, core, flops_per_token,
                    forward, get_status, lib, version, workspace_size)

__all__ = ["BF16", "CrossEntropyConfig", "F32", "IptttError", "LayerConfig", "LinearAttentionConfig",
           "QKNormRopeConfig", "StreamState", "alloc_workspace", "core", "cross_entropy", "cross_entropy_backward",
           "cross_entropy_workspace_size", "flops_per_token", "forward", "get_status", "lib", "linear_attention",
           "linear_attention_backward", "linear_attention_step", "linear_attention_workspace_size", "qk_norm_rope",
           "qk_norm_rope_backward", "version", "workspace_size"]
