"""GB300-native (sm_103a) gated delta rule: chunkwise forward and slot-indexed decode.

The kernels live in ``libgdn.so`` (C ABI in ``include/gdn.h``); this package is
its thin PyTorch binding:

* :func:`chunk_gated_delta_rule` -- chunkwise forward (training / prefill,
  packed varlen via ``cu_seqlens``, optional slot-cache state I/O).
* :func:`gated_delta_decode` -- one token per request on a slot-indexed
  recurrent-state cache, ``-1`` = padding; :func:`gated_delta_decode_multi` for
  several tokens per request.
* ``*_fused_gates`` -- the same with g and beta computed in the kernels.
* :func:`chunk_gated_delta_product`, :func:`gated_delta_product_decode` -- the Gated
  Delta Product (several delta-rule writes per token).
* :func:`chunk_gated_delta_rule_bwd` -- the backward (dq, dk, dv, dg, dbeta, d_initial_state);
  :func:`chunk_gated_delta_rule_trainable` -- forward + backward as a torch autograd op;
  :func:`chunk_gated_delta_rule_bwd_fused_gates` and
  :func:`chunk_gated_delta_rule_fused_gates_trainable` -- the same through the fused gates
  (gradients w.r.t. a, b, A_log, dt_bias).
* :func:`chunk_linear_attn`, :func:`chunk_linear_attn_bwd`, :func:`chunk_linear_attn_trainable`,
  :func:`linear_attn_decode` -- linear attention with a decay for each head: chunked forward,
  backward, autograd op and single-token decode on the same slot cache.
* :func:`gated_linear_recurrence`, ``*_bwd``, ``*_trainable``, ``*_decode`` and each with
  ``_fused_gates`` -- the gated linear recurrence of each channel: forward over dense or packed
  sequences, backward, autograd op, single-token decode on a slot cache.
* :func:`qk_norm_rotate`, :func:`qk_norm_rotate_bwd`, :func:`qk_norm_rotate_trainable` -- the norm of
  each head's queries and keys with the rotation of their positions (one or several axes).
* :func:`group_norm_act`, :func:`group_norm_act_bwd`, :func:`group_norm_act_trainable` -- group
  norm with an activation or gate, channels last: forward, backward, autograd op.

Device-side errors (bad slot, bad ``cu_seqlens``, a timed-out in-kernel wait) reach the
caller only through a ``dev_status`` tensor, or as :class:`GdnDeviceError` with ``check=True``.
"""
from .api import (GdnDeviceError, GdnError, chunk_fwd_path, chunk_gated_delta_product, chunk_gated_delta_rule,
                  chunk_gated_delta_rule_bwd, chunk_gated_delta_rule_bwd_fused_gates,
                  chunk_gated_delta_rule_fused_gates, chunk_gated_delta_rule_fused_gates_trainable,
                  chunk_gated_delta_rule_trainable, chunk_workspace_size, gated_delta_decode,
                  gated_delta_decode_fused_gates, gated_delta_decode_multi,
                  gated_delta_product_decode)
from .group_norm import group_norm_act, group_norm_act_bwd, group_norm_act_trainable
from .linear_attn import (chunk_linear_attn, chunk_linear_attn_bwd, chunk_linear_attn_trainable,
                          linear_attn_decode)
from .qk_rotate import qk_norm_rotate, qk_norm_rotate_bwd, qk_norm_rotate_trainable
from .recurrence import (gated_linear_recurrence, gated_linear_recurrence_bwd,
                         gated_linear_recurrence_bwd_fused_gates, gated_linear_recurrence_decode,
                         gated_linear_recurrence_decode_fused_gates, gated_linear_recurrence_fused_gates,
                         gated_linear_recurrence_fused_gates_trainable, gated_linear_recurrence_trainable)

__all__ = ["chunk_gated_delta_rule", "gated_delta_decode", "gated_delta_decode_multi",
           "chunk_gated_delta_rule_fused_gates", "gated_delta_decode_fused_gates",
           "chunk_gated_delta_product", "gated_delta_product_decode",
           "chunk_gated_delta_rule_bwd", "chunk_gated_delta_rule_trainable",
           "chunk_gated_delta_rule_bwd_fused_gates", "chunk_gated_delta_rule_fused_gates_trainable",
           "chunk_linear_attn", "chunk_linear_attn_bwd", "chunk_linear_attn_trainable",
           "linear_attn_decode", "group_norm_act", "group_norm_act_bwd", "group_norm_act_trainable",
           "gated_linear_recurrence", "gated_linear_recurrence_fused_gates",
           "gated_linear_recurrence_bwd", "gated_linear_recurrence_bwd_fused_gates",
           "gated_linear_recurrence_trainable", "gated_linear_recurrence_fused_gates_trainable",
           "gated_linear_recurrence_decode", "gated_linear_recurrence_decode_fused_gates",
           "qk_norm_rotate", "qk_norm_rotate_bwd", "qk_norm_rotate_trainable",
           "chunk_workspace_size", "chunk_fwd_path", "GdnError", "GdnDeviceError"]
__version__ = "0.1.0"
