"""Linear attention with a decay for each head: the PyTorch binding of the ``gdn_linear_attn_*``
entry points (argument checks, outputs and scratch; every computation runs in the kernels).

    S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t

per (sequence, value head h) with a K x V fp32 state in the layout of the gated delta rule's, so
both kinds of layer share a slot cache.  ``log_decay`` is a constant of the layer: no gradient.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .api import DEVICE_ERRORS_DOC, _DT, _need, _ptr, _raise_on_status, _scale, _status

__all__ = ["chunk_linear_attn", "chunk_linear_attn_bwd", "chunk_linear_attn_trainable",
           "linear_attn_decode"]


def _fit(dev, *wanted) -> bool:
    """Whether every (tensor or None, dtype, shape) is contiguous, on ``dev`` and as said.  One quick
    test for the usual case (a decode step's call takes longer on the host than on the device);
    where it fails, the caller goes through ``_need`` one by one for the message."""
    try:
        for t, dtype, shape in wanted:
            if t is not None and not (t.dtype is dtype and t.shape == shape and t.device == dev
                                      and t.is_contiguous()):
                return False
        return True
    except AttributeError:
        return False


def _stream(dev) -> int:
    """The current stream's handle (without a Stream object around it)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _int32(name, *sizes):
    """Refuses what the C interface's integers do not hold (ctypes would cut it down to 32 bits)."""
    if max(sizes) >= 1 << 31:
        raise ValueError("sizes beyond 2^31 - 1 rejected by %s: %s" % (name, sizes))


def _inputs(q, k, v, log_decay, cu_seqlens):
    """Checks shared by the chunked calls; returns (device, dtype, sizes, N)."""
    if (isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 4 and q.dtype in _DT
            and isinstance(v, torch.Tensor) and v.dim() == 4):
        dev, dt = q.device, q.dtype
        B, T, Hqk, K = q.shape
        Hv, V = v.shape[2:]
        _int32("linear attention", B, T, Hqk, K, Hv, V)
        if _fit(dev, (q, dt, (B, T, Hqk, K)), (k, dt, (B, T, Hqk, K)), (v, dt, (B, T, Hv, V)),
                (log_decay, torch.float32, (Hv,))) and log_decay is not None and k is not None:
            if cu_seqlens is None:
                return dev, dt, (B, T, Hqk, Hv, K, V), B
            if B == 1 and _fit(dev, (cu_seqlens, torch.int32, cu_seqlens.shape)) \
                    and cu_seqlens.dim() == 1 and cu_seqlens.shape[0] > 0:
                _int32("linear attention", cu_seqlens.shape[0])
                return dev, dt, (B, T, Hqk, Hv, K, V), cu_seqlens.shape[0] - 1
    _need(q, "q", (torch.float32, torch.bfloat16))
    dev, dt = q.device, q.dtype
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hqk, K]")
    _need(k, "k", dt, dev, q.shape)
    _need(v, "v", dt, dev)
    if v.dim() != 4 or v.shape[:2] != q.shape[:2]:
        raise ValueError("v must be [B, T, Hv, V]")
    B, T, Hqk, K = q.shape
    Hv, V = v.shape[2], v.shape[3]
    _need(log_decay, "log_decay", torch.float32, dev, (Hv,))
    N = B
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        if B != 1:
            raise ValueError("cu_seqlens requires B == 1")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [num_seqs + 1]")
        N = cu_seqlens.numel() - 1
    return dev, dt, (B, T, Hqk, Hv, K, V), N


def _scratch(need, name, workspace, dev):
    """The workspace to pass on: the caller's when it is large enough, else a new one."""
    if need == (1 << 64) - 1:
        raise ValueError("sizes rejected by %s" % name)
    if workspace is not None:
        _need(workspace, "workspace", None, dev)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def chunk_linear_attn(q, k, v, log_decay, scale=None, initial_state=None, output_final_state=False,
                      cu_seqlens=None, *, state_indices=None, out=None, final_state=None,
                      workspace=None, dev_status=None, check=False
                      ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked forward through ``gdn_linear_attn_chunk_fwd``.

    q, k [B, T, Hqk, K]; v [B, T, Hv, V]; log_decay [Hv] fp32; scale None -> 1/sqrt(K).  Returns
    ``(o, final_state or None)``.  ``cu_seqlens`` ([N + 1] int32, B == 1), ``state_indices`` (a
    slot cache, -1 = padding, updated in place by default), ``out``, ``final_state``,
    ``workspace``, ``dev_status`` and ``check`` as in :func:`chunk_gated_delta_rule`.

    A NaN or infinity in a token reaches its whole 64-token chunk, also the tokens before it there,
    and what follows in its sequence and head; nothing else.
    """
    dev, dt, (B, T, Hqk, Hv, K, V), N = _inputs(q, k, v, log_decay, cu_seqlens)
    num_slots = 0
    st_shape = (N, Hv, K, V)
    if state_indices is not None:
        _need(state_indices, "state_indices", torch.int32, dev, (N,))
        cache = initial_state if initial_state is not None else final_state
        if cache is None:
            raise ValueError("state_indices needs initial_state or final_state (the slot cache)")
        num_slots = cache.shape[0]
        _int32("linear attention", num_slots)
        st_shape = (num_slots, Hv, K, V)
        if output_final_state and final_state is None:
            final_state = initial_state
    if not output_final_state:
        final_state = None
    if not _fit(dev, (initial_state, torch.float32, st_shape), (final_state, torch.float32, st_shape),
                (out, dt, v.shape)):
        for t, name in ((initial_state, "initial_state"), (final_state, "final_state")):
            if t is not None:
                _need(t, name, torch.float32, dev, st_shape)
        if out is not None:
            _need(out, "out", dt, dev, v.shape)
    if output_final_state and final_state is None:
        final_state = torch.empty(st_shape, dtype=torch.float32, device=dev)
    if out is None:
        out = torch.empty_like(v)
    L = _lib.load()
    need = L.gdn_linear_attn_chunk_fwd_workspace_size(B, T, Hqk, Hv, K, V, N, _DT[dt])
    workspace, ws_bytes = _scratch(need, "gdn_linear_attn_chunk_fwd", workspace, dev)
    dev_status = _status(dev_status, check, dev)
    st = L.gdn_linear_attn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), B, T, Hqk, Hv, K, V,
                                     _DT[dt], _scale(scale), _ptr(initial_state),
                                     int(bool(output_final_state)), _ptr(final_state),
                                     _ptr(cu_seqlens), N, _ptr(state_indices), num_slots, _ptr(out),
                                     _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(dev))
    _lib.check("gdn_linear_attn_chunk_fwd", st)
    _raise_on_status("gdn_linear_attn_chunk_fwd", dev_status, check)
    return out, final_state


def chunk_linear_attn_bwd(q, k, v, log_decay, d_o, d_final_state=None, scale=None,
                          initial_state=None, cu_seqlens=None, *, need_d_initial_state=True,
                          workspace=None, dev_status=None, check=False):
    """Gradients of :func:`chunk_linear_attn` (no slot cache) through
    ``gdn_linear_attn_chunk_bwd``: ``(dq, dk, dv, d_initial_state)``, the first three in q's
    dtype, the last fp32 [N, Hv, K, V] (None when ``need_d_initial_state`` is False)."""
    dev, dt, (B, T, Hqk, Hv, K, V), N = _inputs(q, k, v, log_decay, cu_seqlens)
    st_shape = (N, Hv, K, V)
    if d_o is None or not _fit(dev, (d_o, dt, v.shape), (initial_state, torch.float32, st_shape),
                               (d_final_state, torch.float32, st_shape)):
        _need(d_o, "d_o", dt, dev, (B, T, Hv, V))
        for t, name in ((initial_state, "initial_state"), (d_final_state, "d_final_state")):
            if t is not None:
                _need(t, name, torch.float32, dev, st_shape)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dh0 = torch.empty(st_shape, dtype=torch.float32, device=dev) if need_d_initial_state else None
    L = _lib.load()
    need = L.gdn_linear_attn_chunk_bwd_workspace_size(B, T, Hqk, Hv, K, V, N, _DT[dt])
    workspace, ws_bytes = _scratch(need, "gdn_linear_attn_chunk_bwd", workspace, dev)
    dev_status = _status(dev_status, check, dev)
    st = L.gdn_linear_attn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), B, T, Hqk, Hv, K, V,
                                     _DT[dt], _scale(scale), _ptr(initial_state), _ptr(cu_seqlens),
                                     N, _ptr(d_o), _ptr(d_final_state), _ptr(dq), _ptr(dk),
                                     _ptr(dv), _ptr(dh0), _ptr(workspace), ws_bytes,
                                     _ptr(dev_status), _stream(dev))
    _lib.check("gdn_linear_attn_chunk_bwd", st)
    _raise_on_status("gdn_linear_attn_chunk_bwd", dev_status, check)
    return dq, dk, dv, dh0


def _incoming(t):
    """An incoming gradient as the kernels take it: contiguous, on a 16-byte boundary (a part of a
    larger gradient may start anywhere)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _FirstOnly(torch.autograd.Function):
    """Hands ``count`` gradients on and stands between them and what they depend on, for a second
    derivative to meet: without it they would be constants, and its terms would be missing."""

    @staticmethod
    def forward(ctx, name, count, *tensors):
        ctx.name = name
        return tensors[:count]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("%s has no second derivative" % ctx.name)


def _first_only(name, grads, inputs):
    """What a backward returns under ``create_graph``: ``grads``, made from ``inputs``."""
    made = [g for g in grads if g is not None]
    made = iter(_FirstOnly.apply(name, len(made), *made, *inputs))
    return tuple(None if g is None else next(made) for g in grads)


class _ChunkLinearAttn(torch.autograd.Function):
    """gdn_linear_attn_chunk_fwd forward, gdn_linear_attn_chunk_bwd backward."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, initial_state, scale, output_final_state, cu_seqlens):
        o, fin = chunk_linear_attn(q, k, v, log_decay, scale=scale, initial_state=initial_state,
                                   output_final_state=output_final_state, cu_seqlens=cu_seqlens)
        ctx.save_for_backward(q, k, v, log_decay, initial_state, cu_seqlens)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return o, fin

    @staticmethod
    def backward(ctx, d_o, d_fin):
        q, k, v, log_decay, init, cu = ctx.saved_tensors
        d_o = torch.zeros_like(v) if d_o is None else _incoming(d_o)
        grads = chunk_linear_attn_bwd(
            q, k, v, log_decay, d_o, None if d_fin is None else _incoming(d_fin),
            scale=ctx.scale, initial_state=init, cu_seqlens=cu,
            need_d_initial_state=init is not None and ctx.needs_input_grad[4])
        if torch.is_grad_enabled():
            grads = _first_only("chunk_linear_attn_trainable", grads, (q, k, v, init, d_o, d_fin))
        dq, dk, dv, dh0 = grads
        return dq, dk, dv, None, dh0, None, None, None


def chunk_linear_attn_trainable(q, k, v, log_decay, scale=None, initial_state=None,
                                output_final_state=False, cu_seqlens=None):
    """:func:`chunk_linear_attn` as a differentiable op (torch autograd) in q, k, v and
    ``initial_state``; a second derivative is refused.  Returns ``(o, final_state or None)``."""
    if log_decay.requires_grad:
        raise ValueError("log_decay is a constant of the layer: it has no gradient")
    return _ChunkLinearAttn.apply(q, k, v, log_decay, initial_state, scale,
                                  bool(output_final_state), cu_seqlens)


def linear_attn_decode(q, k, v, log_decay, ssm_state, batch_indices=None, scale=None, *, out=None,
                       dev_status=None, check=False) -> torch.Tensor:
    """One token per request through ``gdn_linear_attn_decode`` (the recurrent form);
    ``ssm_state`` is updated in place.

    q, k [n, Hqk, K]; v [n, Hv, V]; log_decay [Hv] fp32; ssm_state [num_slots, Hv, K, V] fp32;
    batch_indices [n] int32 (-1 = padding: a zero row) or None (request i uses slot i).  Returns
    o [n, Hv, V].
    """
    usual = False
    if isinstance(q, torch.Tensor) and isinstance(v, torch.Tensor) and q.dim() == 3 and v.dim() == 3:
        dev, dt = q.device, q.dtype
        n, Hqk, K = q.shape
        Hv, V = v.shape[1:]
        usual = (q.is_cuda and dt in _DT and k is not None and log_decay is not None
                 and isinstance(ssm_state, torch.Tensor) and ssm_state.dim() == 4
                 and _fit(dev, (q, dt, (n, Hqk, K)), (k, dt, (n, Hqk, K)), (v, dt, (n, Hv, V)),
                          (log_decay, torch.float32, (Hv,)), (out, dt, (n, Hv, V)),
                          (ssm_state, torch.float32, (ssm_state.shape[0], Hv, K, V)),
                          (batch_indices, torch.int32, (n,))))
    if not usual:
        _need(q, "q", (torch.float32, torch.bfloat16))
        dev, dt = q.device, q.dtype
        if q.dim() != 3:
            raise ValueError("q must be [n, Hqk, K]")
        n, Hqk, K = q.shape
        _need(k, "k", dt, dev, q.shape)
        _need(v, "v", dt, dev)
        if v.dim() != 3 or v.shape[0] != n:
            raise ValueError("v must be [n, Hv, V]")
        Hv, V = v.shape[1], v.shape[2]
        _need(log_decay, "log_decay", torch.float32, dev, (Hv,))
        _need(ssm_state, "ssm_state", torch.float32, dev)
        if ssm_state.dim() != 4 or tuple(ssm_state.shape[1:]) != (Hv, K, V):
            raise ValueError("ssm_state must be [num_slots, Hv, K, V]")
        if batch_indices is not None:
            _need(batch_indices, "batch_indices", torch.int32, dev, (n,))
        if out is not None:
            _need(out, "out", dt, dev, (n, Hv, V))
    _int32("linear attention", n, Hqk, K, Hv, V, ssm_state.shape[0])
    if out is None:
        out = torch.empty_like(v)
    dev_status = _status(dev_status, check, dev)
    st = _lib.load().gdn_linear_attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
                                            _ptr(ssm_state), ssm_state.shape[0],
                                            _ptr(batch_indices), n, Hqk, Hv, K, V, _DT[dt],
                                            _scale(scale), _ptr(out), _ptr(dev_status),
                                            _stream(dev))
    _lib.check("gdn_linear_attn_decode", st)
    _raise_on_status("gdn_linear_attn_decode", dev_status, check)
    return out


for _f in (chunk_linear_attn, chunk_linear_attn_bwd, linear_attn_decode):
    _f.__doc__ += DEVICE_ERRORS_DOC
