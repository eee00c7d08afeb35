"""Norm of queries and keys for each head with the rotation of their positions, in one pass: the
PyTorch binding of the ``gdn_qk_norm_rotate_*`` entry points.

    n = x / sqrt(mean(x^2) + eps) * w       ("rms"; "l2": the sum instead of the mean; None: x w)

for each head x, then the first R = 2 len(inv_freq) values of n turn in pairs: pair j, values
(j, j + R / 2) or interleaved (2 j, 2 j + 1), by the angle position * inv_freq[j].
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .api import _DT, _need, _ptr
from .linear_attn import _first_only, _fit, _int32, _scratch, _stream
from .recurrence import _elsewhere

__all__ = ["qk_norm_rotate", "qk_norm_rotate_bwd", "qk_norm_rotate_trainable"]

_NORM = {None: _lib.GDN_NORM_NONE, "none": _lib.GDN_NORM_NONE, "rms": _lib.GDN_NORM_RMS,
         "l2": _lib.GDN_NORM_L2}
_Strides = ctypes.c_longlong * 3


def _heads(t, name, dtype, dev):
    """Checks t [B, T, H, K] or [n, H, K] (one token a row); its sizes and strides as [B, T, H, K]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != dev or t.device.type != "cuda":
        if t.device.type != "cuda":
            raise ValueError("%s must be a CUDA tensor (got %s)" % (name, t.device))
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.dim() not in (3, 4):
        raise ValueError("%s must be [B, T, H, K] or [n, H, K]" % name)
    shape, strides = tuple(t.shape), t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s must have the values of a head next to each other" % name)
    if t.dim() == 3:
        return (shape[0], 1) + shape[1:], (strides[0], 0, strides[1])
    return shape, strides[:3]


def _inputs(q, k, inv_freq, positions, q_weight, k_weight, norm, eps, sections):
    """Checks shared by the calls; returns (device, what forward's and backward's C calls share)."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dev = q.device
    (B, T, Hq, K), qs = _heads(q, "q", (torch.float32, torch.bfloat16), dev)
    (Bk, Tk, Hk, Kk), ks = _heads(k, "k", q.dtype, dev)
    if k.dim() != q.dim() or (Bk, Tk, Kk) != (B, T, K):
        raise ValueError("k has shape %s, which does not go with q's %s" % (tuple(k.shape), tuple(q.shape)))
    if Hq < 1 or Hk < 1 or not 1 <= K <= 256:
        raise ValueError("q and k need at least a head, of 1 to 256 values")
    _int32("the norm of q and k", B, T, B * T, Hq, Hk)
    R = 0
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float32, dev)
        if inv_freq.dim() != 1 or 2 * inv_freq.shape[0] > K:
            raise ValueError("inv_freq must be [R / 2] with R at most %d" % K)
        R = 2 * inv_freq.shape[0]
    axes = 1
    if sections is not None:
        sections = tuple(int(n) for n in sections)
        axes = len(sections)
        if not 1 <= axes <= 4 or min(sections) < 0 or sum(sections) != R // 2:
            raise ValueError("sections must be 1 to 4 counts that make %d pairs (got %s)" % (R // 2, sections))
    lead = tuple(q.shape[:-2])
    if positions is not None:
        shape = lead if axes == 1 else (axes,) + lead
        if not _fit(dev, (positions, torch.int32, shape)) and not (
                axes == 1 and _fit(dev, (positions, torch.int32, (1,) + lead))):
            _need(positions, "positions", torch.int32, dev, shape)
    wb = None
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            if not isinstance(t, torch.Tensor) or t.dtype != wb or not _fit(dev, (t, wb, (K,))):
                _need(t, name, (q.dtype, torch.float32) if wb is None else wb, dev, (K,))
            wb = t.dtype
    if norm not in _NORM:
        raise ValueError("norm must be 'rms', 'l2' or None (got %r)" % (norm,))
    eps = float(eps)
    if not eps >= 0.0:
        raise ValueError("eps must not be negative (got %r)" % eps)
    return dev, _Call((_Strides(*qs), _Strides(*ks), B, T, Hq, Hk, K, R, _DT[q.dtype], _NORM[norm], eps),
                      _DT[wb or torch.float32], (axes, (ctypes.c_int * axes)(*sections) if axes > 1 else None))


class _Call:
    """The arguments of a C call that are not tensors."""

    def __init__(self, sizes, w_dtype, axes):
        self.sizes, self.w_dtype, self.axes = sizes, w_dtype, axes

    def args(self, inv_freq, positions, q_weight, k_weight, interleaved):
        return (*self.sizes, _ptr(q_weight), _ptr(k_weight), self.w_dtype, _ptr(inv_freq), _ptr(positions), *self.axes,
                interleaved)


def qk_norm_rotate(q, k, inv_freq=None, positions=None, q_weight=None, k_weight=None, *, norm="rms", eps=1e-6,
                   sections=None, interleaved=False, out_q=None, out_k=None):
    """Forward through ``gdn_qk_norm_rotate_fwd``: ``(q, k)`` normalised and turned, contiguous.

    q [B, T, Hq, K] and k [B, T, Hk, K] in fp32 or bf16 ([n, H, K]: one token a row), K at most 256, with
    any strides but the last axis's, so they may be parts of one projection.  inv_freq [R / 2] fp32, R at
    most K, or None (no rotation).  positions [B, T] int32 ([n] for rows of one token) or None: token t of a
    row has position t.  With several axes (``sections``: how many pairs turn by each, in order) positions
    [axes, B, T].  q_weight, k_weight [K] in fp32 or q's dtype, or None.  norm "rms", "l2" or None.
    ``out_q``, ``out_k``: contiguous, each may be its input.
    """
    dev, call = _inputs(q, k, inv_freq, positions, q_weight, k_weight, norm, eps, sections)
    return _forward(q, k, inv_freq, positions, q_weight, k_weight, call, int(bool(interleaved)), out_q, out_k)


def _forward(q, k, inv_freq, positions, q_weight, k_weight, call, interleaved, out_q=None, out_k=None):
    """The forward's outputs and call, after the checks of its inputs."""
    dev = q.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return _forward(q, k, inv_freq, positions, q_weight, k_weight, call, interleaved, out_q, out_k)
    if out_q is None:
        out_q = torch.empty(q.shape, dtype=q.dtype, device=dev)
    elif not _fit(dev, (out_q, q.dtype, q.shape)):
        _need(out_q, "out_q", q.dtype, dev, q.shape)
    if out_k is None:
        out_k = torch.empty(k.shape, dtype=q.dtype, device=dev)
    elif not _fit(dev, (out_k, q.dtype, k.shape)):
        _need(out_k, "out_k", q.dtype, dev, k.shape)
    st = _lib.load().gdn_qk_norm_rotate_fwd(
        q.data_ptr(), k.data_ptr(), *call.args(inv_freq, positions, q_weight, k_weight, interleaved),
        out_q.data_ptr(), out_k.data_ptr(), _stream(dev))
    _lib.check("gdn_qk_norm_rotate_fwd", st)
    return out_q, out_k


def qk_norm_rotate_bwd(d_q, d_k, q, k, inv_freq=None, positions=None, q_weight=None, k_weight=None, *,
                       norm="rms", eps=1e-6, sections=None, interleaved=False, need_weights=True,
                       workspace=None):
    """Gradients of :func:`qk_norm_rotate` through ``gdn_qk_norm_rotate_bwd``: ``(dq, dk, dq_weight,
    dk_weight)`` from d_q, d_k (contiguous, like the outputs) and the forward's inputs; dq, dk in q's
    dtype, the weights' fp32 [K] (None without ``need_weights``)."""
    dev, call = _inputs(q, k, inv_freq, positions, q_weight, k_weight, norm, eps, sections)
    if d_q is None or d_k is None or not _fit(dev, (d_q, q.dtype, q.shape), (d_k, q.dtype, k.shape)):
        _need(d_q, "d_q", q.dtype, dev, q.shape)
        _need(d_k, "d_k", q.dtype, dev, k.shape)
    return _backward(d_q, d_k, q, k, inv_freq, positions, q_weight, k_weight, call, int(bool(interleaved)),
                     need_weights, workspace)


def _backward(d_q, d_k, q, k, inv_freq, positions, q_weight, k_weight, call, interleaved, need_weights, workspace):
    """The backward's outputs, scratch and call, after the checks."""
    dev = q.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return _backward(d_q, d_k, q, k, inv_freq, positions, q_weight, k_weight, call, interleaved,
                             need_weights, workspace)
    dq, dk = torch.empty_like(d_q), torch.empty_like(d_k)
    L = _lib.load()
    dwq = dwk = None
    ws_bytes = 0
    if need_weights:
        B, T, Hq, Hk, K = call.sizes[2:7]
        dwq, dwk = torch.empty(K, dtype=torch.float32, device=dev), torch.empty(K, dtype=torch.float32, device=dev)
        need = L.gdn_qk_norm_rotate_bwd_workspace_size(B, T, Hq, Hk, K, 1)
        workspace, ws_bytes = _scratch(need, "gdn_qk_norm_rotate_bwd", workspace, dev)
    elif workspace is not None:
        _need(workspace, "workspace", None, dev)
    st = L.gdn_qk_norm_rotate_bwd(
        d_q.data_ptr(), d_k.data_ptr(), q.data_ptr(), k.data_ptr(),
        *call.args(inv_freq, positions, q_weight, k_weight, interleaved), dq.data_ptr(), dk.data_ptr(), _ptr(dwq),
        _ptr(dwk), _ptr(workspace), ws_bytes, _stream(dev))
    _lib.check("gdn_qk_norm_rotate_bwd", st)
    return dq, dk, dwq, dwk


class _QkNormRotate(torch.autograd.Function):
    """gdn_qk_norm_rotate_fwd forward, gdn_qk_norm_rotate_bwd backward, which does not check again what the
    forward has checked."""

    @staticmethod
    def forward(ctx, q, k, inv_freq, positions, q_weight, k_weight, norm, eps, sections, interleaved):
        _, call = _inputs(q, k, inv_freq, positions, q_weight, k_weight, norm, eps, sections)
        out = _forward(q, k, inv_freq, positions, q_weight, k_weight, call, interleaved)
        ctx.save_for_backward(q, k, inv_freq, positions, q_weight, k_weight)
        ctx.call = call, interleaved
        ctx.strides = q.stride(), k.stride()
        ctx.options = norm, eps, sections
        return out

    @staticmethod
    def backward(ctx, d_q, d_k):
        q, k, inv_freq, positions, q_weight, k_weight = ctx.saved_tensors
        call, interleaved = ctx.call
        if (q.stride(), k.stride()) != ctx.strides:   # (saved elsewhere, they may come back in another layout)
            _, call = _inputs(q, k, inv_freq, positions, q_weight, k_weight, *ctx.options)
        need = ctx.needs_input_grad
        dq, dk, dwq, dwk = _backward(d_q.contiguous(), d_k.contiguous(), q, k, inv_freq, positions, q_weight,
                                     k_weight, call, interleaved, need[4] or need[5], None)
        grads = (dq, dk, dwq.to(q_weight.dtype) if need[4] else None,
                 dwk.to(k_weight.dtype) if need[5] else None)
        if torch.is_grad_enabled():
            grads = _first_only("qk_norm_rotate_trainable", grads, (q, k, q_weight, k_weight, d_q, d_k))
        dq, dk, dwq, dwk = grads
        return dq, dk, None, None, dwq, dwk, None, None, None, None


def qk_norm_rotate_trainable(q, k, inv_freq=None, positions=None, q_weight=None, k_weight=None, *, norm="rms",
                             eps=1e-6, sections=None, interleaved=False):
    """:func:`qk_norm_rotate` as a differentiable op (torch autograd) in q, k, q_weight and k_weight; a
    second derivative is refused.  Captured into a CUDA graph with its backward as
    :func:`gated_linear_recurrence_trainable` says."""
    if inv_freq is not None and inv_freq.requires_grad:
        raise ValueError("inv_freq is a constant of the layer: it has no gradient")
    return _QkNormRotate.apply(q, k, inv_freq, positions, q_weight, k_weight, norm, eps, sections,
                               int(bool(interleaved)))
