"""Gated linear recurrence: the PyTorch binding of the ``gdn_linear_recurrence_*`` entry points.

    h_t = a_t h_{t-1} + b_t,    y_t = h_t      per channel, with an fp32 state h [N, D]

gates given:  a_t = exp(g_t), b_t = x_t;
fused gates:  a_t = exp(-c softplus(lam) sigmoid(r_t)), b_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t.

x, g, r, i may be slices of a wider projection along the last axis: their rows need not be next to
each other.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .api import DEVICE_ERRORS_DOC, _DT, _need, _ptr, _raise_on_status, _status
from .linear_attn import _first_only, _fit, _int32, _scratch, _stream

__all__ = ["gated_linear_recurrence", "gated_linear_recurrence_fused_gates",
           "gated_linear_recurrence_bwd", "gated_linear_recurrence_bwd_fused_gates",
           "gated_linear_recurrence_trainable", "gated_linear_recurrence_fused_gates_trainable",
           "gated_linear_recurrence_decode", "gated_linear_recurrence_decode_fused_gates"]


def _elsewhere(dev) -> bool:
    """Whether the tensors' device is not the current one, which launches and their plans go by."""
    return torch._C._cuda_getDevice() != dev.index


def _pitch(t, name, dtype, dev, shape):
    """Elements from one token of t to the next, after the checks: t [..., D] of ``shape`` whose rows
    are evenly spaced over all its leading axes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != dev:
        if t.device.type != "cuda":
            raise ValueError("%s must be a CUDA tensor (got %s)" % (name, t.device))
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    D = shape[-1]
    if t.is_contiguous():
        return D
    pitch, tokens = None, 1
    for size, stride in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if pitch is None:
            pitch = stride
        elif stride != pitch * tokens:
            raise ValueError("%s must have evenly spaced rows" % name)
        tokens *= size
    if (D > 1 and t.stride(-1) != 1) or (pitch is not None and pitch < D):
        raise ValueError("%s must have contiguous rows that do not overlap" % name)
    return D if pitch is None else pitch


def _inputs(x, g, i, lam, c, dims, g_name):
    """Checks shared by the calls; returns (device, (x, g, i pitches), c)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.device.type != "cuda":
        raise ValueError("x must be a CUDA tensor (got %s)" % x.device)
    if x.dim() != dims:
        raise ValueError("x must be %s" % ("[B, T, D]" if dims == 3 else "[n, D]"))
    dev, shape = x.device, x.shape
    if not 1 <= shape[-1] <= 1 << 28:
        raise ValueError("x needs 1 to 2^28 channels (got %d)" % shape[-1])
    _int32("gated linear recurrence", *shape)
    px = _pitch(x, "x", (torch.float32, torch.bfloat16), dev, shape)
    pg = _pitch(g, g_name, (x.dtype, torch.float32), dev, shape)
    if lam is None:
        return dev, (px, pg, 0), 0.0
    pi = _pitch(i, "i", g.dtype, dev, shape)
    if not _fit(dev, (lam, torch.float32, shape[-1:])):
        _need(lam, "lam", torch.float32, dev, shape[-1:])
    c = float(c)
    if not 0.0 <= c <= 3.0e38:
        raise ValueError("c must be finite and not negative (got %r)" % c)
    return dev, (px, pg, pi), c


def _sequences(x, cu_seqlens):
    """The number of sequences."""
    if cu_seqlens is None:
        return x.shape[0]
    _need(cu_seqlens, "cu_seqlens", torch.int32, x.device)
    if x.shape[0] != 1:
        raise ValueError("cu_seqlens requires B == 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [num_seqs + 1]")
    if cu_seqlens.numel() - 1 > 1 << 30:
        raise ValueError("cu_seqlens packs at most 2^30 sequences (got %d)" % (cu_seqlens.numel() - 1))
    return cu_seqlens.numel() - 1


def _forward(x, g, i, lam, c, initial_state, output_final_state, cu_seqlens, state_indices, out,
             final_state, return_carries, workspace, dev_status, check, g_name):
    """Checks and the forward's call: (y, final state, carries, (c, pitches, number of sequences))."""
    dev, pitches, c = _inputs(x, g, i, lam, c, 3, g_name)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return _forward(x, g, i, lam, c, initial_state, output_final_state, cu_seqlens, state_indices, out,
                            final_state, return_carries, workspace, dev_status, check, g_name)
    B, T, D = x.shape
    N = _sequences(x, cu_seqlens)
    num_slots = 0
    st_shape = (N, D)
    if state_indices is not None:
        _need(state_indices, "state_indices", torch.int32, dev, (N,))
        cache = initial_state if initial_state is not None else final_state
        if cache is None:
            raise ValueError("state_indices needs initial_state or final_state (the slot cache)")
        num_slots = cache.shape[0]
        _int32("gated linear recurrence", num_slots)
        st_shape = (num_slots, D)
        if output_final_state and final_state is None:
            final_state = initial_state
    if not output_final_state:
        final_state = None
    if not _fit(dev, (initial_state, torch.float32, st_shape), (final_state, torch.float32, st_shape),
                (out, x.dtype, x.shape)):
        for t, name in ((initial_state, "initial_state"), (final_state, "final_state")):
            if t is not None:
                _need(t, name, torch.float32, dev, st_shape)
        if out is not None:
            _need(out, "out", x.dtype, dev, x.shape)
    if output_final_state and final_state is None:
        final_state = torch.empty(st_shape, dtype=torch.float32, device=dev)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    L = _lib.load()
    carries = None
    if return_carries:
        need = L.gdn_linear_recurrence_carries_size(B, T, D)
        if need == (1 << 64) - 1:
            raise ValueError("sizes rejected by gdn_linear_recurrence_fwd")
        carries = torch.empty((need // (4 * D), D), dtype=torch.float32, device=dev)
    need = L.gdn_linear_recurrence_fwd_workspace_size(B, T, D, N)
    workspace, ws_bytes = _scratch(need, "gdn_linear_recurrence_fwd", workspace, dev)
    dev_status = _status(dev_status, check, dev)
    st = L.gdn_linear_recurrence_fwd(_ptr(x), _ptr(g), _ptr(i), _ptr(lam), c, *pitches, B, T, D,
                                     _DT[x.dtype], _DT[g.dtype], _ptr(initial_state),
                                     int(bool(output_final_state)), _ptr(final_state), _ptr(cu_seqlens),
                                     N, _ptr(state_indices), num_slots, _ptr(out), _ptr(carries),
                                     _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(dev))
    _lib.check("gdn_linear_recurrence_fwd", st)
    _raise_on_status("gdn_linear_recurrence_fwd", dev_status, check)
    return out, final_state, carries, (c, pitches, N)


def gated_linear_recurrence(x, g, initial_state=None, output_final_state=False, cu_seqlens=None, *,
                            state_indices=None, out=None, final_state=None, return_carries=False,
                            workspace=None, dev_status=None, check=False
                            ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Forward through ``gdn_linear_recurrence_fwd`` with given log-decays g (at most 0).

    x [B, T, D]; g [B, T, D] in fp32 or x's dtype.  Returns ``(y, final_state or None)``, and with
    ``return_carries`` also what :func:`gated_linear_recurrence_bwd` starts from.  Also with a slot
    cache ``state_indices`` [N] (-1 = padding) on states [num_slots, D], ``cu_seqlens``, ``out``,
    ``final_state``, ``workspace``, ``dev_status`` and ``check`` as in :func:`chunk_gated_delta_rule`; a bad
    ``cu_seqlens`` leaves zero rows and every state as it was.
    """
    y, fin, carries, _ = _forward(x, g, None, None, 0.0, initial_state, output_final_state, cu_seqlens,
                               state_indices, out, final_state, return_carries, workspace, dev_status, check, "g")
    return (y, fin, carries) if return_carries else (y, fin)


def gated_linear_recurrence_fused_gates(x, r, i, lam, c=8.0, initial_state=None, output_final_state=False,
                                        cu_seqlens=None, *, state_indices=None, out=None, final_state=None,
                                        return_carries=False, workspace=None, dev_status=None, check=False
                                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """:func:`gated_linear_recurrence` with its gates computed in the kernel: r, i [B, T, D] in fp32 or
    x's dtype, lam [D] fp32, c a constant of the layer."""
    _need(lam, "lam")
    y, fin, carries, _ = _forward(x, r, i, lam, c, initial_state, output_final_state, cu_seqlens, state_indices,
                               out, final_state, return_carries, workspace, dev_status, check, "r")
    return (y, fin, carries) if return_carries else (y, fin)


def _backward(x, g, i, lam, c, d_y, d_final_state, initial_state, cu_seqlens, need_lam,
              need_d_initial_state, carries, workspace, dev_status, check, g_name):
    dev, pitches, c = _inputs(x, g, i, lam, c, 3, g_name)
    B, T, D = x.shape
    N = _sequences(x, cu_seqlens)
    if d_y is None or not _fit(dev, (d_y, x.dtype, x.shape), (initial_state, torch.float32, (N, D)),
                               (d_final_state, torch.float32, (N, D)),
                               (carries, torch.float32, (-(-B * T // 32), D))):
        _need(d_y, "d_y", x.dtype, dev, x.shape)
        for t, name in ((initial_state, "initial_state"), (d_final_state, "d_final_state")):
            if t is not None:
                _need(t, name, torch.float32, dev, (N, D))
        if carries is not None:
            _need(carries, "carries", torch.float32, dev, (-(-B * T // 32), D))
    dev_status = _status(dev_status, check, dev)
    grads = _gradients(x, g, i, lam, c, pitches, N, d_y, d_final_state, initial_state, cu_seqlens, need_lam,
                       need_d_initial_state, carries, workspace, dev_status)
    _raise_on_status("gdn_linear_recurrence_bwd", dev_status, check)
    return grads


def _gradients(x, g, i, lam, c, pitches, N, d_y, d_final_state, initial_state, cu_seqlens, need_lam,
               need_d_initial_state, carries, workspace, dev_status):
    """The backward's outputs, scratch and call, after the checks."""
    dev = x.device
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return _gradients(x, g, i, lam, c, pitches, N, d_y, d_final_state, initial_state, cu_seqlens, need_lam,
                              need_d_initial_state, carries, workspace, dev_status)
    B, T, D = x.shape
    L = _lib.load()
    need = L.gdn_linear_recurrence_bwd_workspace_size(B, T, D, N, int(lam is not None))
    workspace, ws_bytes = _scratch(need, "gdn_linear_recurrence_bwd", workspace, dev)
    dx = torch.empty_like(d_y)
    dg = torch.empty_like(d_y, dtype=g.dtype)
    di = dlam = dh0 = None
    if lam is not None:
        di = torch.empty_like(dg)
        if need_lam:
            dlam = torch.empty_like(lam)
    if need_d_initial_state:
        dh0 = torch.empty((N, D), dtype=torch.float32, device=dev)
    st = L.gdn_linear_recurrence_bwd(_ptr(x), _ptr(g), _ptr(i), _ptr(lam), c, *pitches, B, T, D,
                                     _DT[x.dtype], _DT[g.dtype], _ptr(initial_state), _ptr(cu_seqlens), N,
                                     _ptr(d_y), _ptr(d_final_state), _ptr(carries), _ptr(dx), _ptr(dg),
                                     _ptr(di), _ptr(dlam), _ptr(dh0), _ptr(workspace), ws_bytes,
                                     _ptr(dev_status), _stream(dev))
    _lib.check("gdn_linear_recurrence_bwd", st)
    return dx, dg, di, dlam, dh0


def gated_linear_recurrence_bwd(x, g, d_y, d_final_state=None, initial_state=None, cu_seqlens=None, *,
                                need_d_initial_state=True, carries=None, workspace=None, dev_status=None,
                                check=False):
    """Gradients of :func:`gated_linear_recurrence` (no slot cache) through
    ``gdn_linear_recurrence_bwd``: ``(dx, dg, d_initial_state)``, each in its input's dtype, the last
    fp32 [N, D] (None when ``need_d_initial_state`` is False).  Without ``carries`` of the same inputs'
    forward they are made again."""
    dx, dg, _, _, dh0 = _backward(x, g, None, None, 0.0, d_y, d_final_state, initial_state, cu_seqlens, False,
                                  need_d_initial_state, carries, workspace, dev_status, check, "g")
    return dx, dg, dh0


def gated_linear_recurrence_bwd_fused_gates(x, r, i, lam, d_y, d_final_state=None, c=8.0, initial_state=None,
                                            cu_seqlens=None, *, need_d_initial_state=True, carries=None,
                                            workspace=None, dev_status=None, check=False):
    """Gradients of :func:`gated_linear_recurrence_fused_gates`: ``(dx, dr, di, dlam,
    d_initial_state)``, dlam fp32 [D]."""
    _need(lam, "lam")
    return _backward(x, r, i, lam, c, d_y, d_final_state, initial_state, cu_seqlens, True,
                     need_d_initial_state, carries, workspace, dev_status, check, "r")


def _strides(*ts):
    return [None if t is None else t.stride() for t in ts]


class _Recurrence(torch.autograd.Function):
    """gdn_linear_recurrence_fwd forward, gdn_linear_recurrence_bwd backward, which does not check again what
    the forward has checked."""

    @staticmethod
    def forward(ctx, x, g, i, lam, initial_state, c, output_final_state, cu_seqlens):
        y, fin, carries, call = _forward(x, g, i, lam, c, initial_state, output_final_state, cu_seqlens, None,
                                         None, None, any(ctx.needs_input_grad), None, None, False,
                                         "g" if lam is None else "r")
        ctx.save_for_backward(x, g, i, lam, initial_state, cu_seqlens, carries)
        ctx.call = call
        ctx.strides = _strides(x, g, i)
        ctx.set_materialize_grads(False)
        return y, fin

    @staticmethod
    def backward(ctx, d_y, d_fin):
        x, g, i, lam, init, cu, carries = ctx.saved_tensors
        c, pitches, N = ctx.call
        if _strides(x, g, i) != ctx.strides:   # (tensors that were saved elsewhere may come back in another layout)
            _, pitches, _ = _inputs(x, g, i, lam, c, 3, "g")
        need = ctx.needs_input_grad
        d_y = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if d_y is None else d_y.contiguous()
        if d_fin is not None:
            d_fin = d_fin.contiguous()
        grads = _gradients(x, g, i, lam, c, pitches, N, d_y, d_fin, init, cu, need[3], init is not None and need[4],
                           carries, None, None)
        if torch.is_grad_enabled():
            grads = _first_only("gated_linear_recurrence_trainable", grads, (x, g, i, lam, init, d_y, d_fin))
        return (*grads, None, None, None)


def gated_linear_recurrence_trainable(x, g, initial_state=None, output_final_state=False, cu_seqlens=None):
    """:func:`gated_linear_recurrence` as a differentiable op (torch autograd) in x, g and
    ``initial_state``; a second derivative is refused.  Returns ``(y, final_state or None)``.

    To capture a step with its backward into a CUDA graph, let no graph of an eager call on the same leaves be alive:
    autograd's engine would join the captured stream to the eager one, and the capture fails.
    """
    return _Recurrence.apply(x, g, None, None, initial_state, 0.0, bool(output_final_state), cu_seqlens)


def gated_linear_recurrence_fused_gates_trainable(x, r, i, lam, c=8.0, initial_state=None,
                                                  output_final_state=False, cu_seqlens=None):
    """:func:`gated_linear_recurrence_fused_gates` as a differentiable op in x, r, i, lam and
    ``initial_state``; a second derivative is refused.  Returns ``(y, final_state or None)``; captured as
    :func:`gated_linear_recurrence_trainable` says."""
    _need(lam, "lam")
    return _Recurrence.apply(x, r, i, lam, initial_state, float(c), bool(output_final_state), cu_seqlens)


def _decode(x, g, i, lam, c, state, batch_indices, out, dev_status, check, g_name):
    dev, pitches, c = _inputs(x, g, i, lam, c, 2, g_name)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return _decode(x, g, i, lam, c, state, batch_indices, out, dev_status, check, g_name)
    n, D = x.shape
    if not (isinstance(state, torch.Tensor) and state.dim() == 2
            and _fit(dev, (state, torch.float32, (state.shape[0], D)), (batch_indices, torch.int32, (n,)),
                     (out, x.dtype, x.shape))):
        _need(state, "state", torch.float32, dev)
        if state.dim() != 2 or state.shape[1] != D:
            raise ValueError("state must be [num_slots, D]")
        if batch_indices is not None:
            _need(batch_indices, "batch_indices", torch.int32, dev, (n,))
        if out is not None:
            _need(out, "out", x.dtype, dev, x.shape)
    _int32("gated linear recurrence", state.shape[0])
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dev_status = _status(dev_status, check, dev)
    st = _lib.load().gdn_linear_recurrence_decode(_ptr(x), _ptr(g), _ptr(i), _ptr(lam), c, *pitches, n, D,
                                                  _DT[x.dtype], _DT[g.dtype], _ptr(state), state.shape[0],
                                                  _ptr(batch_indices), _ptr(out), _ptr(dev_status),
                                                  _stream(dev))
    _lib.check("gdn_linear_recurrence_decode", st)
    _raise_on_status("gdn_linear_recurrence_decode", dev_status, check)
    return out


def gated_linear_recurrence_decode(x, g, state, batch_indices=None, *, out=None, dev_status=None,
                                   check=False) -> torch.Tensor:
    """One token per request through ``gdn_linear_recurrence_decode``; ``state`` [num_slots, D] fp32 is
    updated in place.

    x [n, D]; g [n, D] in fp32 or x's dtype; batch_indices [n] int32 (-1 = padding: a zero row) or
    None (request i uses slot i).  Returns y [n, D].
    """
    return _decode(x, g, None, None, 0.0, state, batch_indices, out, dev_status, check, "g")


def gated_linear_recurrence_decode_fused_gates(x, r, i, lam, state, batch_indices=None, c=8.0, *, out=None,
                                               dev_status=None, check=False) -> torch.Tensor:
    """:func:`gated_linear_recurrence_decode` with its gates computed in the kernel: r, i [n, D], lam [D]."""
    _need(lam, "lam")
    return _decode(x, r, i, lam, c, state, batch_indices, out, dev_status, check, "r")


for _f in (gated_linear_recurrence, gated_linear_recurrence_fused_gates, gated_linear_recurrence_bwd,
           gated_linear_recurrence_bwd_fused_gates, gated_linear_recurrence_decode,
           gated_linear_recurrence_decode_fused_gates):
    _f.__doc__ += DEVICE_ERRORS_DOC
