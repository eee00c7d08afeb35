"""Group norm with an activation, channels last: the PyTorch binding of ``gdn_group_norm_act_*``.

For each row and group of C / G channels, mean and (biased) variance over the positions and the
group's channels; ``u`` is the normalised, scaled and shifted value, and

    y = act(u)              without a gate,
    y = u * act(gate)       with one.
"""
from __future__ import annotations

import torch

from . import _lib
from .api import _DT, _need, _ptr
from .linear_attn import _first_only, _fit, _incoming, _int32, _scratch, _stream

__all__ = ["group_norm_act", "group_norm_act_bwd", "group_norm_act_trainable"]

_ACT = {None: _lib.GDN_ACT_NONE, "none": _lib.GDN_ACT_NONE, "silu": _lib.GDN_ACT_SILU}


def _inputs(x, num_groups, weight, bias, activation, gate):
    """Checks shared by the calls; returns (N, L, C, G, wb dtype code, act code)."""
    quick = (isinstance(x, torch.Tensor) and x.is_cuda and x.dim() >= 2 and x.dtype in _DT
             and x.is_contiguous())
    if not quick:
        _need(x, "x", (torch.float32, torch.bfloat16))
    if x.dim() < 2:
        raise ValueError("x must be [N, ..., C]")
    N, C, G = x.shape[0], x.shape[-1], int(num_groups)
    if G < 1 or C < 1 or C % G:
        raise ValueError("%d channels do not split into %d groups" % (C, G))
    if activation not in _ACT:
        raise ValueError("activation must be None or 'silu' (got %r)" % (activation,))
    L = 1
    for s in x.shape[1:-1]:
        L *= s
    _int32("group norm", N, L, C)
    if quick:
        wb = weight.dtype if isinstance(weight, torch.Tensor) else \
            bias.dtype if isinstance(bias, torch.Tensor) else torch.float32
        if (wb is torch.float32 or wb is x.dtype) and \
                _fit(x.device, (weight, wb, (C,)), (bias, wb, (C,)), (gate, x.dtype, x.shape)):
            return N, L, C, G, _DT[wb], _ACT[activation]
    wb = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _need(t, name, (x.dtype, torch.float32) if wb is None else wb, x.device, (C,))
            wb = t.dtype
    if gate is not None:
        _need(gate, "gate", x.dtype, x.device, x.shape)
    return N, L, C, G, _DT[wb or torch.float32], _ACT[activation]


def group_norm_act(x, num_groups, weight=None, bias=None, eps=1e-5, activation="silu", gate=None, *,
                   out=None, return_stats=False, workspace=None):
    """Forward through ``gdn_group_norm_act_fwd``.

    x [N, ..., C] contiguous (channels last; the middle dims are the positions, and x [N, C]
    normalises each row by itself, as behind linear attention: N tokens, C = H V, G = H);
    weight, bias [C] in fp32 or x's dtype, or None; activation "silu" or None; gate like x or
    None.  Returns y, or ``(y, mean, rstd)`` with ``return_stats`` (both [N, G] fp32, what
    :func:`group_norm_act_bwd` takes).
    """
    N, L, C, G, wb, act = _inputs(x, num_groups, weight, bias, activation, gate)
    dev = x.device
    if out is None:
        out = torch.empty_like(x)
    elif not _fit(dev, (out, x.dtype, x.shape)):
        _need(out, "out", x.dtype, dev, x.shape)
    mean = rstd = None
    if return_stats:
        make = torch.empty if L else torch.zeros
        mean = make((N, G), dtype=torch.float32, device=dev)
        rstd = make((N, G), dtype=torch.float32, device=dev)
    lib = _lib.load()
    need = lib.gdn_group_norm_act_fwd_workspace_size(N, L, C, G, _DT[x.dtype])
    workspace, ws_bytes = _scratch(need, "gdn_group_norm_act_fwd", workspace, dev)
    st = lib.gdn_group_norm_act_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), N, L, C, G,
                                    _DT[x.dtype], wb, float(eps), act, _ptr(out), _ptr(mean),
                                    _ptr(rstd), _ptr(workspace), ws_bytes, _stream(dev))
    _lib.check("gdn_group_norm_act_fwd", st)
    return (out, mean, rstd) if return_stats else out


def group_norm_act_bwd(dy, x, mean, rstd, num_groups, weight=None, bias=None, activation="silu",
                       gate=None, *, need_params=True, workspace=None):
    """Gradients of :func:`group_norm_act` through ``gdn_group_norm_act_bwd``: ``(dx, dweight,
    dbias, dgate)``, dx and dgate in x's dtype, dweight and dbias fp32 [C] (None without
    ``need_params``), dgate None without a gate."""
    N, L, C, G, wb, act = _inputs(x, num_groups, weight, bias, activation, gate)
    dev = x.device
    if dy is None or mean is None or rstd is None or not _fit(
            dev, (dy, x.dtype, x.shape), (mean, torch.float32, (N, G)), (rstd, torch.float32, (N, G))):
        _need(dy, "dy", x.dtype, dev, x.shape)
        _need(mean, "mean", torch.float32, dev, (N, G))
        _need(rstd, "rstd", torch.float32, dev, (N, G))
    return _backward(dy, x, _ptr(mean), _ptr(rstd), (N, L, C, G, wb, act), weight, bias, gate,
                     need_params, workspace)


def _backward(dy, x, mean, rstd, sizes, weight, bias, gate, need_params, workspace):
    """The backward's outputs, scratch and call; mean, rstd as addresses."""
    N, L, C, G, wb, act = sizes
    dev = x.device
    dx = torch.empty_like(x)
    dgate = None if gate is None else torch.empty_like(x)
    dw = db = None
    if need_params:
        dw = torch.empty(C, dtype=torch.float32, device=dev)
        db = torch.empty(C, dtype=torch.float32, device=dev)
    lib = _lib.load()
    need = lib.gdn_group_norm_act_bwd_workspace_size(N, L, C, G, _DT[x.dtype])
    workspace, ws_bytes = _scratch(need, "gdn_group_norm_act_bwd", workspace, dev)
    st = lib.gdn_group_norm_act_bwd(_ptr(dy), _ptr(x), _ptr(weight), _ptr(bias), _ptr(gate),
                                    mean, rstd, N, L, C, G, _DT[x.dtype], wb, act, _ptr(dx),
                                    _ptr(dgate), _ptr(dw), _ptr(db), _ptr(workspace), ws_bytes,
                                    _stream(dev))
    _lib.check("gdn_group_norm_act_bwd", st)
    return dx, dw, db, dgate


class _GroupNormAct(torch.autograd.Function):
    """gdn_group_norm_act_fwd forward, gdn_group_norm_act_bwd backward.  (For small inputs the
    host's part is most of both: mean, rstd and the forward's scratch share one allocation, and the
    backward does not check again what the forward has checked.)"""

    @staticmethod
    def forward(ctx, x, num_groups, weight, bias, eps, activation, gate):
        sizes = N, L, C, G, wb, act = _inputs(x, num_groups, weight, bias, activation, gate)
        dev = x.device
        lib = _lib.load()
        need = lib.gdn_group_norm_act_fwd_workspace_size(N, L, C, G, _DT[x.dtype])
        if need == (1 << 64) - 1:
            raise ValueError("sizes rejected by gdn_group_norm_act_fwd")
        y = torch.empty_like(x)
        at = (8 * N * G + 255) // 256 * 256      # where the scratch starts
        stats = torch.empty(at + need, dtype=torch.uint8, device=dev)
        mean = stats.data_ptr()
        st = lib.gdn_group_norm_act_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), N, L, C, G,
                                        _DT[x.dtype], wb, float(eps), act, _ptr(y), mean,
                                        mean + 4 * N * G, mean + at if need else None, need,
                                        _stream(dev))
        _lib.check("gdn_group_norm_act_fwd", st)
        ctx.save_for_backward(x, weight, bias, gate, stats)
        ctx.sizes = sizes
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, gate, stats = ctx.saved_tensors
        need, sizes = ctx.needs_input_grad, ctx.sizes
        dy = _incoming(dy)
        if not _fit(x.device, (dy, x.dtype, x.shape)):
            _need(dy, "dy", x.dtype, x.device, x.shape)
        mean = stats.data_ptr()
        dx, dw, db, dgate = _backward(dy, x, mean, mean + 4 * sizes[0] * sizes[3], sizes, weight,
                                      bias, gate, need[2] or need[3], None)
        grads = (dx, dw.to(weight.dtype) if need[2] else None, db.to(bias.dtype) if need[3] else None,
                 dgate)
        if torch.is_grad_enabled():
            grads = _first_only("group_norm_act_trainable", grads, (x, weight, bias, gate, dy))
        dx, dw, db, dgate = grads
        return dx, None, dw, db, None, None, dgate


def group_norm_act_trainable(x, num_groups, weight=None, bias=None, eps=1e-5, activation="silu",
                             gate=None):
    """:func:`group_norm_act` as a differentiable op (torch autograd) in x, weight, bias, gate; a second
    derivative is refused."""
    return _GroupNormAct.apply(x, num_groups, weight, bias, eps, activation, gate)
