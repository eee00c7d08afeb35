"""Plain 64-bit linear attention with a decay for each head: the recurrence token by token, over a
list of sequences, for the tests (CPU or GPU tensors, differentiable)."""
import math

import torch


def bounds(q, cu):
    B, T = q.shape[:2]
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    c = [int(x) for x in cu]
    return [(0, c[n], c[n + 1]) for n in range(len(c) - 1)]


def forward(q, k, v, log_decay, scale=None, h0=None, cu=None):
    """(o, final states) in fp64; h0 [N, Hv, K, V] or None."""
    q, k, v = q.double(), k.double(), v.double()
    rep = v.shape[2] // q.shape[2]
    scale = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    gamma = torch.exp(log_decay.double())[:, None, None]
    o = torch.zeros(v.shape, dtype=torch.float64, device=q.device)
    rows, fins = [], []
    for n, (b, s, e) in enumerate(bounds(q, cu)):
        S = (torch.zeros(v.shape[2], q.shape[3], v.shape[3], dtype=torch.float64, device=q.device)
             if h0 is None else h0[n].double())
        for t in range(s, e):
            kt, qt = (x[b, t].repeat_interleave(rep, 0) for x in (k, q))
            S = gamma * S + kt[:, :, None] * v[b, t][:, None, :]
            rows.append((b, t, scale * (qt[:, None, :] @ S)[:, 0]))
        fins.append(S)
    if rows:
        ib = torch.tensor([r[0] for r in rows], device=q.device)
        it = torch.tensor([r[1] for r in rows], device=q.device)
        o = o.index_put((ib, it), torch.stack([r[2] for r in rows]))
    fin = torch.stack(fins) if fins else torch.zeros(0, v.shape[2], q.shape[3], v.shape[3])
    return o, fin


def rel(x, ref):
    x, ref = x.detach().double().cpu(), ref.detach().double().cpu()
    assert torch.isfinite(x).all()
    n = ref.norm().item()
    return (x - ref).norm().item() / (n if n > 0 else 1.0)
