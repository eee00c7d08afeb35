"""The gated linear recurrence token by token in 64 bits, differentiable."""
import torch


def gates(x, g, i=None, lam=None, c=8.0):
    """a_t and what is added to the state."""
    if lam is None:
        return torch.exp(g), x
    la = -c * torch.nn.functional.softplus(lam) * torch.sigmoid(g)
    # a channel that does not decay: the root is 0, and so is its slope's share of the gradients
    live = la != 0
    root = torch.where(live, torch.sqrt(-torch.expm1(2 * torch.where(live, la, -1.0))), 0.0)
    return torch.exp(la), root * torch.sigmoid(i) * x


def one(a, b, h):
    """One sequence a, b [T, D] from h [D]: (y [T, D], the last state)."""
    ys = []
    for t in range(a.shape[0]):
        h = a[t] * h + b[t]
        ys.append(h)
    return (torch.stack(ys) if ys else a[:0]), h


def recurrence(x, g, i=None, lam=None, c=8.0, h0=None, lens=None):
    """x [B, T, D] (every argument in 64 bits), or [1, T, D] with ``lens``, the packed sequences' lengths
    (tokens behind them: zeros).  Returns (y, final states [N, D])."""
    a, b = gates(x, g, i, lam, c)
    B, T, D = x.shape
    spans = [(r, 0, T) for r in range(B)]
    if lens is not None:
        spans, at = [], 0
        for n in lens:
            spans.append((0, at, at + n))
            at += n
    ys, fins = [], []
    for n, (r, t0, t1) in enumerate(spans):
        y, fin = one(a[r, t0:t1], b[r, t0:t1], x.new_zeros(D) if h0 is None else h0[n])
        ys.append(y)
        fins.append(fin)
    fin = torch.stack(fins) if fins else x.new_zeros(0, D)
    if lens is None:
        return torch.stack(ys), fin
    return torch.cat(ys + [x.new_zeros(T - sum(lens), D)])[None], fin
