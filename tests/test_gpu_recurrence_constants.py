"""The gated linear recurrence with other constants c than 8, which forward, backward, decode and the autograd op
each take by themselves, and decode of every request in its own slot; against the 64-bit recurrence, tolerances
as in test_gpu_recurrence."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from tests.recurrence_ref import recurrence
from tests.test_gpu_recurrence import BF16, F32, TOL, backward, forward, make, rel, seeded, tol  # noqa: F401

pytestmark = pytest.mark.gpu
NAMES = ("dx", "dr", "di", "dlam", "dh0")


def reference(ins, c, h0, lens=None, dy=None, dfin=None):
    leaves = [t.detach().double().requires_grad_() for t in (*ins, h0)]
    y, fin = recurrence(*leaves[:4], c=c, h0=leaves[4], lens=lens)
    if dy is None:
        return y, fin
    return y, fin, torch.autograd.grad((y * dy.double()).sum() + (fin * dfin.double()).sum(), leaves)


@pytest.mark.parametrize("dtype,gdt", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("c", [0.5, 1.0, 8.0, 20.0])
@pytest.mark.parametrize("lens", [None, [3, 0, 170, 1]])
def test_forward_backward_and_autograd(lens, c, dtype, gdt):
    B, T = (2, 150) if lens is None else (1, sum(lens) + 5)
    N = B if lens is None else len(lens)
    ins = make((B, T, 72), dtype, gdt, fused=True)
    h0, dfin, dy = torch.randn(N, 72, device="cuda"), torch.randn(N, 72, device="cuda"), torch.randn_like(ins[0])
    kw = {}
    if lens is not None:
        kw["cu_seqlens"] = torch.tensor([sum(lens[:n]) for n in range(N + 1)], dtype=torch.int32, device="cuda")
    y, fin, grads = reference(ins, c, h0, lens, dy, dfin)
    got, got_fin, carries = forward(ins, c=c, initial_state=h0, output_final_state=True, return_carries=True, **kw)
    assert rel(got, y) <= tol(got) and rel(got_fin, fin) <= TOL[F32]
    for saved in (carries, None):
        have = backward(ins, dy, d_final_state=dfin, c=c, initial_state=h0, carries=saved, **kw)
        for name, a, b in zip(NAMES, have, grads):
            assert rel(a, b) <= tol(a), name
    leaves = [t.requires_grad_() for t in (*ins, h0)]
    y2, fin2 = gdn.gated_linear_recurrence_fused_gates_trainable(*leaves[:4], c, initial_state=h0,
                                                                 output_final_state=True, **kw)
    assert torch.equal(y2, got) and torch.equal(fin2, got_fin)
    for name, a, b in zip(NAMES, torch.autograd.grad((y2, fin2), leaves, (dy, dfin)), have):
        assert torch.equal(a, b), name


def test_in_segments():
    """One chain that is cut: every launch of it has the constant."""
    ins, c = make((1, 9000, 24), F32, fused=True), 2.0
    h0, dfin, dy = torch.randn(1, 24, device="cuda"), torch.randn(1, 24, device="cuda"), torch.randn_like(ins[0])
    y, fin, grads = reference(ins, c, h0, None, dy, dfin)
    got, got_fin = forward(ins, c=c, initial_state=h0, output_final_state=True)
    assert rel(got, y) <= TOL[F32] and rel(got_fin, fin) <= TOL[F32]
    for name, a, b in zip(NAMES, backward(ins, dy, d_final_state=dfin, c=c, initial_state=h0), grads):
        assert rel(a, b) <= TOL[F32], name


@pytest.mark.parametrize("dtype,gdt", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("c", [None, 0.5, 8.0, 20.0])
@pytest.mark.parametrize("n,D", [(1, 5), (7, 33), (64, 512), (300, 12)])
def test_decode_in_the_requests_own_slots(n, D, c, dtype, gdt):
    """No batch_indices: request i in slot i, slots behind them untouched.  (c None: gates given.)  Two terms, each off
    by a few 2^-24 of itself: 1e-6 of their sizes; the output is rounded once more."""
    ins = make((n, D), dtype, gdt, fused=c is not None, seed=n)
    cache = torch.randn(n + 2, D, device="cuda")
    before = cache.clone()
    if c is None:
        y = gdn.gated_linear_recurrence_decode(*ins, cache)
    else:
        y = gdn.gated_linear_recurrence_decode_fused_gates(*ins, cache, None, c)
    rows = [t.double()[:, None] if t.dim() == 2 else t.double() for t in ins]
    args = dict(c=8.0 if c is None else c)
    want, fin = recurrence(*rows, h0=before[:n].double(), **args)
    _, size = recurrence(rows[0].abs(), *rows[1:], h0=before[:n].double().abs(), **args)
    assert ((cache[:n].double() - fin).abs() <= 1e-6 * size).all()
    half = 2.0 ** -8 if dtype is BF16 else 2.0 ** -24
    assert ((y.double() - want[:, 0]).abs() <= 1e-6 * size + half * want[:, 0].abs()).all()
    assert torch.equal(cache[n:], before[n:])
    # and what the same slots give by their numbers
    again = before.clone()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    if c is None:
        y2 = gdn.gated_linear_recurrence_decode(*ins, again, slots)
    else:
        y2 = gdn.gated_linear_recurrence_decode_fused_gates(*ins, again, slots, c)
    assert torch.equal(y2, y) and torch.equal(again, cache)
