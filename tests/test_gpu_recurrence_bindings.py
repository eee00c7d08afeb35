"""The gated linear recurrence's and the q / k norm's bindings where tensors and calls are unlike the usual:
gradients that start at any element, tensors saved elsewhere, sizes beyond 31 bits, two calls at once."""
import threading

import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from tests.test_gpu_recurrence import BF16, F32, backward, forward, make
from tests.test_gpu_qk_rotate import freqs

pytestmark = pytest.mark.gpu


def shifted(t):
    """t, contiguous, one element behind where an allocation starts."""
    room = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    return room[1:].view(t.shape).copy_(t)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fused", [False, True])
def test_gradients_at_any_element(fused, dtype):
    ins = make((2, 200, 64), dtype, fused=fused)
    dy, h0, dfin = torch.randn_like(ins[0]), torch.randn(2, 64, device="cuda"), torch.randn(2, 64, device="cuda")
    kw = dict(d_final_state=dfin, initial_state=h0)
    want = backward(ins, dy, **kw)
    for a, b in zip(backward(ins, shifted(dy), d_final_state=shifted(dfin), initial_state=shifted(h0)), want):
        assert torch.equal(a, b)
    y, _ = forward(ins, out=shifted(dy))
    assert torch.equal(y, forward(ins)[0])
    moved = [shifted(t) for t in ins]
    assert all(torch.equal(a, b) for a, b in zip(backward(moved, dy, **kw), want))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotated_gradients_at_any_element(dtype):
    q, k = torch.randn(2, 50, 4, 64, device="cuda").to(dtype), torch.randn(2, 50, 2, 64, device="cuda").to(dtype)
    w, freq = torch.rand(64, device="cuda"), freqs(64)
    run = lambda dq, dk: gdn.qk_norm_rotate_bwd(dq, dk, q, k, freq, None, w, w)
    # (narrower vectors sum a head's squares in another order)
    want, got = run(q, k), run(shifted(q), shifted(k))
    tol = 2.0 ** -7 if dtype is BF16 else 2e-6
    for a, b in zip(got, want):
        a, b = a.double(), b.double()
        assert ((a - b).norm() / b.norm()).item() <= (tol if a.dim() > 1 else 1e-5)


def test_tensors_saved_elsewhere():
    """Saved tensors that come back in another layout: parts of a projection as tensors of their own."""
    lam = torch.linspace(-6, -3, 40, device="cuda")
    proj = torch.randn(2, 300, 120, device="cuda").to(BF16).requires_grad_()
    heads = torch.randn(2, 300, 6, 32, device="cuda").to(BF16).requires_grad_()
    freq = freqs(32)

    def grads():
        y, _ = gdn.gated_linear_recurrence_fused_gates_trainable(*proj.split(40, -1), lam)
        a, b = gdn.qk_norm_rotate_trainable(heads[:, :, :4], heads[:, :, 4:], freq)
        return torch.autograd.grad(y.sum() + (a[..., 0].sum() - b[..., 3].sum()), (proj, heads))
    want = grads()
    with torch.autograd.graph.save_on_cpu():
        got = grads()
    for a, b in zip(got, want):
        a, b = a.double(), b.double()
        assert ((a - b).norm() / b.norm()).item() <= 2.0 ** -7


def test_sizes_beyond_31_bits():
    if torch.cuda.mem_get_info()[0] < 3 << 32:
        pytest.skip("not enough free memory")
    x = torch.empty(1, (1 << 31) + 64, 1, dtype=BF16, device="cuda")
    for call in (lambda: gdn.gated_linear_recurrence(x, x), lambda: gdn.gated_linear_recurrence_trainable(x, x),
                 lambda: gdn.gated_linear_recurrence_bwd(x, x, x),
                 lambda: gdn.qk_norm_rotate(x[..., None], x[..., None]),
                 lambda: gdn.qk_norm_rotate_bwd(x[..., None], x[..., None], x[..., None], x[..., None])):
        with pytest.raises(ValueError, match="sizes"):
            call()


def test_two_calls_at_once():
    """Threads with streams of their own, on the same inputs."""
    ins = make((1, 4000, 64), BF16, fused=True)
    dy = torch.randn_like(ins[0])
    q, k = torch.randn(1, 500, 8, 64, device="cuda").to(BF16), torch.randn(1, 500, 2, 64, device="cuda").to(BF16)
    freq, w = freqs(64), torch.rand(64, device="cuda")

    def run():
        return (forward(ins, output_final_state=True) + tuple(backward(ins, dy, need_d_initial_state=False)[:-1])
                + gdn.qk_norm_rotate(q, k, freq, None, w, w) + gdn.qk_norm_rotate_bwd(q, k, q, k, freq, None, w, w))
    want = run()
    torch.cuda.synchronize()
    results = {}

    def work(n):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            results[n] = [run() for _ in range(10)]
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(results) == 2
    for runs in results.values():
        for got in runs:
            assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_widest_rows():
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("not enough free memory")
    x = torch.empty(1, (1 << 28) + 1, dtype=BF16, device="cuda")
    state = torch.empty(1, 1, device="cuda")
    for call in (lambda: gdn.gated_linear_recurrence(x[None], x[None]),
                 lambda: gdn.gated_linear_recurrence_bwd(x[None], x[None], x[None]),
                 lambda: gdn.gated_linear_recurrence_decode(x, x, state)):
        with pytest.raises(ValueError, match="channels"):
            call()
    x = torch.randn(2, 1 << 28, device="cuda").to(BF16)[:, :]
    g = torch.full_like(x, -1.0)
    y, _ = gdn.gated_linear_recurrence(x[None], g[None])
    want = x[0, -1000:].double() * torch.exp(torch.tensor(-1.0, dtype=torch.float64)).item() + x[1, -1000:].double()
    assert ((y[0, 1, -1000:].double() - want).norm() / want.norm()).item() <= 2.5e-3
