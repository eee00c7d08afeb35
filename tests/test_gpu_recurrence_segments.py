"""The gated linear recurrence where a few chains are cut into segments, over several launches: against the
64-bit recurrence (tolerances as in test_gpu_recurrence), with states that are read in one segment and
written in another's place, in a row on one scratch, from graphs, and on bad packed lengths."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from chunked_gated_delta_gdn_gb300 import _lib
from tests.test_gpu_recurrence import BF16, F32, NAN, backward, check, forward, make, reference, rel, seeded, tol  # noqa: F401

pytestmark = pytest.mark.gpu
LENS = [700, 1, 0, 2500, 300, 0, 5, 2400, 40]       # whole forwards, cut backwards
LONG = [3000, 1, 0, 9000, 1300, 0, 5, 9600, 40]     # both cut


def cut(T, D, N):
    """Whether such a batch is cut at all on this device."""
    return _lib.load().gdn_linear_recurrence_fwd_workspace_size(1, T, D, N) > 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("lens,tail,D", [(LENS, 77, 24), (LONG, 77, 24), ([5000], 0, 70), ([1, 4097, 0], 3, 8), ([256] * 16, 0, 40),
                                         ([2100, 2100], 0, 40), ([40] * 90, 500, 33), ([0, 3000], 3000, 16)])
def test_packed(lens, tail, D, fused, dtype):
    if len(lens) < 4 or lens is LONG:   # (many sequences are parts enough, and stay whole)
        assert cut(sum(lens) + tail, D, len(lens))
    check((1, sum(lens) + tail, D), dtype, None, fused, lens=lens)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("shape", [(1, 4500, 72), (2, 2049, 20), (3, 2048, 130)])
def test_dense(shape, fused):
    check(shape, BF16, F32, fused)
    check(shape, F32, F32, fused, state=False)


@pytest.mark.parametrize("lens", [LENS, LONG])
@pytest.mark.parametrize("fused", [False, True])
def test_slots_in_place(fused, lens):
    """States come from and go to the same slots, which sequences of several segments share in time."""
    T, D = sum(lens) + 50, 40
    ins = make((1, T, D), F32, fused=fused)
    cu = torch.tensor([sum(lens[:n]) for n in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 9, 1, 0, 7, -1, 5, 2, -1], dtype=torch.int32, device="cuda")
    start = torch.randn(11, D, device="cuda")
    assert cut(T, D, len(lens)) == (lens is LONG)
    live = [n for n in range(len(lens)) if slots[n] >= 0]
    rows = torch.cat([torch.arange(int(cu[n]), int(cu[n + 1]), device="cuda") for n in live])
    want, fin, _ = reference([t[:, rows] if t.dim() == 3 else t for t in ins], start[slots[live].long()],
                             [lens[n] for n in live])
    for t in ins[:3]:
        if t.dim() == 3:
            t[:, int(cu[8]):] = NAN      # padding's and no sequence's
    runs = []
    for _ in range(3):
        cache = start.clone()
        y, got = forward(ins, initial_state=cache, output_final_state=True, cu_seqlens=cu, state_indices=slots,
                         out=torch.full_like(ins[0], NAN), check=True)
        assert got is cache
        runs.append((y, cache))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))
    y, cache = runs[0]
    assert rel(y[:, rows], want) <= tol(y) and rel(cache[slots[live].long()], fin) <= 1e-5
    assert not y[:, int(cu[8]):].any()
    rest = torch.ones(11, dtype=torch.bool)
    rest[slots[live].long().cpu()] = False
    assert torch.equal(cache[rest.cuda()], start[rest.cuda()])
    # the same into another cache
    other = torch.full_like(start, NAN)
    y2, _ = forward(ins, initial_state=start, output_final_state=True, cu_seqlens=cu, state_indices=slots,
                    final_state=other)
    assert torch.equal(y2, y) and torch.equal(other[slots[live].long()], cache[slots[live].long()])


@pytest.mark.parametrize("fused", [False, True])
def test_in_a_row_and_from_graphs(fused):
    ins, other = make((1, 5000, 48), BF16, fused=fused), make((1, 5000, 48), BF16, fused=fused, seed=8)
    dy = torch.randn_like(ins[0])
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    run = lambda ins: forward(ins, output_final_state=True, workspace=ws) + tuple(backward(ins, dy, workspace=ws))
    same = lambda a, b: all((s is None and t is None) or torch.equal(s, t) for s, t in zip(a, b))
    torch.cuda.synchronize()
    want, want2 = run(ins), None
    torch.cuda.synchronize()
    want2 = run(other)
    torch.cuda.synchronize()
    got = [run(t) for t in (ins, other, ins, other)]
    assert same(got[0], want) and same(got[1], want2) and same(got[2], want) and same(got[3], want2)
    graphs, outs = [], []
    for t in (ins, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(t))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert same(outs[0], want) and same(outs[1], want2)


def test_bad_packed_lengths():
    x, g = make((1, 6000, 24), F32)
    h0 = torch.randn(2, 24, device="cuda")
    for cu in ([0, 4000, 3999], [1, 5, 9], [0, 5, 6001]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        fin, status = torch.full_like(h0, 3.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        y, _ = gdn.gated_linear_recurrence(x, g, h0, True, cu, final_state=fin, dev_status=status,
                                           out=torch.full_like(x, NAN))
        assert status.item() == 2 and not y.any() and (fin == 3.0).all()
        grads = gdn.gated_linear_recurrence_bwd(x, g, x, h0, h0, cu)
        assert not any(t.any() for t in grads)


@pytest.mark.parametrize("tail", [0, 9000])     # (the longer one is cut in the forward, too)
def test_non_finite_values_stay_in_their_sequence(tail):
    cu = torch.tensor([0, 900, 2200, 2900, 4700 + tail], dtype=torch.int32, device="cuda")
    x, g = make((1, 4700 + tail, 16), F32)
    dy = torch.randn_like(x)
    y, fin = gdn.gated_linear_recurrence(x, g, None, True, cu)
    dx, dg, _ = gdn.gated_linear_recurrence_bwd(x, g, dy, cu_seqlens=cu)
    x2, d2 = x.clone(), dy.clone()
    x2[0, 1000, 3] = NAN
    d2[0, 2800, 5] = NAN
    y2, fin2 = gdn.gated_linear_recurrence(x2, g, None, True, cu)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 1000:2200, 3] = True
    assert torch.equal(y2[~hit], y[~hit]) and y2[hit].isnan().all() and torch.equal(fin2[[0, 2, 3]], fin[[0, 2, 3]])
    got = gdn.gated_linear_recurrence_bwd(x, g, d2, cu_seqlens=cu)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 2200:2801, 5] = True
    assert torch.equal(got[0][~hit], dx[~hit]) and torch.equal(got[1][~hit], dg[~hit])


def test_workspaces():
    """One that the kernels cannot use is refused, one that is too small replaced."""
    x, g = make((1, 5000, 48), F32)
    for call in (lambda ws: gdn.gated_linear_recurrence(x, g, workspace=ws)[0],
                 lambda ws: gdn.gated_linear_recurrence_bwd(x, g, x, workspace=ws)[0]):
        want = call(None)
        with pytest.raises(ValueError, match="CUDA"):
            call(torch.empty(1 << 24, dtype=torch.uint8))
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.empty(1 << 25, dtype=torch.uint8, device="cuda")[::2])
        with pytest.raises(TypeError):
            call(1 << 24)
        assert torch.equal(call(torch.empty(16, dtype=torch.uint8, device="cuda")), want)
        assert torch.equal(call(torch.empty(1 << 24, dtype=torch.uint8, device="cuda")), want)


def test_captured_training_step():
    """A step captured by hand, backward and all; eager graphs of the same leaves are gone by then (while one
    lives, the engine itself ends such a capture with an error) and are made again behind it."""
    x, r, i, lam = make((1, 3000, 32), BF16, fused=True)
    leaves = [t.requires_grad_() for t in (x, r, i, lam)]
    dy = torch.randn(1, 3000, 32, device="cuda").to(BF16)
    step = lambda: torch.autograd.grad(gdn.gated_linear_recurrence_fused_gates_trainable(*leaves)[0], leaves, dy)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    alive, _ = gdn.gated_linear_recurrence_fused_gates_trainable(*leaves)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(alive, leaves, dy), want))
