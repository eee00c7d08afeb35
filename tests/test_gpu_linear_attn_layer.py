"""The example layer: its three ways of running agree with one another and with a plain 64-bit form
that takes the layer's own bf16 projections.  (Where q . k is small next to |q| |k|, the projections'
rounding is a large share of it, and the norm brings such a token's o back to size: that error is
the layer's choice of bf16 there, the same for any way of computing what follows.)

Tolerances (relative 2-norm), in bf16: each rounding of a tensor costs 1.7e-3 (2^-9 uniform), and
what follows a projection is a sum of independent ones: projections' outputs, P or the state's bf16
operand, o, the norm's output, the last projection's: five of them, 4e-3; 1e-2 allowed for the
normalisation's and the gate's slopes.  The gradient passes twice as many: 2e-2.
"""
import pytest
import torch

from chunked_gated_delta_gdn_gb300.examples.linear_attn_layer import LinearAttnLayer, main

pytestmark = pytest.mark.gpu


def plain(layer, x, weights):
    """[T, dim] in 64 bits, token by token, for one sequence."""
    wi, wo, w, b = weights
    full = x @ wi.T
    rounded = layer.inp(x.detach().to(torch.bfloat16)).double()   # (its gradient is full's)
    q, k, v, z = (full + (rounded - full).detach()).split(layer.splits, -1)
    T, G = x.shape[0], layer.Hv // layer.Hqk
    q, k = (t.view(T, layer.Hqk, layer.K).repeat_interleave(G, 1) for t in (q, k))
    v = v.view(T, layer.Hv, layer.V)
    S = x.new_zeros(layer.Hv, layer.K, layer.V)
    decay = layer.log_decay.double().exp()[:, None, None]
    o = []
    for t in range(T):
        S = decay * S + k[t][:, :, None] * v[t][:, None, :]
        o.append((S * q[t][:, :, None]).sum(1) / layer.K ** 0.5)
    o = torch.stack(o)
    o = (o - o.mean(-1, keepdim=True)) / torch.sqrt(o.var(-1, unbiased=False, keepdim=True) + 1e-5)
    y = (o.flatten(1) * w + b) * torch.nn.functional.silu(z)
    return y @ wo.T


def rel(a, b):
    a, b = a.double(), b.double()
    assert torch.isfinite(a).all()
    return ((a - b).norm() / b.norm()).item()


def weights_of(layer):
    return [p.detach().double().requires_grad_() for p in
            (layer.inp.weight, layer.out.weight, layer.weight, layer.bias)]


@pytest.mark.parametrize("heads", [(2, 4, 64, 64), (3, 3, 128, 32)])
def test_training_step_against_plain(heads):
    torch.manual_seed(1)
    layer = LinearAttnLayer(96, *heads)
    x = torch.randn(2, 77, 96, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    dy = torch.randn_like(x)
    y = layer(x)
    mine = torch.autograd.grad(y, [x, layer.inp.weight, layer.out.weight, layer.weight, layer.bias], dy)
    ws, xd = weights_of(layer), x.detach().double().requires_grad_()
    want = torch.stack([plain(layer, xd[i], ws) for i in range(2)])
    grads = torch.autograd.grad(want, [xd] + ws, dy.double())
    assert rel(y, want) < 1e-2
    for a, b in zip(mine, grads):
        assert rel(a, b) < 2e-2


def test_prefill_then_decode_continues_the_sequence():
    torch.manual_seed(2)
    layer = LinearAttnLayer(128)
    lens, more = [70, 1, 0, 130], 3
    x = [torch.randn(n + more, 128, device="cuda", dtype=torch.bfloat16) for n in lens]
    cu = torch.tensor([0, 70, 71, 71, 201], dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 0, 6, 2], dtype=torch.int32, device="cuda")
    cache = torch.zeros(8, layer.Hv, layer.K, layer.V, device="cuda")
    y = layer.prefill(torch.cat([t[:n] for t, n in zip(x, lens)])[None], cu, cache, slots)[0]
    outs = [[y[int(cu[i]):int(cu[i + 1])]] for i in range(4)]
    padded = torch.cat([slots, slots.new_tensor([-1])])
    for s in range(more):
        tok = torch.stack([t[n + s] for t, n in zip(x, lens)] + [x[0][0]])
        o = layer.decode(tok, cache, padded)
        for i in range(4):
            outs[i].append(o[i:i + 1])
    ws = [w.detach() for w in weights_of(layer)]
    for t, o in zip(x, outs):
        assert rel(torch.cat(o), plain(layer, t.double(), ws)) < 1e-2
    assert (cache[[1, 3, 4, 7]] == 0).all()


def test_packed_training_equals_rows_apart():
    torch.manual_seed(3)
    layer = LinearAttnLayer(64)
    x = torch.randn(1, 150, 64, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0, 64, 65, 150], dtype=torch.int32, device="cuda")
    y = layer(x, cu)
    ws = [w.detach() for w in weights_of(layer)]
    for a, b in ((0, 64), (64, 65), (65, 150)):
        assert rel(y[0, a:b], plain(layer, x[0, a:b].double(), ws)) < 1e-2


def test_decode_replays_from_a_graph():
    torch.manual_seed(4)
    layer = LinearAttnLayer(64)
    x = torch.randn(3, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    cache = torch.randn(4, layer.Hv, layer.K, layer.V, device="cuda")
    twin = cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(x, cache.clone(), slots)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.decode(x, cache, slots)
    for _ in range(2):
        graph.replay()
        want = layer.decode(x, twin, slots)
        assert torch.equal(y, want)
    assert torch.equal(cache, twin)


def test_example_runs(capsys):
    main()
    out = capsys.readouterr().out.splitlines()
    assert len(out) == 5 and all("nan" not in line for line in out)
    losses = [float(line.split()[-1]) for line in out[:3]]
    assert losses[2] < losses[0]
