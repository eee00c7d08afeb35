"""The example block, the operators one behind the other as a stack runs them: its training step against a
plain 64-bit form that takes the layers' own bf16 projections, its prefill and decode against its training
forward, decode replayed from a graph.

Tolerances (relative 2-norm) in bf16: a rounding of a tensor costs 1.7e-3, what follows a projection is a sum
of independent ones.  A layer has six (projection, rotated q and k, the mixer's operands, its output, the
norm's output, the last projection), two layers twelve with the sums: 6e-3 added as squares; 1.5e-2
allowed for the slopes of norms and gates, 3e-2 for gradients, which pass twice as many.
"""
import pytest
import torch

from chunked_gated_delta_gdn_gb300.examples.hybrid_block import HybridBlock, RecurrentLayer, main, packed
from tests.recurrence_ref import recurrence

pytestmark = pytest.mark.gpu


def rel(a, b):
    a, b = a.double(), b.double()
    assert torch.isfinite(a).all()
    return ((a - b).norm() / b.norm()).item()


def projected(layer, x, w):
    """The projection's parts with the layer's bf16 values and the 64-bit gradient."""
    full = x @ w.T
    rounded = layer.inp(x.detach().to(torch.bfloat16)).double()
    return (full + (rounded - full).detach()).split(layer.parts, -1)


def finish(layer, o, z, weight, out):
    o = o.unflatten(-1, (layer.groups, -1))
    o = (o - o.mean(-1, keepdim=True)) / torch.sqrt(o.var(-1, unbiased=False, keepdim=True) + 1e-5)
    return (o.flatten(-2) * weight * torch.nn.functional.silu(z)) @ out.T


def attention(layer, x, w):
    q, k, v, z = projected(layer, x, w["inp.weight"])
    T = x.shape[0]
    phi = torch.arange(T, device="cuda")[:, None, None] * layer.inv_freq.double()

    def turned(t, weight):
        t = t.view(T, layer.Hqk, -1)
        t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * weight
        u, s = t.chunk(2, -1)
        t = torch.cat([u * phi.cos() - s * phi.sin(), s * phi.cos() + u * phi.sin()], -1)
        return t.repeat_interleave(layer.Hv // layer.Hqk, 1)
    q, k, v = turned(q, w["q_weight"]), turned(k, w["k_weight"]), v.view(T, layer.Hv, -1)
    dist = (torch.arange(T, device="cuda")[:, None] - torch.arange(T, device="cuda")).double()
    decay = torch.exp(layer.log_decay.double()[:, None, None] * dist.clamp(min=0)) * (dist >= 0)
    o = torch.einsum("thk,shk,hts,shv->thv", q, k, decay, v) / q.shape[-1] ** 0.5
    return finish(layer, o.flatten(1), z, w["weight"], w["out.weight"])


def plain(block, x, weights):
    """One sequence [T, dim] in 64 bits."""
    for layer, w in zip(block.layers, weights):
        if isinstance(layer, RecurrentLayer):
            u, r, i, z = projected(layer, x, w["inp.weight"])
            h, _ = recurrence(u[None], r[None], i[None], w["lam"], 8.0)
            x = x + finish(layer, h[0], z, w["weight"], w["out.weight"])
        else:
            x = x + attention(layer, x, w)
    return x


def weights_of(block):
    return [{n: p.detach().double().requires_grad_() for n, p in layer.named_parameters()} for layer in block.layers]


def test_training_step_against_plain():
    torch.manual_seed(1)
    block = HybridBlock(96)
    x = torch.randn(2, 77, 96, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    dy = torch.randn_like(x)
    y = block(x)
    names = [(n, name) for n, layer in enumerate(block.layers) for name, _ in layer.named_parameters()]
    mine = torch.autograd.grad(y, [x] + [dict(block.layers[n].named_parameters())[m] for n, m in names], dy)
    ws, xd = weights_of(block), x.detach().double().requires_grad_()
    want = torch.stack([plain(block, xd[b], ws) for b in range(2)])
    assert rel(y, want) <= 1.5e-2
    grads = torch.autograd.grad(want, [xd] + [ws[n][m] for n, m in names], dy.double())
    for (n, m), a, b in zip([(-1, "x")] + names, mine, grads):
        assert rel(a, b) <= 3e-2, (n, m)


def test_prefill_and_decode_follow_the_training_forward():
    torch.manual_seed(2)
    block = HybridBlock(64, Hqk=2, Hv=2, K=32, V=64)
    lens, more = [33, 1, 0, 150], 3
    x = [torch.randn(n + more, 64, device="cuda", dtype=torch.bfloat16) for n in lens]
    want = [block(t[None]).detach()[0] for t in x]
    cu, pos = packed(lens)
    slots = torch.tensor([4, 1, 0, 6], dtype=torch.int32, device="cuda")
    caches = block.caches(7)
    y = block.prefill(torch.cat([t[:n] for t, n in zip(x, lens)])[None], cu, pos, caches, slots)
    assert rel(y[0], torch.cat([t[:n] for t, n in zip(want, lens)])) <= 1.5e-2
    before = [c.clone() for c in caches]
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    token = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    graph, out = torch.cuda.CUDAGraph(), None
    for step in range(more):
        tokens = torch.stack([t[n + step] for t, n in zip(x, lens)])
        got = block.decode(tokens, at + step, caches, slots)
        assert rel(got, torch.stack([t[n + step] for t, n in zip(want, lens)])) <= 1.5e-2
    # the same steps replayed from a graph on the caches as the prefill left them: bit for bit
    after = [c.clone() for c in caches]
    for c, b in zip(caches, before):
        c.copy_(b)
    where = at.clone()
    with torch.cuda.graph(graph):
        out = block.decode(token, where, caches, slots)
    for c, b in zip(caches, before):
        c.copy_(b)
    for step in range(more):
        token.copy_(torch.stack([t[n + step] for t, n in zip(x, lens)]))
        where.copy_(at + step)
        graph.replay()
    assert torch.equal(out, got) and all(torch.equal(a, b) for a, b in zip(caches, after))


def test_packed_training_is_the_sequences_one_by_one():
    torch.manual_seed(3)
    block = HybridBlock(64, Hqk=1, Hv=2, K=64, V=32)
    lens = [40, 130, 1]
    x = torch.randn(1, sum(lens), 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    cu, pos = packed(lens)
    y = block(x, cu, pos)
    parts = [block(t) for t in x.split(lens, 1)]
    assert rel(y, torch.cat(parts, 1)) <= 1.5e-2
    dy = torch.randn_like(y)
    a, = torch.autograd.grad(y, x, dy)
    b, = torch.autograd.grad(torch.cat(parts, 1), x, dy)
    assert rel(a, b) <= 3e-2


def test_main_runs(capsys):
    main()
    assert capsys.readouterr().out.count("norms") == 2
