"""Calls of several launches, of which the later ones start before the earlier ones have ended: one
after the other on the same scratch and outputs, and replayed from a CUDA graph, they give what a
call by itself gives, bit for bit."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


def linear_attn(dtype, B=1, T=1500, H=4):
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k, v, do = (r(B, T, H, 64).to(dtype) for _ in range(4))
    ld, h0 = torch.log1p(-torch.rand(H, generator=g, device="cuda") / 8), r(B, H, 64, 64)

    def call(ws=None):
        o, fin = gdn.chunk_linear_attn(q, k, v, ld, initial_state=h0, output_final_state=True, workspace=ws)
        return (o, fin) + gdn.chunk_linear_attn_bwd(q, k, v, ld, do, fin, initial_state=h0, workspace=ws)
    return call


def group_norm(dtype, shape=(3, 999, 96), G=8, gate=True):
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, z, dy = (r(*shape).to(dtype) for _ in range(3))
    w, b = r(shape[-1]), r(shape[-1])
    z = z if gate else None

    def call(ws=None):
        y, m, s = gdn.group_norm_act(x, G, w, b, gate=z, return_stats=True, workspace=ws)
        return (y, m, s) + gdn.group_norm_act_bwd(dy, x, m, s, G, w, b, gate=z, workspace=ws)
    return call


CASES = {
    "attention": lambda dt: linear_attn(dt),
    "attention, a rest": lambda dt: linear_attn(dt, B=2, T=1100, H=80),
    "norm, slabs": lambda dt: group_norm(dt),
    "norm, rows": lambda dt: group_norm(dt, shape=(3000, 512)),
    "norm, wide": lambda dt: group_norm(dt, shape=(2, 65, 4100), G=1, gate=False),
}


def same(a, b):
    for x, y in zip(a, b):
        assert (x is None) == (y is None) and (x is None or torch.equal(x, y))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("name", sorted(CASES))
def test_calls_in_a_row_and_from_a_graph(name, dtype):
    call = CASES[name](dtype)
    want = call()
    torch.cuda.synchronize()
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    runs = [call(ws) for _ in range(6)]     # every call on the scratch of the one before it
    for got in runs:
        same(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        same(call(ws), want)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(ws)
    for _ in range(3):
        for t in got:
            if t is not None:
                t.zero_()
        ws.zero_()
        graph.replay()
        same(got, want)
