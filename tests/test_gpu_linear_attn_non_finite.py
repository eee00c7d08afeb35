"""How far a NaN or an infinity in one token reaches: its 64-token chunk and what follows it in its
sequence and head (backwards, what comes before it).  The chunks before it, other heads and the other
sequences keep their bits."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from tests.test_gpu_linear_attn import BF16, F32, make, on_gpu

pytestmark = pytest.mark.gpu


def run(x, do):
    o, fin = gdn.chunk_linear_attn(x["q"], x["k"], x["v"], x["log_decay"], initial_state=x["h0"],
                                   output_final_state=True)
    return (o, fin) + gdn.chunk_linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], do,
                                                initial_state=x["h0"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,at", [(200, 100), (200, 64), (2000, 1300)])     # (2000: cut into segments)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_reach(T, at, bad, dtype):
    x = on_gpu(make(B=2, T=T, Hqk=2, Hv=2, K=64, V=64, dtype=dtype, seed=T))
    do = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    want = run(x, do)
    start = at // 64 * 64
    for name in ("k", "v"):
        y = {**x, name: x[name].clone()}
        y[name][0, at, 0, 3] = bad
        o, fin, dq, dk, dv, dh0 = run(y, do)
        assert torch.equal(o[1], want[0][1]) and torch.equal(o[0, :, 1], want[0][0, :, 1])
        assert torch.equal(fin[1], want[1][1]) and torch.equal(fin[0, 1], want[1][0, 1])
        assert torch.equal(o[0, :start], want[0][0, :start])
        assert not torch.isfinite(o[0, at:, 0].float()).all()
        assert torch.equal(dq[0, :start], want[2][0, :start])
        for got, ref in zip((dq, dk, dv), want[2:5]):
            assert torch.equal(got[1], ref[1]) and torch.equal(got[0, :, 1], ref[0, :, 1])
    y = do.clone()
    y[0, at, 0, 3] = bad
    _, _, dq, dk, dv, dh0 = run(x, y)
    for got, ref in zip((dk, dv), want[3:5]):
        assert torch.equal(got[0, start + 64:], ref[0, start + 64:])
        assert torch.equal(got[1], ref[1]) and torch.equal(got[0, :, 1], ref[0, :, 1])
    assert torch.equal(dh0[1], want[5][1]) and torch.equal(dh0[0, 1], want[5][0, 1])
