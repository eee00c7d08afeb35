"""Linear attention where its chains are many: uniform batches of which a part is cut into segments,
packed ones whose sequences start longest first.  Against the 64-bit recurrence; tolerances as in
test_gpu_linear_attn.py (fp32 5e-6; bf16 4e-3), whose reasons hold here: no chain is longer than
there, and a cut adds one rounding of the state to 24 bits.
"""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from tests import linear_attn_ref as ref
from tests.test_gpu_linear_attn import BF16, F32, TOL, check_forward, grads_ref, make, on_gpu

pytestmark = pytest.mark.gpu


# (chains of a launch: 154, 160, 192 on 152 SMs; the last length leaves a partial chunk)
@pytest.mark.parametrize("B,Hv,T", [(2, 77, 1500), (4, 40, 2048), (3, 64, 1537)])
def test_uniform_batch_with_a_rest(B, Hv, T):
    x = make(B=B, T=T, Hqk=Hv, Hv=Hv, K=32, V=64, seed=B)
    o, fin = check_forward(x)
    c = on_gpu(x)
    # in place: the entry states are read before anything is written over them
    cache = c["h0"].clone()
    o2, fin2 = gdn.chunk_linear_attn(c["q"], c["k"], c["v"], c["log_decay"], initial_state=cache,
                                     output_final_state=True, final_state=cache, check=True)
    assert torch.equal(o, o2) and torch.equal(fin, fin2) and fin2 is cache


@pytest.mark.parametrize("state", [True, False])
def test_uniform_backward_with_a_rest(state):
    x = on_gpu(make(B=2, T=1090, Hqk=13, Hv=26, K=64, V=32, h0=state, seed=7))   # 156 chains
    g = torch.Generator().manual_seed(8)
    do = torch.randn(x["v"].shape, generator=g).to(BF16).cuda()
    dh = torch.randn(x["h0"].shape, generator=g).cuda() if state else None
    got = gdn.chunk_linear_attn_bwd(x["q"], x["k"], x["v"], x["log_decay"], do, dh,
                                    initial_state=x["h0"], check=True)
    errs = [ref.rel(a, b) for a, b in zip(got, grads_ref(x, do, dh))]
    assert all(e <= TOL[BF16] for e in errs[:3])
    if state:
        assert errs[3] <= TOL[F32]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [128, 129, 300])
def test_many_packed_sequences(n, dtype):
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 150, (n,), generator=g).tolist()
    lens[3] = lens[17] = 700     # equal, and the longest
    check_forward(make(lens=lens, Hqk=1, Hv=2, K=64, V=32, dtype=dtype, tail=5, seed=n))
