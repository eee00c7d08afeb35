"""Packed sequences of one to three chunks, whose CTAs look their place up by length and load their
first chunk right after: run after run the same bits, and the 64-bit recurrence's values (tolerances as
in test_gpu_linear_attn.py; no sequence is longer than there)."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from tests import linear_attn_ref as ref
from tests.test_gpu_linear_attn import BF16, F32, TOL, make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2, 40, 128])
def test_packed_runs_repeat(n):
    lens = torch.randint(1, 193, (n,), generator=torch.Generator().manual_seed(n)).tolist()
    x = on_gpu(make(lens=lens, Hqk=1, Hv=2, K=128, V=128, dtype=BF16, seed=n))

    def call():
        return gdn.chunk_linear_attn(x["q"], x["k"], x["v"], x["log_decay"], initial_state=x["h0"],
                                     output_final_state=True, cu_seqlens=x["cu"])

    o, fin = call()
    runs = [call() for _ in range(30)]
    assert all(torch.equal(o, a) and torch.equal(fin, b) for a, b in runs)
    o_ref, fin_ref = ref.forward(x["q"], x["k"], x["v"], x["log_decay"], h0=x["h0"], cu=x["cu"].cpu())
    assert ref.rel(o, o_ref) <= TOL[BF16] and ref.rel(fin, fin_ref) <= TOL[F32]
