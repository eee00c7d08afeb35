"""The gated linear recurrence with final_state the initial states' own tensor, without a slot cache: whole chains
and chains that are cut, where one launch writes what another one reads.  Bit for bit what separate tensors get."""
import pytest
import torch

from tests.test_gpu_recurrence import BF16, F32, forward, make, seeded  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("shape,lens", [((3, 150, 40), None), ((1, 9000, 24), None), ((3, 5000, 16), None),
                                        ((1, 14000, 40), [3000, 1, 0, 9000, 1300, 0, 5, 90]), ((1, 9000, 8), [0, 1, 8990, 0])])
def test_final_states_in_the_initial_ones_place(shape, lens, fused, dtype):
    ins = make(shape, dtype, fused=fused)
    N = shape[0] if lens is None else len(lens)
    h0 = torch.randn(N, shape[-1], device="cuda")
    kw = {}
    if lens is not None:
        kw["cu_seqlens"] = torch.tensor([sum(lens[:n]) for n in range(N + 1)], dtype=torch.int32, device="cuda")
    y, fin = forward(ins, initial_state=h0, output_final_state=True, **kw)
    for _ in range(3):
        place = h0.clone()
        y2, got = forward(ins, initial_state=place, final_state=place, output_final_state=True, **kw)
        assert got is place and torch.equal(y2, y) and torch.equal(place, fin)
