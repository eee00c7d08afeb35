"""A workspace that the kernels cannot use is refused by the binding: one that is not in this device's
memory, not contiguous (its bytes are counted from its elements), or not a tensor."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


def calls():
    q = torch.randn(1, 1100, 1, 64, device="cuda")
    ld = torch.full((1,), -0.01, device="cuda")
    x = torch.randn(2, 3000, 64, device="cuda")
    _, mean, rstd = gdn.group_norm_act(x, 4, return_stats=True)
    return {"attention": lambda ws: gdn.chunk_linear_attn(q, q, q, ld, workspace=ws)[0],
            "attention, gradients": lambda ws: gdn.chunk_linear_attn_bwd(q, q, q, ld, q, workspace=ws)[0],
            "norm": lambda ws: gdn.group_norm_act(x, 4, workspace=ws),
            "norm, gradients": lambda ws: gdn.group_norm_act_bwd(x, x, mean, rstd, 4, workspace=ws)[0]}


def test_workspaces():
    big = 1 << 24
    for name, call in calls().items():
        want = call(None)
        with pytest.raises(ValueError, match="CUDA"):
            call(torch.empty(big, dtype=torch.uint8))
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.empty(2 * big, dtype=torch.uint8, device="cuda")[::2])
        with pytest.raises(TypeError):
            call(big)
        assert torch.equal(call(torch.empty(big, dtype=torch.uint8, device="cuda")), want), name
        assert torch.equal(call(torch.empty(16, dtype=torch.uint8, device="cuda")), want), name   # (replaced)
