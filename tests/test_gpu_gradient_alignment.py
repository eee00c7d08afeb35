"""Incoming gradients start where the graph behind the op left them: a part of a larger tensor (the
gradient of a concatenation, say) starts at any element.  The autograd ops take them as they come and
give the gradients of the same values elsewhere, bit for bit."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


def behind_a_concatenation(outs, leaves, seed):
    """Gradients of the leaves through outs, each flattened behind one more element, and without it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ds = [torch.randn(o.numel() + 1, generator=g, device="cuda").to(o.dtype) for o in outs]
    head = [torch.zeros(1, dtype=o.dtype, device="cuda", requires_grad=True) for o in outs]
    joined = [torch.cat([h, o.flatten()]) for h, o in zip(head, outs)]
    got = torch.autograd.grad(joined, leaves, ds, retain_graph=True)
    want = torch.autograd.grad(outs, leaves, [d[1:].clone().view(o.shape) for d, o in zip(ds, outs)])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_attention(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    leaves = [torch.randn(2, 70, 2, 32, generator=g, device="cuda").to(dtype).requires_grad_() for _ in range(3)]
    h0 = torch.randn(2, 2, 32, 32, generator=g, device="cuda", requires_grad=True)
    ld = torch.tensor([-0.1, -0.01], device="cuda")
    outs = gdn.chunk_linear_attn_trainable(*leaves, ld, initial_state=h0, output_final_state=True)
    behind_a_concatenation(outs, leaves + [h0], 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape,G", [((3, 5), 1), ((4, 64), 4), ((2, 500, 24), 3)])
def test_group_norm(shape, G, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    x, z = (torch.randn(*shape, generator=g, device="cuda").to(dtype).requires_grad_() for _ in range(2))
    w = torch.randn(shape[-1], generator=g, device="cuda", requires_grad=True)
    for gate in (None, z):
        y = gdn.group_norm_act_trainable(x, G, w, None, gate=gate)
        behind_a_concatenation([y], [x, w] + ([] if gate is None else [z]), 4)
