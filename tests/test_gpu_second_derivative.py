"""The autograd ops of linear attention and group norm have first derivatives only.  With
``create_graph`` the gradients are those without it; a second derivative through them is refused,
also where the rest of the loss has one (a term that went missing would go unnoticed)."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


def attention():
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(1, 70, 2, 32, generator=g, device="cuda", requires_grad=True) for _ in range(3))
    h0 = torch.randn(1, 2, 32, 32, generator=g, device="cuda", requires_grad=True)
    ld = torch.tensor([-0.1, -0.01], device="cuda")

    def call():
        o, fin = gdn.chunk_linear_attn_trainable(q, k, v, ld, initial_state=h0, output_final_state=True)
        return o.sum() + fin.sum()
    return call, (q, k, v, h0)


def norm(gate):
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(9, 64, generator=g, device="cuda", requires_grad=True)
    w, b = (torch.randn(64, generator=g, device="cuda", requires_grad=True) for _ in range(2))
    z = torch.randn(9, 64, generator=g, device="cuda", requires_grad=True) if gate else None
    return (lambda: gdn.group_norm_act_trainable(x, 4, w, b, gate=z).square().sum()), \
        (x, w, b) + ((z,) if gate else ())


CASES = {"attention": attention, "norm": lambda: norm(False), "gated norm": lambda: norm(True)}


@pytest.mark.parametrize("name", sorted(CASES))
def test_second_derivative_is_refused(name):
    call, leaves = CASES[name]()
    want = torch.autograd.grad(call(), leaves)
    got = torch.autograd.grad(call(), leaves, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for leaf, grad in zip(leaves, got):
        penalty = grad.square().sum() + leaf.pow(3).sum()
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(penalty, leaf, retain_graph=True)
    # what does not lead through the op is differentiated as ever
    (twice,) = torch.autograd.grad(leaves[0].pow(3).sum(), leaves[0], create_graph=True)
    (twice,) = torch.autograd.grad(twice.sum(), leaves[0])
    assert torch.allclose(twice, 6 * leaves[0].detach())


def test_only_what_needs_a_gradient():
    g = torch.Generator(device="cuda").manual_seed(3)
    x, z = (torch.randn(9, 64, generator=g, device="cuda") for _ in range(2))
    w = torch.randn(64, generator=g, device="cuda", requires_grad=True)
    y = gdn.group_norm_act_trainable(x, 4, w, None, gate=z)
    (a,) = torch.autograd.grad(y.sum(), w, create_graph=True)
    y = gdn.group_norm_act_trainable(x, 4, w, None, gate=z)
    (b,) = torch.autograd.grad(y.sum(), w)
    assert torch.equal(a, b)
