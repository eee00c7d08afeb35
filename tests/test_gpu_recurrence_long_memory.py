"""Memories of up to a million tokens: constant decays, for which every tile's factor is the same and an error of
it would add up, against the closed sums in 64 bits.

Tolerance, for every value by itself.  With inputs of 1 all terms have one sign.  A window's and a tile's own sums
are off by at most 16 + 16 roundings of 2^-24 and 16 powers of 2^-22, in total 6e-6, whatever the number of tiles;
what a tile adds to the state in front of it keeps its rounding for the next one.  A sum of logarithms is off by as
many roundings, 2e-6, and a state by no more than that of it.  Segments are joined with 10 + 16 roundings more, 1.6e-6.
So 1e-5.  (With a rounded factor for each tile
it would be some 2^-24 for each tile of the memory, 2.4e-4 at 4096.)
"""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from chunked_gated_delta_gdn_gb300 import _lib

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def ones_sum(n, g):
    """1 + a + ... + a^(n - 1) for a = e^g."""
    return torch.expm1(n * g) / torch.expm1(g)


def worst(x, want):
    return ((x.double() - want) / want).abs().max().item()


def test_a_million_tokens_in_segments():
    T, D = 1 << 20, 16
    assert _lib.load().gdn_linear_recurrence_fwd_workspace_size(1, T, D, 1) > 0
    rate = -torch.logspace(-6.5, -3, D, device="cuda")
    g, x = rate.expand(1, T, D).contiguous(), torch.ones(1, T, D, device="cuda")
    rate = rate.double()
    n = torch.arange(1, T + 1, device="cuda", dtype=torch.float64)[:, None]
    y, fin = gdn.gated_linear_recurrence(x, g, output_final_state=True)
    dx, _, dh0 = gdn.gated_linear_recurrence_bwd(x, g, x, initial_state=torch.ones(1, D, device="cuda"))
    errors = dict(y=worst(y[0], ones_sum(n, rate)), state=worst(fin[0], ones_sum(T, rate)),
                  dx=worst(dx[0].flip(0), ones_sum(n, rate)), dh0=worst(dh0[0], torch.exp(rate) * ones_sum(T, rate)))
    print(errors)
    assert max(errors.values()) <= 1e-5


def test_half_a_million_tokens_in_one_chain():
    """Enough channels that nothing is cut: 2048 tiles one after the other forwards, 4096 backwards."""
    T, D = 1 << 19, 8192
    if torch.cuda.mem_get_info()[0] < 8 * 2 * T * D:
        pytest.skip("not enough free memory")
    rate = (-torch.logspace(-6.5, -3, D, device="cuda")).to(BF16)
    g, x = rate.expand(1, T, D).contiguous(), torch.ones(1, T, D, device="cuda", dtype=BF16)
    rate = rate.double()
    fin = gdn.gated_linear_recurrence(x, g, output_final_state=True)[1]
    dh0 = gdn.gated_linear_recurrence_bwd(x, g, x, initial_state=torch.ones(1, D, device="cuda"))[2]
    errors = dict(state=worst(fin[0], ones_sum(T, rate)), dh0=worst(dh0[0], torch.exp(rate) * ones_sum(T, rate)))
    print(errors)
    assert max(errors.values()) <= 1e-5


def test_a_million_tokens_with_fused_gates():
    """c = 1e-5, 1e-6: open gates of a memory as long.  The inputs' factor sqrt(1 - a^2) is common to all of them."""
    T, D = 1 << 20, 8
    lam = torch.linspace(-1.0, 1.0, D, device="cuda")
    x, gate = torch.ones(1, T, D, device="cuda"), torch.full((1, T, D), 30.0, device="cuda")   # (a sigmoid of 1)
    for c in (1e-5, 1e-6):
        y, fin = gdn.gated_linear_recurrence_fused_gates(x, gate, gate, lam, c, output_final_state=True)
        rate = -torch.tensor(c, dtype=F32).double().item() * torch.nn.functional.softplus(lam.double())
        scale = torch.sqrt(-torch.expm1(2 * rate))
        error = worst(fin[0], scale * ones_sum(T, rate))
        print(c, error)
        assert error <= 1e-5
