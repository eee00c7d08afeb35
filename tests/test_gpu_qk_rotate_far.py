"""Angles of every int32 position and every finite frequency, against integers of 500 bits.

Tolerance (relative 2-norm of a head): an angle of less than half a turn is rounded to fp32, 2^-24 of pi,
1.9e-7; sine and cosine by some 2^-23, products and sums by 2^-24 each: 1e-6.  bf16 outputs are rounded
once, 2^-8 of the value, and their sines and cosines are off by 2^-20.
"""
import math
import struct

import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn

BITS = 500
POSITIONS = [0, 1, -1, 2, 1000, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321, 2000000011]
FREQS = [1.0, 5.9, -5.9, 100.0, 1000.7, 0.15915494, 6.2831855, 3.1415927, 65536.0, 1e6, 1.6777215e7, 1.6777216e7,
         12345678848.0, 1e18, -1e18, 1e30, 3.4028235e38, -3.4028235e38, 1.7014118e38, 0.1, 1e-3, 1e-6, 1e-9, -1e-9, 1e-12,
         1e-20, 1e-30, 1.17549435e-38, 1e-40, 1e-45, 0.0, -0.0]


def two_pi(bits):
    """2 pi in units of 2^-bits, by Machin's formula."""
    one = 1 << (bits + 32)

    def arctan_inverse(n):
        total = term = one // n
        k = 1
        while term:
            term //= n * n
            total += (-1 if k & 1 else 1) * (term // (2 * k + 1))
            k += 1
        return total
    return 2 * (4 * (4 * arctan_inverse(5) - arctan_inverse(239))) >> 32


TWO_PI = two_pi(BITS)


def angle(position, freq):
    """position * freq in [0, 2 pi), of integers."""
    freq = struct.unpack("f", struct.pack("f", freq))[0]
    num, den = float(freq).as_integer_ratio()
    phase = position * num * (1 << BITS) // den   # units of 2^-BITS
    return (phase % TWO_PI) / (1 << BITS)


def test_the_oracle():
    assert abs(TWO_PI / (1 << BITS) - 2 * math.pi) < 1e-15
    for position, freq in ((3, 1.0), (1000, 0.5), (-7, 0.25), (123456, 1.0)):
        assert abs(math.sin(angle(position, freq)) - math.sin(position * freq)) < 1e-10


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_position_and_frequency(dtype):
    P, F = len(POSITIONS), len(FREQS)
    freq = torch.tensor(FREQS, dtype=torch.float32, device="cuda")
    pos = torch.tensor(POSITIONS, dtype=torch.int32, device="cuda")
    phi = torch.tensor([[angle(p, f) for f in FREQS] for p in POSITIONS], dtype=torch.float64, device="cuda")[:, None]
    gen = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randn(P, 2, 2 * F, generator=gen, device="cuda").to(dtype)
    got, _ = gdn.qk_norm_rotate(q, q, freq, pos, norm=None)
    u, v = q[..., :F].double(), q[..., F:].double()
    want = torch.stack([u * phi.cos() - v * phi.sin(), v * phi.cos() + u * phi.sin()], -1)
    have = torch.stack([got[..., :F], got[..., F:]], -1).double()
    error = (have - want).norm(dim=-1) / want.norm(dim=-1)   # of each pair
    print(dtype, error.max().item(), FREQS[error.amax((0, 1)).argmax().item()])
    assert error.max().item() <= (1e-6 if dtype is torch.float32 else 2.0 ** -8 + 2e-6)
    dq = gdn.qk_norm_rotate_bwd(got, got, q, q, freq, pos, norm=None, need_weights=False)[0]
    du, dv = got[..., :F].double(), got[..., F:].double()
    want = torch.stack([du * phi.cos() + dv * phi.sin(), dv * phi.cos() - du * phi.sin()], -1)
    have = torch.stack([dq[..., :F], dq[..., F:]], -1).double()
    assert ((have - want).norm(dim=-1) / want.norm(dim=-1)).max().item() <= (
        1e-6 if dtype is torch.float32 else 2.0 ** -8 + 2e-6)
