"""Linear attention over thousands of tokens with a long memory: what is multiplied or added once a
token or chunk must not err in the same direction each time, and not more often than it has to.

u = 2^-24; a value rounded to 24 bits errs by 0.42 u of itself in the mean square.
"""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from tests import linear_attn_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_for_thousands_of_tokens(dtype):
    """One rounding a token or two (the decayed state, the sum): 0.6 u of the state then, over n = 4096
    tokens 0.6 u sqrt(n) = 38 u = 2.3e-6 at most; 5e-6 leaves a factor of two.  A decay rounded to
    24 bits is off by up to u / 2 each time: n u / 2 = 1.2e-4; a decayed state that is rounded by itself
    errs in the same direction each time where the decay is not much more than u.

    The state between two tokens is fp32 and so is the reference's, rounded once a token from 64 bits:
    where a token takes less than half a unit in the last place off (-3e-8 here) and k v^T of bf16 values
    leaves the state on its grid, no fp32 state decays.  Where the decay is 16 u and more the state
    is held to the recurrence in 64 bits as well."""
    n, K, V = 4096, 16, 32
    ld = torch.tensor([-2.3e-4, -1e-6, -3e-8, -0.0078, 0.0])
    H = len(ld)
    g = torch.Generator().manual_seed(5)
    q, k = (torch.randn(n, 1, 1, K, generator=g).to(dtype).cuda() for _ in range(2))
    v = torch.randn(n, 1, H, V, generator=g).to(dtype).cuda()
    h0 = 30 * torch.randn(1, H, K, V, generator=g)
    cache, ldc = h0.cuda(), ld.cuda()
    for t in range(n):
        o = gdn.linear_attn_decode(q[t], k[t], v[t], ldc, cache)
    S = h0[0].cuda().double()
    R = S.clone()
    gamma = torch.exp(ldc.double())[:, None, None]
    for t in range(n):
        kv = k[t, 0, :, :, None].double() * v[t, 0, :, None, :].double()
        S = gamma * S + kv
        R = (gamma * R + kv).float().double()
    errs = [ref.rel(cache[0, h], R[h]) for h in range(H)]
    exact = [ref.rel(cache[0, h], S[h]) for h in range(H)]
    print(["%.1e" % e for e in errs], ["%.1e" % e for e in exact])
    assert max(errs) <= 5e-6
    assert all(e <= 5e-6 for e, x in zip(exact, ld.tolist()) if x <= -1e-6 or x == 0)
    assert ref.rel(o[0], (q[-1, 0].double() @ R)[:, 0] / K ** 0.5) <= (5e-6 if dtype == torch.float32 else 4e-3)


@pytest.mark.parametrize("K,V", [(64, 64), (128, 96)])
def test_fp32_state_is_rounded_once_a_chunk(K, V):
    """A chunk's 64 products are summed and then added to the state, which is rounded once: with a
    memory of 4096 tokens, 32 chunks in the mean square, 0.42 u sqrt(32) = 2.4 u; the chunk's sum, 0.18
    of the state, by 0.42 u sqrt(32) of itself a chunk, the same again; the decay table's 1 u: about 4 u.
    10 u allowed.  (Added to the state one by one they err by 0.42 u sqrt(2048) = 19 u.)"""
    g = torch.Generator().manual_seed(6)
    T = 8192
    q, k, v = (torch.randn(1, T, 1, D, generator=g).cuda() for D in (K, K, V))
    ld = torch.tensor([-2.0 ** -12], device="cuda")
    h0 = 45 * torch.randn(1, 1, K, V, generator=g).cuda()     # as 2048 tokens leave it
    _, fin = gdn.chunk_linear_attn(q, k, v, ld, initial_state=h0, output_final_state=True)
    # the recurrence in 64 bits, 256 tokens at a time
    S, t = h0[0, 0].double(), torch.arange(256, device="cuda", dtype=torch.float64)
    left = torch.exp((255 - t) * ld.double())[:, None]
    for b in range(0, T, 256):
        S = torch.exp(256 * ld.double()) * S + (k[0, b:b + 256, 0].double() * left).T @ v[0, b:b + 256, 0].double()
    e = ref.rel(fin[0, 0], S)
    print("%.2f u" % (e * 2 ** 24))
    assert e <= 10 * 2.0 ** -24
