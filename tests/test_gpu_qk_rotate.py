"""The norm of queries and keys with rotation on the GPU against a plain 64-bit form.

Tolerances (relative 2-norm): an fp32 output is a few products and a sum of up to 256 squares, each
off by 2^-24, sines and cosines by some 2^-23: 1e-6.  The weights' gradients are sums over tokens and
heads, a thread's part one after the other: sqrt(n) 2^-24 for runs of n up to 10^4, 6e-6 allowed.
bf16 outputs are rounded once: at most 2^-8 of the value, so 2^-8 in the 2-norm; over many values 1.7e-3,
2.5e-3 allowed from 500 values on.  A gradient behind a norm is a difference of two terms, each as
large as the gradient without the second, r d w (heads of one value have next to nothing left of
them): its tolerance is relative to itself, and 1e-6 of those terms.
"""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-6, BF16: 2.5e-3}
NAN = float("nan")


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(0)


def tol(x):
    """The tolerance of an output, of its type and count."""
    return 2.0 ** -8 + 1e-6 if x.dtype is BF16 and x.numel() < 500 else TOL[x.dtype]


def rel(x, ref):
    x, ref = x.detach().double(), ref.detach().double()
    assert x.shape == ref.shape and torch.isfinite(x).all()
    return ((x - ref).norm() / ref.norm().clamp(min=1e-30)).item()


def plain(x, freq, pos, w, norm, eps, sections, interleaved):
    """x [..., H, K] in 64 bits; pos [axes, ...]."""
    if norm == "rms":
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    elif norm == "l2":
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) + eps)
    if w is not None:
        x = x * w
    if freq is None or freq.numel() == 0:
        return x
    n = freq.shape[0]
    axis = [a for a, c in enumerate(sections) for _ in range(c)] if sections else [0] * n
    phi = torch.stack([pos[axis[j]].double() * freq[j].double() for j in range(n)], -1)[..., None, :]
    lo = torch.arange(n, device="cuda") * (2 if interleaved else 1)
    hi = lo + (1 if interleaved else n)
    u, v = x[..., lo], x[..., hi]
    y = x.index_copy(-1, lo, u * torch.cos(phi) - v * torch.sin(phi))
    return y.index_copy(-1, hi, v * torch.cos(phi) + u * torch.sin(phi))


def freqs(R, base=10000.0):
    return (base ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / max(R, 1))).float()


def make(B, T, Hq, Hk, K, dtype, seed=0, wdt=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k = (2 * rn(B, T, Hq, K)).to(dtype), rn(B, T, Hk, K).to(dtype)
    wq, wk = (1 + 0.3 * rn(K)).to(wdt), (1 + 0.3 * rn(K)).to(wdt)
    return q, k, wq, wk, rn(B, T, Hq, K).to(dtype), rn(B, T, Hk, K).to(dtype)


def check(B, T, Hq, Hk, K, R, dtype, norm="rms", eps=1e-6, sections=None, interleaved=False, weights=(True, True),
          positions="some", wdt=F32, view=None, seed=0):
    q, k, wq, wk, dq, dk = make(B, T, Hq, Hk, K, dtype, seed, wdt)
    wq, wk = (wq if weights[0] else None), (wk if weights[1] else None)
    if view is not None:
        q, k = view(q), view(k)
    freq = freqs(R) if R else None
    axes = len(sections) if sections else 1
    g = torch.Generator(device="cuda").manual_seed(seed + 7)
    pos = torch.randint(0, 1 << 20, (axes, B, T), generator=g, device="cuda").to(torch.int32)
    if positions is None:
        pos = torch.arange(T, device="cuda", dtype=torch.int32).expand(axes, B, T)
    given = None if positions is None else pos if axes > 1 else pos[0]
    kw = dict(norm=norm, eps=eps, sections=sections, interleaved=interleaved)
    leaves = [t.detach().double().requires_grad_() if t is not None else None for t in (q, k, wq, wk)]
    want = [plain(leaves[n], freq, pos, leaves[2 + n], norm, eps, sections, interleaved) for n in (0, 1)]
    bufs = [torch.full(t.shape, NAN, dtype=dtype, device="cuda") for t in (q, k)]
    got = gdn.qk_norm_rotate(q, k, freq, given, wq, wk, out_q=bufs[0], out_k=bufs[1], **kw)
    assert got[0] is bufs[0] and got[1] is bufs[1]
    for a, b in zip(got, want):
        assert rel(a, b) <= tol(a)
        assert ((a.double() - b).abs() <= (2.0 ** -8 if dtype is BF16 else 0) * b.abs() + 1e-5 * b.abs().max()).all()
    have = [t for t in leaves if t is not None]
    grads = iter(torch.autograd.grad(want, have, [dq.double(), dk.double()]))
    grads = [next(grads) if t is not None else None for t in leaves]
    mine = gdn.qk_norm_rotate_bwd(dq, dk, q, k, freq, given, wq, wk, **kw)
    for n in (0, 1):
        assert mine[n].dtype is dtype and mine[n].is_contiguous()
        x, w, d = leaves[n], leaves[2 + n], (dq, dk)[n].double()
        r = 1.0 if norm is None else (x.square().mean(-1, keepdim=True) * (1 if norm == "rms" else K) + eps).rsqrt()
        terms = ((d if w is None else d * w.abs().max()) * r).norm()
        assert (mine[n].double() - grads[n]).norm() <= tol(mine[n]) * grads[n].norm() + 1e-6 * terms, n
        if grads[2 + n] is not None:
            assert rel(mine[2 + n], grads[2 + n]) <= 6e-6, n
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,K,R", [
    (1, 1, 1, 1, 128, 128), (2, 7, 4, 2, 64, 64), (1, 300, 16, 4, 128, 128), (3, 33, 6, 2, 80, 40), (1, 19, 5, 3, 96, 96),
    (2, 5, 3, 1, 256, 64), (2, 40, 2, 2, 256, 256), (1, 9, 4, 4, 72, 36), (1, 11, 3, 2, 7, 0), (1, 11, 3, 2, 7, 4),
    (1, 5, 33, 1, 6, 2), (1, 13, 2, 1, 250, 250), (2, 3, 2, 2, 1, 0), (1, 6, 40, 10, 2, 2), (1, 4, 3, 3, 128, 32),
    (1, 3, 7, 5, 255, 254), (5000, 1, 2, 1, 32, 32), (1, 4, 64, 8, 192, 128), (4, 1, 1, 1, 20, 12)])
def test_shapes(B, T, Hq, Hk, K, R, interleaved, dtype):
    check(B, T, Hq, Hk, K, R, dtype, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
def test_norms_and_weights(norm, dtype):
    for K, R in ((128, 128), (48, 20)):
        for weights in ((True, True), (False, False), (True, False), (False, True)):
            check(2, 21, 6, 3, K, R, dtype, norm=norm, weights=weights, wdt=dtype, eps=0.25)
        check(2, 21, 6, 3, K, R, dtype, norm=norm, positions=None)
        check(2, 21, 6, 3, K, 0, dtype, norm=norm)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("K,sections", [(128, (16, 24, 24)), (64, (32,)), (64, (0, 32)), (80, (1, 2, 3, 4)), (128, (40, 0, 8)),
                                        (96, (16, 16, 16))])
def test_axes(K, sections, interleaved, dtype):
    check(2, 37, 6, 2, K, 2 * sum(sections), dtype, sections=sections, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(dtype):
    """Slices of one projection at any element, heads before tokens, one head for all: bit for bit what
    contiguous tensors give."""
    B, T, Hq, Hk = 2, 29, 4, 2
    for K, lead in ((128, 0), (64, 1), (64, 2), (64, 4), (40, 3)):
        wide = torch.randn(B, T, lead + (Hq + 2 * Hk) * K, device="cuda").to(dtype)[..., lead:]
        q = wide[..., :Hq * K].unflatten(-1, (Hq, K))
        k = wide[..., Hq * K:(Hq + Hk) * K].unflatten(-1, (Hk, K))
        pairs = [(q, k), (q.transpose(1, 2).contiguous().transpose(1, 2), k), (q, k[:, :, :1].expand(B, T, Hk, K)),
                 (q.flip(0)[:, ::2], k[:, ::2])]
        for a, b in pairs:
            dq, dk = torch.randn(a.shape, device="cuda").to(dtype), torch.randn(b.shape, device="cuda").to(dtype)
            pos = torch.randint(0, 9999, a.shape[:2], device="cuda").to(torch.int32)
            w = torch.rand(K, device="cuda")
            args = (freqs(K // 2), pos, w, w)
            flat = a.contiguous(), b.contiguous()
            for x, y in zip(gdn.qk_norm_rotate(a, b, *args), gdn.qk_norm_rotate(*flat, *args)):
                assert rel(x, y) <= (1e-6 if dtype is F32 else 2.0 ** -7)
            for x, y in zip(gdn.qk_norm_rotate_bwd(dq, dk, a, b, *args), gdn.qk_norm_rotate_bwd(dq, dk, *flat, *args)):
                assert rel(x, y) <= (6e-6 if x.dtype is F32 else 2.0 ** -7)
    check(2, 15, 3, 3, 64, 64, dtype, view=lambda t: torch.cat([t, t], -1)[..., 64:])
    check(2, 15, 3, 3, 64, 64, dtype, view=lambda t: t.transpose(1, 2).contiguous().transpose(1, 2))
    check(2, 15, 3, 3, 64, 32, dtype, view=lambda t: torch.cat([t[..., :1], t], -1)[..., 1:])


def test_far_positions():
    """Angles of positions over the whole range of int32 to fp32 rounding: 2^-23 of a unit vector's length,
    with the product's and the sum's roundings 1e-6."""
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321, 77], device="cuda",
                       dtype=torch.int32)
    for freq in (freqs(64), torch.rand(32, device="cuda") * 6, -freqs(64), freqs(64, 1e6)):
        q = torch.randn(10, 2, 64, device="cuda")
        got, _ = gdn.qk_norm_rotate(q, q, freq, pos, norm=None)
        # in 64 bits a product of 31 and 24 bits is off by 2^-53 of 2^34 turns: 2^-19 of one; so the exact
        # product is split in two that 53 bits hold
        turn = 2 * torch.pi
        p = pos.double()
        hi = torch.floor(p / 65536) * 65536
        phi = torch.fmod(hi[:, None] * freq.double(), turn) + torch.fmod((p - hi)[:, None] * freq.double(), turn)
        c, s = torch.cos(phi)[:, None], torch.sin(phi)[:, None]
        u, v = q[..., :32].double(), q[..., 32:].double()
        want = torch.cat([u * c - v * s, v * c + u * s], -1)
        assert ((got.double() - want).norm(dim=(1, 2)) <= 2e-6 * want.norm(dim=(1, 2))).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_in_place(dtype):
    q, k, wq, wk, dq, dk = make(2, 50, 5, 2, 96, dtype)
    freq = freqs(96)
    want = gdn.qk_norm_rotate(q, k, freq, None, wq, wk)
    grads = gdn.qk_norm_rotate_bwd(dq, dk, q, k, freq, None, wq, wk)
    got = gdn.qk_norm_rotate(q, k, freq, None, wq, wk, out_q=q, out_k=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert all(torch.isfinite(t).all() for t in grads)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_requests_of_one_token(dtype):
    """[n, H, K] and positions [n] are rows of one token."""
    q, k, wq, wk, dq, dk = make(9, 1, 4, 2, 64, dtype)
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 1000
    a = gdn.qk_norm_rotate(q, k, freqs(64), pos[:, None], wq, wk)
    b = gdn.qk_norm_rotate(q[:, 0], k[:, 0], freqs(64), pos, wq, wk)
    assert b[0].shape == (9, 4, 64) and torch.equal(a[0][:, 0], b[0]) and torch.equal(a[1][:, 0], b[1])
    c = gdn.qk_norm_rotate(q.transpose(0, 1), k.transpose(0, 1), freqs(64), pos[None], wq, wk)
    assert torch.equal(c[0][0], b[0]) and torch.equal(c[1][0], b[1])
    a = gdn.qk_norm_rotate_bwd(dq, dk, q, k, freqs(64), pos[:, None], wq, wk)
    b = gdn.qk_norm_rotate_bwd(dq[:, 0], dk[:, 0], q[:, 0], k[:, 0], freqs(64), pos, wq, wk)
    assert all(torch.equal(s.reshape(t.shape), t) for s, t in zip(a, b))


def test_rows_of_zeros_and_non_finite_values():
    """Zeros stay zeros; a NaN or infinity stays in its head."""
    q, k, wq, wk, dq, dk = make(1, 12, 4, 4, 64, F32)
    q[0, 3], k[0, 5, 1] = 0.0, 0.0
    freq = freqs(64)
    for norm in ("rms", "l2", None):
        a, b = gdn.qk_norm_rotate(q, k, freq, None, wq, wk, norm=norm)
        assert not a[0, 3].any() and not b[0, 5, 1].any() and torch.isfinite(a).all()
        da, _, _, _ = gdn.qk_norm_rotate_bwd(dq, dk, q, k, freq, None, wq, wk, norm=norm)
        assert torch.isfinite(da).all()
        q2 = q.clone()
        q2[0, 7, 2, 9], q2[0, 8, 1, 40] = NAN, float("inf")
        c, d = gdn.qk_norm_rotate(q2, k, freq, None, wq, wk, norm=norm)
        hit = torch.zeros(1, 12, 4, dtype=torch.bool, device="cuda")
        hit[0, 7, 2] = hit[0, 8, 1] = True
        assert torch.equal(c[~hit], a[~hit]) and torch.equal(d, b) and not torch.isfinite(c[hit]).all(-1).any()


@pytest.mark.parametrize("norm", ["rms", "l2", None])
def test_gradients_against_differences(norm):
    """Along random directions, of the 64-bit form: central differences at 1e-4 are off by some 1e-8 of the
    gradient, the fp32 gradients by 6e-6."""
    q, k, wq, wk, dq, dk = make(2, 9, 3, 2, 24, F32, seed=4)
    freq, pos = freqs(16), torch.randint(0, 5000, (2, 9), device="cuda").to(torch.int32)
    grads = gdn.qk_norm_rotate_bwd(dq, dk, q, k, freq, pos, wq, wk, norm=norm)

    def loss(q, k, wq, wk):
        a, b = (plain(x, freq, pos[None], w, norm, 1e-6, None, False) for x, w in ((q, wq), (k, wk)))
        return (a * dq.double()).sum() + (b * dk.double()).sum()

    at = [t.double() for t in (q, k, wq, wk)]
    for n, p in enumerate(at):
        v = torch.randn(p.shape, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").double()
        ends = [loss(*at[:n], p + e * v, *at[n + 1:]) for e in (1e-4, -1e-4)]
        want = (ends[0] - ends[1]).item() / 2e-4
        size = (grads[n].double() * v).norm().item() * v.numel() ** 0.5
        assert abs((grads[n].double() * v).sum().item() - want) <= 1e-5 * size, n


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd(dtype):
    q, k, wq, wk, dq, dk = make(2, 30, 4, 2, 64, dtype, wdt=dtype)
    freq = freqs(64)
    both = torch.cat([q, k], 2).requires_grad_()
    wq.requires_grad_()
    qv, kv = both[:, :, :4], both[:, :, 4:]
    a, b = gdn.qk_norm_rotate_trainable(qv, kv, freq, None, wq, wk, norm="l2", eps=1e-5)
    got = torch.autograd.grad((a, b), (both, wq), (dq, dk), retain_graph=True)
    want = gdn.qk_norm_rotate_bwd(dq, dk, qv.detach(), kv.detach(), freq, None, wq.detach(), wk, norm="l2", eps=1e-5)
    assert torch.equal(got[0], torch.cat(want[:2], 2)) and torch.equal(got[1], want[2].to(dtype))
    only = torch.autograd.grad(a.sum(), both)[0]
    assert not only[:, :, 4:].any() and only[:, :, :4].any()
    a, b = gdn.qk_norm_rotate_trainable(both[:, :, :4], both[:, :, 4:], freq)
    with pytest.raises(RuntimeError, match="second derivative"):
        g, = torch.autograd.grad(a.float().square().sum(), both, create_graph=True)
        g.float().sum().backward()
    with pytest.raises(ValueError, match="inv_freq"):
        gdn.qk_norm_rotate_trainable(qv, kv, freq.clone().requires_grad_())


def test_same_bits_streams_and_graphs():
    q, k, wq, wk, dq, dk = make(2, 700, 8, 2, 128, BF16)
    freq = freqs(128)
    run = lambda: gdn.qk_norm_rotate(q, k, freq, None, wq, wk) + gdn.qk_norm_rotate_bwd(dq, dk, q, k, freq, None, wq, wk)
    want = run()
    assert all(torch.equal(a, b) for _ in range(3) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append(g)
    q.copy_(q.flip(1))
    want = run()
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out in outs for a, b in zip(out, want))


def test_offsets_beyond_32_bits():
    """Rows behind element 2^31 and 2^32."""
    B, T, H, K = 1, 140000, 256, 128
    if torch.cuda.mem_get_info()[0] < 10 * B * T * H * K:
        pytest.skip("not enough free memory")
    q = torch.empty(B, T, H, K, dtype=BF16, device="cuda").normal_()
    k = torch.randn(B, T, 1, K, device="cuda").to(BF16)
    freq = freqs(K)
    a, _ = gdn.qk_norm_rotate(q, k, freq)
    da, _, _, _ = gdn.qk_norm_rotate_bwd(q, k, q, k, freq, need_weights=False)
    for t in (65536, 131072, T - 4):
        pos = torch.arange(t, t + 4, device="cuda")[None, None]
        x = q[:, t:t + 4].double().requires_grad_()
        want = plain(x, freq, pos, None, "rms", 1e-6, None, False)
        assert rel(a[:, t:t + 4], want) <= TOL[BF16]
        assert rel(da[:, t:t + 4], torch.autograd.grad(want, x, x.detach())[0]) <= TOL[BF16]


def test_refusals():
    q, k, wq, wk, _, _ = make(2, 6, 4, 2, 32, F32)
    f, freq = gdn.qk_norm_rotate, freqs(32)
    with pytest.raises(TypeError):
        f(q, k.bfloat16())
    with pytest.raises(TypeError):
        f(q.half(), k.half())
    with pytest.raises(ValueError, match="go with"):
        f(q, k[:, :5])
    with pytest.raises(ValueError, match="go with"):
        f(q, k[..., :30])
    with pytest.raises(ValueError, match="B, T, H, K"):
        f(q[0, 0], k[0, 0])
    with pytest.raises(ValueError, match="next to each other"):
        f(q.transpose(2, 3).contiguous().transpose(2, 3), k)
    with pytest.raises(ValueError, match="1 to 256"):
        f(torch.zeros(1, 1, 1, 257, device="cuda"), torch.zeros(1, 1, 1, 257, device="cuda"))
    with pytest.raises(ValueError, match="inv_freq"):
        f(q, k, freqs(34))
    with pytest.raises(TypeError):
        f(q, k, freq.double())
    with pytest.raises(TypeError):
        f(q, k, freq, torch.zeros(2, 6, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError, match="positions"):
        f(q, k, freq, torch.zeros(2, 7, device="cuda", dtype=torch.int32))
    for sections in ((8, 9), (), (-1, 17), (4, 4, 4, 2, 2)):
        with pytest.raises(ValueError, match="sections"):
            f(q, k, freq, sections=sections)
    with pytest.raises(ValueError, match="positions"):
        f(q, k, freq, torch.zeros(2, 6, device="cuda", dtype=torch.int32), sections=(8, 8))
    with pytest.raises(ValueError, match="q_weight"):
        f(q, k, freq, None, wq[:31])
    with pytest.raises(TypeError):
        f(q, k, freq, None, wq, wk.bfloat16())
    with pytest.raises(ValueError, match="norm"):
        f(q, k, norm="layer")
    for eps in (-1.0, NAN):
        with pytest.raises(ValueError, match="eps"):
            f(q, k, eps=eps)
    with pytest.raises(ValueError, match="out_q"):
        f(q, k, out_q=k)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.qk_norm_rotate_bwd(q[:, :1].expand(2, 6, 4, 32), k, q, k)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.qk_norm_rotate_bwd(q, k, q, k, workspace=torch.empty(1 << 20, dtype=torch.uint8))


def test_nothing_to_do():
    for B, T in ((0, 4), (3, 0)):
        q, k, wq, wk, dq, dk = make(B, T, 2, 1, 16, F32)
        a, b = gdn.qk_norm_rotate(q, k, freqs(16), None, wq, wk)
        assert a.shape == q.shape and b.shape == k.shape
        _, _, dwq, dwk = gdn.qk_norm_rotate_bwd(dq, dk, q, k, freqs(16), None, wq, wk)
        assert not dwq.any() and not dwk.any()
