"""The gated linear recurrence on the GPU against the 64-bit recurrence.

Tolerances (relative 2-norm).  A state is a sum over the tokens of its memory, at most 2000 here, each
with a factor of its own of a few roundings of 2^-24; they have no common sign, so some
sqrt(2000) 2^-24 = 2.7e-6 of it may be off: fp32 outputs, states and their gradients 1e-5.  bf16
outputs are rounded once: at most 2^-8 of the value, so 2^-8 in the 2-norm; over many values 1.7e-3,
2.5e-3 allowed from 500 values on.  Gradients
of the gates add one more factor, and 1 / sqrt(1 - a^2) is at most 100 times their own terms' size
where a channel keeps 0.9999 of its state: it multiplies terms of a's own rounding, within the same
1e-5.  dlam is a sum over all tokens: likewise.
"""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from tests.recurrence_ref import recurrence

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 1e-5, BF16: 2.5e-3}
NAN = float("nan")


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(0)


def tol(x):
    """The tolerance of an output, of its type and count."""
    return 2.0 ** -8 + 1e-5 if x.dtype is BF16 and x.numel() < 500 else TOL[x.dtype]


def rel(x, ref):
    x, ref = x.detach().double(), ref.detach().double()
    assert x.shape == ref.shape and torch.isfinite(x).all()
    if ref.numel() == 0:
        return 0.0
    return ((x - ref).norm() / ref.norm().clamp(min=1e-30)).item()


def make(shape, dtype, gdt=None, fused=False, seed=0):
    """(x, g) or (x, r, i, lam)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    gdt = gdt or dtype
    x = rn(*shape).to(dtype)
    if not fused:
        return x, (-torch.exp(1.5 * rn(*shape) - 3.0)).to(gdt)
    u = 0.9 + 0.0999 * torch.rand(shape[-1], generator=gen, device="cuda")
    return x, rn(*shape).to(gdt), rn(*shape).to(gdt), torch.log(torch.expm1(-torch.log(u) / 8.0))


def forward(ins, **kw):
    return (gdn.gated_linear_recurrence if len(ins) == 2 else gdn.gated_linear_recurrence_fused_gates)(*ins, **kw)


def backward(ins, dy, **kw):
    """The gradients of ins, then of the initial states."""
    if len(ins) == 2:
        return gdn.gated_linear_recurrence_bwd(*ins, dy, **kw)
    return gdn.gated_linear_recurrence_bwd_fused_gates(*ins, dy, **kw)


def reference(ins, h0=None, lens=None, dy=None, dfin=None):
    """(y, final states, gradients of ins and h0) in 64 bits."""
    leaves = [t.detach().double().requires_grad_() for t in ins]
    B, D = ins[0].shape[0], ins[0].shape[-1]
    N = B if lens is None else len(lens)
    h = (torch.zeros(N, D, device="cuda") if h0 is None else h0).double().requires_grad_()
    y, fin = recurrence(*leaves[:2], *(leaves[2:] or (None, None)), h0=h, lens=lens)
    if dy is None:
        return y, fin, None
    loss = (y * dy.double()).sum() + (0 if dfin is None else (fin * dfin.double()).sum())
    if not loss.requires_grad:      # no sequence
        return y, fin, [torch.zeros_like(t) for t in leaves + [h]]
    got = torch.autograd.grad(loss, leaves + [h], allow_unused=True)
    return y, fin, [torch.zeros_like(t) if g is None else g for g, t in zip(got, leaves + [h])]


def check(shape, dtype, gdt=None, fused=False, lens=None, state=True, seed=0):
    ins = make(shape, dtype, gdt, fused, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    B, T, D = shape
    N = B if lens is None else len(lens)
    h0 = torch.randn(N, D, generator=gen, device="cuda") if state else None
    dfin = torch.randn(N, D, generator=gen, device="cuda") if state else None
    dy = torch.randn(*shape, generator=gen, device="cuda").to(dtype)
    cu = None
    if lens is not None:
        cu = torch.tensor([sum(lens[:n]) for n in range(N + 1)], dtype=torch.int32, device="cuda")
    y, fin, grads = reference(ins, h0, lens, dy, dfin)
    out = torch.full(shape, NAN, dtype=dtype, device="cuda")
    got, got_fin, carries = forward(ins, initial_state=h0, output_final_state=True, cu_seqlens=cu, out=out,
                                    return_carries=True, check=True)
    assert got is out
    assert rel(got, y) <= tol(got)
    assert rel(got_fin, fin) <= TOL[F32]
    # a rounding to bf16 is off by 2^-8 of the value at most, element by element
    scale = y.abs().max().item() if y.numel() else 0.0
    assert ((got.double() - y).abs() <= (2.0 ** -8 if dtype is BF16 else 0) * y.abs() + 3e-5 * scale).all()
    for c in (carries, None):
        have = backward(ins, dy, d_final_state=dfin, initial_state=h0, cu_seqlens=cu, carries=c, check=True)
        names = ["dx", "dg", "dh0"] if not fused else ["dx", "dr", "di", "dlam", "dh0"]
        for name, a, b, t in zip(names, have, grads, list(ins) + [None]):
            want = dtype if name == "dx" else F32 if name in ("dh0", "dlam") else t.dtype
            assert a.dtype is want
            assert rel(a, b) <= tol(a), name
    return ins


SHAPES = [(1, 1, 1), (1, 1, 8), (2, 3, 5), (1, 17, 64), (3, 129, 40), (2, 300, 333), (1, 1000, 130), (16, 70, 64),
          (5, 128, 2), (1, 128, 66), (1, 513, 1), (2, 256, 34), (130, 1, 16), (40, 7, 24)]


@pytest.mark.parametrize("dtype,gdt", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_dense(shape, fused, dtype, gdt):
    check(shape, dtype, gdt, fused, state=shape[1] != 128)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("lens,tail", [([0, 1, 0, 5, 130, 0, 257, 1, 1, 16, 15], 0), ([1] * 70, 3), ([0, 0, 0], 40),
                                       ([300], 1), ([128, 128, 256], 0), ([], 9), ([16] * 40, 0), ([0, 700, 0], 200),
                                       ([3, 900, 2], 0), ([1, 2, 3, 4, 5, 6, 7, 8, 9] * 20, 129), ([0], 0)])
def test_packed(lens, tail, fused, dtype):
    for D in (48, 131):
        check((1, sum(lens) + tail, D), dtype, None, fused, lens=lens)


@pytest.mark.parametrize("fused", [False, True])
def test_many_short_sequences(fused):
    """More sequences than tokens a CTA holds, empty ones among them in long runs."""
    gen = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 3, (700,), generator=gen).tolist()
    lens[100:400] = [0] * 300
    check((1, sum(lens), 20), F32, None, fused, lens=lens)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fused", [False, True])
def test_slots(fused, dtype):
    """A slot cache: padding and bad slots' rows are zero whatever their input, other slots keep every bit."""
    lens, D = [5, 0, 140, 33, 1, 64], 70
    ins = make((1, sum(lens) + 7, D), dtype, None, fused)
    for t in ins[:3]:
        t[:, 145:178] = NAN       # sequence 3, padding
        t[:, sum(lens):] = NAN    # no sequence's
    cu = torch.tensor([0, 5, 5, 145, 178, 179, 243], dtype=torch.int32, device="cuda")
    slots = torch.tensor([7, 2, 0, -1, 9, 5], dtype=torch.int32, device="cuda")
    cache = torch.randn(12, D, device="cuda")
    before = cache.clone()
    live = [0, 1, 2, 4, 5]
    cut = lambda t: torch.cat([t[:, :145], t[:, 178:243]], 1)
    want, fin, _ = reference([cut(t) if t.dim() == 3 else t for t in ins], before[slots.long()[live]],
                             [lens[n] for n in live])
    out = torch.full(ins[0].shape, NAN, dtype=dtype, device="cuda")
    y, got = forward(ins, initial_state=cache, output_final_state=True, cu_seqlens=cu, state_indices=slots, out=out,
                     check=True)
    assert got is cache
    assert rel(torch.cat([y[:, :145], y[:, 178:243]], 1), want) <= TOL[dtype]
    assert not y[:, 145:178].any() and not y[:, 243:].any()
    at = slots.long()[live]
    assert rel(cache[at], fin) <= TOL[F32]
    assert torch.equal(cache[slots[1]], before[slots[1]])
    rest = torch.ones(12, dtype=torch.bool)
    rest[at.cpu()] = False
    assert torch.equal(cache[rest.cuda()], before[rest.cuda()])
    # into another cache; no states wanted; a bad slot
    other = torch.full_like(cache, NAN)
    y2, _ = forward(ins, initial_state=before, output_final_state=True, cu_seqlens=cu, state_indices=slots,
                    final_state=other)
    assert torch.equal(y2, y) and torch.equal(other[at], cache[at]) and other[rest.cuda()].isnan().all()
    y3, none = forward(ins, initial_state=before, cu_seqlens=cu, state_indices=slots)
    assert none is None and torch.equal(y3, y)
    slots[3] = 12
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y4, _ = forward(ins, initial_state=before, cu_seqlens=cu, state_indices=slots, dev_status=status)
    assert torch.equal(y4, y) and status.item() == 1
    with pytest.raises(gdn.GdnDeviceError, match="SLOT"):
        forward(ins, initial_state=before, cu_seqlens=cu, state_indices=slots, check=True)


@pytest.mark.parametrize("cu", [[1, 5, 9], [0, 6, 5], [0, 4, 21], [0, -3, 7], [0, 1 << 30, 8]])
def test_bad_packed_lengths(cu):
    """Reported; zero rows and gradients, states left alone."""
    x, g = make((1, 20, 70), F32)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h0 = torch.randn(2, 70, device="cuda")
    fin = torch.full_like(h0, 3.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(x, NAN)
    y, _ = gdn.gated_linear_recurrence(x, g, h0, True, cu, final_state=fin, dev_status=status, out=out)
    assert status.item() == 2 and not y.any() and (fin == 3.0).all()
    status.zero_()
    grads = gdn.gated_linear_recurrence_bwd(x, g, x, h0, h0, cu, dev_status=status)
    assert status.item() == 2 and not any(t.any() for t in grads)
    x, r, i, lam = make((1, 20, 70), BF16, fused=True)
    grads = gdn.gated_linear_recurrence_bwd_fused_gates(x, r, i, lam, x, None, initial_state=h0, cu_seqlens=cu)
    assert not any(t.any() for t in grads)
    with pytest.raises(gdn.GdnDeviceError, match="CU_SEQLENS"):
        gdn.gated_linear_recurrence(x, r, cu_seqlens=cu, check=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,lead", [(64, 0), (64, 1), (40, 2), (33, 3), (2, 1), (128, 8)])
def test_slices_of_a_projection(D, lead, dtype):
    """Rows apart from each other and at any element give what contiguous ones give, bit for bit."""
    wide = torch.randn(2, 150, 3 * D + lead, device="cuda").to(dtype)
    x, r, i = wide[..., lead:].split(D, -1)
    lam = torch.linspace(-6, 1, D, device="cuda")
    dy = torch.randn(2, 150, D, device="cuda").to(dtype)
    got = forward((x, r, i, lam))[0]
    flat = [t.contiguous() for t in (x, r, i)]
    want = forward((*flat, lam))[0]
    assert torch.equal(got, want)
    for a, b in zip(backward((x, r, i, lam), dy)[:4], backward((*flat, lam), dy)[:4]):
        assert torch.equal(a, b)
    y1, y2 = forward((x, -r.abs()))[0], forward((flat[0], -flat[1].abs()))[0]
    assert torch.equal(y1, y2)
    state = torch.randn(150, D, device="cuda")
    s2 = state.clone()
    y1 = gdn.gated_linear_recurrence_decode_fused_gates(x[0], r[0], i[0], lam, state)
    y2 = gdn.gated_linear_recurrence_decode_fused_gates(flat[0][0], flat[1][0], flat[2][0], lam, s2)
    assert torch.equal(y1, y2) and torch.equal(state, s2)


@pytest.mark.parametrize("fused", [False, True])
def test_gradients_against_differences(fused):
    """Along random directions: (L(p + e v) - L(p - e v)) / 2e of the 64-bit recurrence is off by e^2
    times a third derivative, some 1e-8 of the gradient at e = 1e-4; the fp32 gradients' own 1e-5
    decides."""
    ins = make((2, 40, 6), F32, fused=fused, seed=3)
    h0 = torch.randn(2, 6, device="cuda")
    dy, dfin = torch.randn(2, 40, 6, device="cuda"), torch.randn(2, 6, device="cuda")
    grads = backward(ins, dy, d_final_state=dfin, initial_state=h0)

    def loss(ps):
        y, fin = recurrence(*ps[:2], *(ps[2:-1] or (None, None)), h0=ps[-1])
        return (y * dy.double()).sum() + (fin * dfin.double()).sum()

    at = [t.double() for t in ins] + [h0.double()]
    for n, p in enumerate(at):
        for seed in range(3):
            v = torch.randn(p.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").double()
            ends = [loss(at[:n] + [p + e * v] + at[n + 1:]) for e in (1e-4, -1e-4)]
            want = (ends[0] - ends[1]).item() / 2e-4
            size = (grads[n].double() * v).norm().item() * v.numel() ** 0.5
            assert abs((grads[n].double() * v).sum().item() - want) <= 2e-5 * size, n


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_autograd(fused, dtype):
    """The autograd op: what forward and backward give, with and without states, packed, and in parts."""
    op = gdn.gated_linear_recurrence_fused_gates_trainable if fused else gdn.gated_linear_recurrence_trainable
    cu = torch.tensor([0, 30, 30, 171], dtype=torch.int32, device="cuda")
    for packed in (False, True):
        ins = make((1, 200, 36) if packed else (3, 100, 36), dtype, fused=fused)
        h0 = torch.randn(3, 36, device="cuda", requires_grad=True)
        leaves = [t.requires_grad_() for t in ins]
        kw = dict(cu_seqlens=cu) if packed else {}
        dy, dfin = torch.randn_like(ins[0]), torch.randn(3, 36, device="cuda")
        y, fin = op(*leaves, initial_state=h0, output_final_state=True, **kw)
        plain = [t.detach() for t in ins]
        y2, fin2 = forward(plain, initial_state=h0.detach(), output_final_state=True, **kw)
        assert torch.equal(y, y2) and torch.equal(fin, fin2)
        got = torch.autograd.grad((y, fin), leaves + [h0], (dy, dfin), retain_graph=True)
        want = backward(plain, dy, d_final_state=dfin, initial_state=h0.detach(), **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        # the states alone; y alone without states; a gradient from a sum (no memory of its own)
        got = torch.autograd.grad(fin, leaves + [h0], dfin)
        want = backward(plain, torch.zeros_like(dy), d_final_state=dfin, initial_state=h0.detach(), **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        y, fin = op(*leaves, **kw)
        assert fin is None
        got = torch.autograd.grad(y.sum(), leaves)
        want = backward(plain, torch.ones_like(dy), need_d_initial_state=False, **kw)
        assert want[-1] is None and all(torch.equal(a, b) for a, b in zip(got, want))
        y, _ = op(*leaves, **kw)
        with pytest.raises(RuntimeError, match="second derivative"):
            gx, = torch.autograd.grad(y.float().square().sum(), leaves[0], create_graph=True)
            gx.float().sum().backward()


@pytest.mark.parametrize("dtype,gdt", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("n,D", [(1, 1), (3, 33), (64, 512), (5, 130), (700, 8)])
def test_decode(n, D, fused, dtype, gdt):
    ins = make((n, D), dtype, gdt, fused)
    cache = torch.randn(n + 3, D, device="cuda")
    before = cache.clone()
    idx = torch.randperm(n + 3, device="cuda")[:n].to(torch.int32)
    if n > 2:
        idx[1] = -1
        for t in ins[:3]:
            if t.dim() == 2:
                t[1] = NAN
    step = gdn.gated_linear_recurrence_decode_fused_gates if fused else gdn.gated_linear_recurrence_decode
    args = ins if not fused else ins[:4]
    out = torch.full_like(ins[0], NAN)
    y = step(*args, cache, idx, out=out, check=True)
    on = idx >= 0
    pick = lambda t: t[on].double()[:, None] if t.dim() == 2 else t.double()
    want, fin = recurrence(*(pick(t) for t in ins[:2]), *([pick(t) for t in ins[2:]] or (None, None)),
                           h0=before[idx[on].long()].double())
    # two terms, which may cancel: each is off by a few 2^-24 of itself, so the sum by 1e-6 of their sizes;
    # the output is rounded once more
    args64 = [pick(t) for t in ins]
    args64[0] = args64[0].abs()
    _, size = recurrence(*args64[:2], *(args64[2:] or (None, None)), h0=before[idx[on].long()].double().abs())
    assert y is out and not y[~on].any()
    assert ((cache[idx[on].long()].double() - fin).abs() <= 1e-6 * size).all()
    half = 2.0 ** -8 if dtype is BF16 else 2.0 ** -24
    assert ((y[on].double() - want[:, 0]).abs() <= 1e-6 * size + half * want[:, 0].abs()).all()
    rest = torch.ones(n + 3, dtype=torch.bool, device="cuda")
    rest[idx[on].long()] = False
    assert torch.equal(cache[rest], before[rest])
    idx[0] = n + 3
    with pytest.raises(gdn.GdnDeviceError, match="SLOT"):
        step(*args, cache, idx, check=True)
    # request i in slot i
    a, b = before.clone(), before.clone()
    ar = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(step(*args, a)[:1], step(*args, b, ar)[:1]) and torch.equal(a[:1], b[:1])


@pytest.mark.parametrize("fused", [False, True])
def test_decode_follows_the_forward(fused):
    """4000 tokens one by one and at once, a constant decay of a memory of 4000 tokens among them: the two
    differ by roundings that do not add up in one direction, sqrt(4000) 2^-24 = 4e-6."""
    ins = list(make((1, 4000, 24), F32, fused=fused))
    if not fused:
        ins[1][..., :8] = -1.0 / 4000
    y, fin = forward(ins, output_final_state=True)
    state = torch.zeros(1, 24, device="cuda")
    step = gdn.gated_linear_recurrence_decode_fused_gates if fused else gdn.gated_linear_recurrence_decode
    for t in range(4000):
        args = [v[:, t] for v in ins[:3] if v.dim() == 3] + ([ins[3]] if fused else [])
        o = step(*args, state)
    assert rel(o, y[:, -1]) <= TOL[F32] and rel(state, fin) <= TOL[F32]


def test_constant_decays():
    """The same decay at every token: its rounding would err in one direction all the way.  Against the
    closed sums in 64 bits, sqrt(8192) 2^-24 = 5.4e-6 of rounding without direction."""
    T, D = 8192, 64
    g = -torch.logspace(-5, 0, D, device="cuda").expand(1, T, D).contiguous()
    x = torch.rand(1, T, D, device="cuda")
    y, fin = gdn.gated_linear_recurrence(x, g, output_final_state=True)
    back = torch.arange(T - 1, -1, -1, device="cuda", dtype=torch.float64)
    want = (torch.exp(back[:, None] * g[0, 0].double()) * x[0].double()).sum(0)
    assert rel(fin[0], want) <= 1e-5
    dx, dg, _ = gdn.gated_linear_recurrence_bwd(x, g, torch.ones_like(x))
    n = torch.arange(T, 0, -1, device="cuda", dtype=torch.float64)
    a = torch.exp(g[0, 0].double())
    assert rel(dx[0], -torch.expm1(n[:, None] * g[0, 0].double()) / (1 - a)) <= 1e-5


def test_gates_at_their_ends():
    """Log-decays of -inf and 0; recurrence gates that are shut (a = 1, nothing enters, no slope) and wide
    open; lam that never decays."""
    x, g = make((1, 40, 6), F32)
    g[:, 10] = -float("inf")
    g[:, 20:30] = 0.0
    y, _ = gdn.gated_linear_recurrence(x, g)
    assert rel(y, reference((x, g))[0]) <= TOL[F32]
    assert torch.equal(y[:, 10], x[:, 10])
    dx, dg, _ = gdn.gated_linear_recurrence_bwd(x, g, x)
    assert torch.isfinite(dx).all() and torch.isfinite(dg).all() and not dg[:, 10].any()
    x, r, i, lam = make((1, 40, 6), F32, fused=True)
    r[:, 10:20] = -200.0
    r[:, 20:30] = 50.0
    lam[0], lam[1], lam[2] = -200.0, 60.0, -30.0
    ins = (x, r, i, lam)
    h0 = torch.randn(1, 6, device="cuda")
    y, fin, grads = reference(ins, h0, None, x)
    got, _ = forward(ins, initial_state=h0)
    assert rel(got, y) <= TOL[F32]
    for name, a, b in zip(("dx", "dr", "di", "dlam", "dh0"), backward(ins, x, initial_state=h0), grads):
        assert rel(a, b) <= TOL[F32], name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_non_finite_values_stay_in_their_sequence(dtype):
    """A NaN or infinity reaches what follows in its sequence and channel (backwards: what is before it),
    and nothing else."""
    lens = [20, 130, 1, 300, 33]
    cu = torch.tensor([0, 20, 150, 151, 451, 484], dtype=torch.int32, device="cuda")
    x, g = make((1, 484, 66), dtype)
    dy = torch.randn_like(x)
    h0 = torch.randn(5, 66, device="cuda")
    y, fin = gdn.gated_linear_recurrence(x, g, h0, True, cu)
    grads = gdn.gated_linear_recurrence_bwd(x, g, dy, initial_state=h0, cu_seqlens=cu)
    for bad in (NAN, float("inf")):
        for t, first, last in ((0, 0, 20), (149, 20, 150), (151, 151, 451), (300, 151, 451), (150, 150, 151)):
            n = cu.tolist().index(first)
            x2 = x.clone()
            x2[0, t, 5] = bad
            y2, fin2 = gdn.gated_linear_recurrence(x2, g, h0, True, cu)
            hit = torch.zeros_like(y, dtype=torch.bool)
            hit[0, t:last, 5] = True
            assert torch.equal(y2[~hit], y[~hit]) and not torch.isfinite(y2[0, t, 5])
            keep = torch.ones_like(fin, dtype=torch.bool)
            keep[n, 5] = False
            assert torch.equal(fin2[keep], fin[keep])
            d2 = dy.clone()
            d2[0, t, 5] = bad
            got = gdn.gated_linear_recurrence_bwd(x, g, d2, initial_state=h0, cu_seqlens=cu)
            hit = torch.zeros_like(y, dtype=torch.bool)
            hit[0, first:t + 1, 5] = True
            for a, b in zip(got[:2], grads[:2]):
                assert torch.equal(a[~hit], b[~hit])
            assert torch.equal(got[2][keep], grads[2][keep])


def test_same_bits_every_time():
    for fused in (False, True):
        ins = make((1, 3000, 200), BF16, fused=fused)
        dy = torch.randn_like(ins[0])
        first = forward(ins, output_final_state=True), backward(ins, dy)
        for _ in range(3):
            again = forward(ins, output_final_state=True), backward(ins, dy)
            for a, b in zip(first, again):
                assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_streams_and_graphs():
    """On another stream, and captured: forward, backward and decode replayed on new inputs, two graphs in
    turn."""
    ins = make((2, 400, 96), BF16, fused=True)
    dy = torch.randn_like(ins[0])
    want = forward(ins, output_final_state=True) + tuple(backward(ins, dy))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = forward(ins, output_final_state=True) + tuple(backward(ins, dy))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    state = torch.zeros(400, 96, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(forward(ins, output_final_state=True) + tuple(backward(ins, dy)) + (
                gdn.gated_linear_recurrence_decode_fused_gates(ins[0][0], ins[1][0], ins[2][0], ins[3], state),))
        graphs.append(g)
    new = make((2, 400, 96), BF16, fused=True, seed=9)
    want = forward(new, output_final_state=True) + tuple(backward(new, dy))
    for a, b in zip(ins, new):
        a.copy_(b)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    check_state = torch.zeros(400, 96, device="cuda")
    for _ in range(4):
        y = gdn.gated_linear_recurrence_decode_fused_gates(new[0][0], new[1][0], new[2][0], new[3], check_state)
    assert torch.equal(state, check_state) and torch.equal(outs[1][-1], y)


def test_offsets_beyond_32_bits():
    """Rows behind element 2^31 and 2^32 of the tensors."""
    D, T = 16384, 300000
    if torch.cuda.mem_get_info()[0] < 8 * 2 * D * T:
        pytest.skip("not enough free memory")
    x = torch.empty(1, T, D, dtype=BF16, device="cuda").normal_()
    g = torch.full((1, T, D), -2.0, dtype=BF16, device="cuda")
    y, fin = gdn.gated_linear_recurrence(x, g, output_final_state=True)
    dx, dg, _ = gdn.gated_linear_recurrence_bwd(x, g, x, need_d_initial_state=False)
    for t in (131072 + 5, 262144 + 7, T - 60):     # a decay of e^-2 forgets 60 tokens by far
        want, _, (wx, wg, _) = reference((x[:, t - 60:t + 60], g[:, t - 60:t + 60]), dy=x[:, t - 60:t + 60])
        assert rel(y[:, t:t + 30], want[:, 60:90]) <= TOL[BF16]
        assert rel(dx[:, t:t + 30], wx[:, 60:90]) <= TOL[BF16]
        assert rel(dg[:, t:t + 30], wg[:, 60:90]) <= TOL[BF16]
    assert rel(fin, want[:, -1]) <= TOL[F32]


def test_refusals():
    x, g = make((2, 6, 8), F32)
    f = gdn.gated_linear_recurrence
    with pytest.raises(TypeError):
        f(x, g.bfloat16())                                # fp32 inputs, bf16 gates
    with pytest.raises(TypeError):
        f(x.half(), g)
    with pytest.raises(ValueError, match="shape"):
        f(x, g[:, :5])
    with pytest.raises(ValueError, match="B, T, D"):
        f(x[0], g[0])
    with pytest.raises(ValueError, match="rows"):
        f(x.transpose(1, 2).contiguous().transpose(1, 2), g)
    with pytest.raises(ValueError, match="rows"):
        f(x[:, :1].expand(2, 6, 8), g)                    # overlapping rows
    with pytest.raises(ValueError, match="rows"):
        f(torch.zeros(3, 6, 8, device="cuda")[::2, ::2], g[:, :3])
    with pytest.raises(ValueError, match="B == 1"):
        f(x, g, cu_seqlens=torch.tensor([0, 6], dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        f(x[:1], g[:1], cu_seqlens=torch.tensor([0, 6], device="cuda"))
    with pytest.raises(ValueError, match="initial_state"):
        f(x, g, torch.zeros(3, 8, device="cuda"))
    with pytest.raises(ValueError, match="slot cache"):
        f(x, g, state_indices=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        f(x, g, out=torch.zeros(2, 6, 9, device="cuda"))
    with pytest.raises(ValueError, match="channels"):
        f(x[..., :0], g[..., :0])
    lam = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="lam"):
        gdn.gated_linear_recurrence_fused_gates(x, g, g, lam[:7])
    for c in (-1.0, NAN, float("inf")):
        with pytest.raises(ValueError, match="c must"):
            gdn.gated_linear_recurrence_fused_gates(x, g, g, lam, c)
    with pytest.raises(ValueError, match="carries"):
        gdn.gated_linear_recurrence_bwd(x, g, x, carries=torch.zeros(2, 8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        gdn.gated_linear_recurrence_bwd(x, g, x[:, :1].expand(2, 6, 8))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gated_linear_recurrence_bwd(x, g, x, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="state"):
        gdn.gated_linear_recurrence_decode(x[0], g[0], torch.zeros(6, 9, device="cuda"))
    with pytest.raises(gdn.GdnError, match="SHAPE"):
        gdn.gated_linear_recurrence_decode(x[0], g[0], torch.zeros(5, 8, device="cuda"))   # fewer slots than requests


def test_nothing_to_do():
    x, g = make((0, 6, 8), BF16)
    y, fin = gdn.gated_linear_recurrence(x, g, output_final_state=True)
    assert y.shape == (0, 6, 8) and fin.shape == (0, 8)
    x, g = make((3, 0, 8), BF16)
    h0 = torch.randn(3, 8, device="cuda")
    y, fin = gdn.gated_linear_recurrence(x, g, h0, True)
    assert y.shape == (3, 0, 8) and torch.equal(fin, h0)
    dx, dg, dh0 = gdn.gated_linear_recurrence_bwd(x, g, x, h0, h0)
    assert torch.equal(dh0, h0)
    assert gdn.gated_linear_recurrence_decode(x[0], g[0], h0).shape == (0, 8)
    x, r, i, lam = make((0, 6, 8), BF16, fused=True)
    assert not gdn.gated_linear_recurrence_bwd_fused_gates(x, r, i, lam, x)[3].any()
