"""Group norm with an activation on the GPU against a plain 64-bit form.

Tolerances (relative 2-norm): fp32 outputs and the parameters' gradients are sums and products of
24-bit values, errors grow with the square root of the terms: 5e-6 for up to some 10^5 terms.  bf16
outputs are rounded once, 1.7e-3 in the 2-norm, 2.5e-3 allowed.
"""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from chunked_gated_delta_gdn_gb300 import _lib

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = {F32: 5e-6, BF16: 2.5e-3}


def plain(x, G, w, b, eps, act, z):
    N, C = x.shape[0], x.shape[-1]
    t = x.double().reshape(N, -1, G, C // G)
    mean = t.mean((1, 3), keepdim=True)
    var = (t - mean).square().mean((1, 3), keepdim=True)
    u = ((t - mean) / torch.sqrt(var + eps)).reshape(x.shape)
    if w is not None:
        u = u * w.double()
    if b is not None:
        u = u + b.double()
    f = (lambda v: v * torch.sigmoid(v)) if act == "silu" else (lambda v: v)
    return f(u) if z is None else u * f(z.double())


def rel(x, ref):
    x, ref = x.detach().double(), ref.detach().double()
    assert x.shape == ref.shape and torch.isfinite(x).all()
    return ((x - ref).norm() / ref.norm().clamp(min=1e-30)).item()


def make(shape, dtype, wdt=F32, gate=False, affine=(True, True), seed=0, mean=0.5, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    C = shape[-1]
    x = (r(*shape) * std + mean).to(dtype)
    w = (1 + 0.2 * r(C)).to(wdt) if affine[0] else None
    b = (0.2 * r(C)).to(wdt) if affine[1] else None
    z = r(*shape).to(dtype) if gate else None
    return x, w, b, z, r(*shape).to(dtype)


def check(shape, G, dtype, act="silu", eps=1e-5, **kw):
    x, w, b, z, dy = make(shape, dtype, **kw)
    tol = TOL[dtype]
    out = torch.full_like(x, float("nan"))
    y, mean, rstd = gdn.group_norm_act(x, G, w, b, eps, act, z, out=out, return_stats=True)
    leaves = [t.double().requires_grad_() if t is not None else None for t in (x, w, b, z)]
    want = plain(leaves[0], G, leaves[1], leaves[2], eps, act, leaves[3])
    e = [rel(y, want)]
    have = [t for t in leaves if t is not None]
    grads = dict(zip([i for i, t in enumerate(leaves) if t is not None],
                     torch.autograd.grad(want, have, dy.double())))
    dx, dw, db, dz = gdn.group_norm_act_bwd(dy, x, mean, rstd, G, w, b, act, z)
    e.append(rel(dx, grads[0]))
    assert e[0] <= tol and e[1] <= tol, e
    if w is not None:
        e.append(rel(dw, grads[1]))
        assert e[-1] <= TOL[F32], e
    if b is not None:
        e.append(rel(db, grads[2]))
        assert e[-1] <= TOL[F32], e
    if z is not None:
        e.append(rel(dz, grads[3]))
        assert e[-1] <= tol, e
    else:
        assert dz is None
    print(["%.1e" % v for v in e])
    return y


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape,G", [((5, 64), 4), ((1, 4096), 32), ((300, 4096), 32), ((7, 96), 1),
                                     ((3, 17, 64), 8), ((2, 9, 11, 320), 32), ((2, 4099, 40), 4),
                                     ((9, 13, 15), 5), ((3, 5, 7, 21), 3), ((1, 70000, 8), 2),
                                     ((4, 33, 1000), 2), ((2, 3, 2048), 1), ((2, 1030, 512), 32)])
def test_shapes(shape, G, gate, dtype):
    check(shape, G, dtype, gate=gate)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape,G", [((511, 8, 4), 4), ((300, 2, 16), 2), ((97, 3, 5, 48), 3), ((40, 7, 21), 3),
                                     ((9, 4, 2048), 32), ((5000, 9, 8), 1), ((2, 31, 264), 2)])
def test_many_small_slabs(shape, G, gate, dtype):
    check(shape, G, dtype, gate=gate)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_options(dtype):
    for gate in (False, True):
        check((6, 10, 64), 8, dtype, act=None, gate=gate)
        check((6, 10, 64), 8, dtype, affine=(False, False), gate=gate)
        check((6, 10, 64), 8, dtype, affine=(True, False), gate=gate, wdt=dtype)
        check((6, 128), 4, dtype, affine=(False, True), gate=gate, wdt=dtype, eps=0.3)


def test_mean_far_from_zero():
    """A mean of a thousand deviations: the variance must not come from E[x^2] - E[x]^2.  The
    input's own rounding to 24 bits is 2^-24 * 1000 = 6e-5 of a deviation, but the input is
    given: only the mean's rounding enters, likewise 6e-5 of a deviation at most."""
    for shape, G in (((3, 500, 64), 4), ((40, 1024), 8), ((2, 20000, 16), 2)):
        x, w, b, _, _ = make(shape, F32, mean=1000.0, std=1.0)
        y = gdn.group_norm_act(x, G, w, b, activation=None)
        assert rel(y, plain(x, G, w, b, 1e-5, None, None)) <= 1e-4


def test_constant_and_tiny_groups():
    """Groups without variance, groups of one element: xhat is 0, u the bias, dx 0 or near it."""
    for shape, G in (((4, 32), 32), ((4, 1, 32), 8), ((3, 40, 16), 4), ((2, 6000, 8), 1)):
        x = torch.full(shape, 3.25, device="cuda")
        b = torch.linspace(-2, 2, shape[-1], device="cuda")
        y, mean, rstd = gdn.group_norm_act(x, G, None, b, activation=None, return_stats=True)
        assert torch.equal(y, b.expand(shape))
        dx, dw, db, _ = gdn.group_norm_act_bwd(torch.ones_like(x), x, mean, rstd, G, None, b, None)
        assert dx.abs().max().item() <= 1e-3 and torch.isfinite(dx).all()


def test_large_values_and_non_finite_groups():
    """A NaN or infinity stays in its own (row, group); silu at +-1e4 is finite."""
    x, w, b, z, dy = make((4, 6, 64), F32, gate=True)
    clean = gdn.group_norm_act(x, 8, w, b, gate=z)
    x2 = x.clone()
    x2[1, 3, 17] = float("nan")     # group 2 of row 1
    x2[2, 0, 60] = float("inf")     # group 7 of row 2
    y = gdn.group_norm_act(x2, 8, w, b, gate=z)
    keep = torch.ones(4, 6, 8, 8, dtype=torch.bool, device="cuda")
    keep[1, :, 2] = keep[2, :, 7] = False
    keep = keep.view(4, 6, 64)
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[1, :, 16:24]).all()
    big = torch.tensor([-1e4, 1e4, -100.0, 0.0] * 16, device="cuda").expand(4, 6, 64).contiguous()
    y, mean, rstd = gdn.group_norm_act(x, 8, w, b, gate=big, return_stats=True)
    dx, _, _, dz = gdn.group_norm_act_bwd(dy, x, mean, rstd, 8, w, b, "silu", big)
    assert all(torch.isfinite(t).all() for t in (y, dx, dz))
    assert torch.count_nonzero(y[..., 0::4]).item() == 0


def test_gradients_match_differences():
    """Central differences of the fp64 loss of fp32 outputs along a direction: the truncation
    error is h^2 / 6 of the third derivative, the rounding 1e-7 |loss terms| / h; at h = 1e-2 both
    are below 1e-3 of |grad| |d|."""
    x, w, b, z, dy = make((2, 40, 64), F32, gate=True)
    for gate in (None, z):
        y, mean, rstd = gdn.group_norm_act(x, 8, w, b, gate=gate, return_stats=True)
        dx, dw, db, dz = gdn.group_norm_act_bwd(dy, x, mean, rstd, 8, w, b, "silu", gate)
        args = dict(x=x, w=w, b=b, z=gate)
        loss = lambda a: (gdn.group_norm_act(a["x"], 8, a["w"], a["b"], gate=a["z"]).double() * dy).sum()
        for name, grad in (("x", dx), ("w", dw), ("b", db), ("z", dz)):
            if grad is None:
                continue
            d = torch.randn_like(args[name])
            h = 1e-2
            up, dn = loss({**args, name: args[name] + h * d}), loss({**args, name: args[name] - h * d})
            assert abs((up - dn) / (2 * h) - (grad.double() * d).sum()) <= 2e-3 * grad.norm() * d.norm()


def test_autograd_op_streams_and_repeats():
    x, w, b, z, dy = make((33, 1024), BF16, gate=True, wdt=BF16)
    leaves = [t.requires_grad_() for t in (x, w, b, z)]

    def call():
        y = gdn.group_norm_act_trainable(leaves[0], 8, leaves[1], leaves[2], gate=leaves[3])
        return (y,) + torch.autograd.grad(y, leaves, dy)

    a = call()
    assert [t.dtype for t in a] == [BF16] * 5
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c = call()
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, c))
    y = gdn.group_norm_act_trainable(leaves[0], 8, None, None)
    (dx,) = torch.autograd.grad(y, leaves[:1], dy)
    assert torch.isfinite(dx.float()).all()


def test_graph_capture():
    x, w, b, z, _ = make((3, 300, 64), BF16, gate=True)
    y = torch.empty_like(x)
    gdn.group_norm_act(x, 8, w, b, gate=z, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.group_norm_act(x, 8, w, b, gate=z, out=y)
    x2 = make((3, 300, 64), BF16, seed=5)[0]
    x.copy_(x2)
    g.replay()
    assert rel(y, plain(x2, 8, w, b, 1e-5, "silu", z)) <= TOL[BF16]


def test_elements_past_32_bit_offsets():
    """More than 2^31 elements: the last row against its own norm."""
    N, C, G = 530000, 4096, 32
    x = torch.zeros(N, C, dtype=BF16, device="cuda")
    x[-1] = torch.randn(C, device="cuda").to(BF16)
    y, mean, rstd = gdn.group_norm_act(x, G, activation="silu", return_stats=True)
    assert rel(y[-1:], plain(x[-1:], G, None, None, 1e-5, "silu", None)) <= TOL[BF16]
    dx = gdn.group_norm_act_bwd(x, x, mean, rstd, G, activation="silu")[0]
    t = x[-1:].double().requires_grad_()
    (want,) = torch.autograd.grad(plain(t, G, None, None, 1e-5, "silu", None), t, x[-1:].double())
    assert rel(dx[-1:], want) <= TOL[BF16]


def test_refusals_and_nothing_to_do():
    x, w, b, z, dy = make((3, 4, 32), F32, gate=True)
    with pytest.raises(ValueError, match="groups"):
        gdn.group_norm_act(x, 5)
    with pytest.raises(ValueError, match="activation"):
        gdn.group_norm_act(x, 4, activation="gelu")
    with pytest.raises(ValueError, match="contiguous"):
        gdn.group_norm_act(x.transpose(0, 1), 4)
    with pytest.raises(TypeError):
        gdn.group_norm_act(x.half(), 4)
    with pytest.raises(ValueError):
        gdn.group_norm_act(x, 4, w[:16].contiguous())
    with pytest.raises(TypeError):
        gdn.group_norm_act(x, 4, w.to(BF16))
    with pytest.raises(ValueError):
        gdn.group_norm_act(x, 4, gate=z[:1].contiguous())
    with pytest.raises(_lib.GdnError):
        gdn.group_norm_act(x, 4, eps=-1.0)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.group_norm_act(x.cpu(), 4)
    e = torch.zeros(0, 4, 32, device="cuda")
    assert gdn.group_norm_act(e, 4).shape == e.shape
    y, mean, rstd = gdn.group_norm_act(e, 4, w, b, return_stats=True)
    _, dw, db, _ = gdn.group_norm_act_bwd(e, e, mean, rstd, 4, w, b)
    assert torch.count_nonzero(dw).item() == 0 and torch.count_nonzero(db).item() == 0
