"""Argument checks of the gated linear recurrence and of the norm of q and k with rotation, on the host
(CPU only)."""
import ctypes

import pytest

from chunked_gated_delta_gdn_gb300 import _lib

FAKE = 1 << 20   # never dereferenced: every call below fails validation first or has nothing to do
NAN = float("nan")
NONE = (1 << 64) - 1


def fwd(**kw):
    a = dict(x=FAKE, g=FAKE, i=None, lam=None, c=8.0, px=64, pg=64, pi=64, B=2, T=16, D=64, io=_lib.GDN_BF16,
             gd=_lib.GDN_F32, init=None, ofs=0, fin=None, cu=None, N=0, si=None, slots=0, y=FAKE, carries=None,
             ws=None, wsb=0, status=None, stream=None)
    a.update(kw)
    return _lib.load().gdn_linear_recurrence_fwd(*a.values())


def bwd(**kw):
    a = dict(x=FAKE, g=FAKE, i=None, lam=None, c=8.0, px=64, pg=64, pi=64, B=2, T=16, D=64, io=_lib.GDN_BF16,
             gd=_lib.GDN_F32, init=None, cu=None, N=0, dy=FAKE, dfin=None, carries=None, dx=FAKE, dg=FAKE, di=None,
             dlam=None, dinit=None, ws=None, wsb=0, status=None, stream=None)
    a.update(kw)
    return _lib.load().gdn_linear_recurrence_bwd(*a.values())


def dec(**kw):
    a = dict(x=FAKE, g=FAKE, i=None, lam=None, c=8.0, px=64, pg=64, pi=64, n=4, D=64, io=_lib.GDN_BF16,
             gd=_lib.GDN_BF16, s=FAKE, slots=8, idx=None, y=FAKE, status=None, stream=None)
    a.update(kw)
    return _lib.load().gdn_linear_recurrence_decode(*a.values())


@pytest.mark.parametrize("call", [fwd, bwd, dec])
def test_recurrence_calls_reject_bad_arguments(call):
    assert call(x=None) == _lib.GDN_ERR_NULL
    assert call(g=None) == _lib.GDN_ERR_NULL
    assert call(lam=FAKE) == _lib.GDN_ERR_NULL              # fused gates without the input gate
    assert call(i=FAKE) == _lib.GDN_ERR_NULL                # an input gate without lam
    assert call(D=0) == _lib.GDN_ERR_SHAPE
    assert call(px=63) == _lib.GDN_ERR_SHAPE
    assert call(pg=0) == _lib.GDN_ERR_SHAPE
    assert call(lam=FAKE, i=FAKE, pi=1) == _lib.GDN_ERR_SHAPE
    for c in (-1.0, NAN, float("inf")):
        assert call(lam=FAKE, i=FAKE, c=c) == _lib.GDN_ERR_SHAPE
    assert call(io=7) == _lib.GDN_ERR_DTYPE
    assert call(io=_lib.GDN_F32, gd=_lib.GDN_BF16) == _lib.GDN_ERR_DTYPE
    assert call(x=FAKE + 1) == _lib.GDN_ERR_LAYOUT
    assert call(lam=FAKE + 2, i=FAKE) == _lib.GDN_ERR_LAYOUT


def test_recurrence_batches():
    for call in (fwd, bwd):
        assert call(B=2, cu=FAKE) == _lib.GDN_ERR_SHAPE
        assert call(B=1, cu=FAKE, N=-1) == _lib.GDN_ERR_SHAPE
        assert call(B=-1) == _lib.GDN_ERR_SHAPE
        assert call(B=1 << 16, T=1 << 15) == _lib.GDN_ERR_SHAPE
        assert call(B=0) == _lib.GDN_OK
        assert call(B=1, T=0, cu=FAKE, N=0) == _lib.GDN_OK
        assert call(B=1, cu=FAKE + 2, N=3) == _lib.GDN_ERR_LAYOUT
        assert call(init=FAKE + 2) == _lib.GDN_ERR_LAYOUT
    assert fwd(y=None) == _lib.GDN_ERR_NULL
    assert fwd(ofs=1) == _lib.GDN_ERR_NULL
    assert fwd(si=FAKE) == _lib.GDN_ERR_SHAPE
    assert fwd(si=FAKE, slots=4) == _lib.GDN_ERR_SHAPE      # slots of no cache
    assert bwd(dx=None) == _lib.GDN_ERR_NULL
    assert bwd(di=FAKE) == _lib.GDN_ERR_NULL
    assert bwd(lam=FAKE, i=FAKE) == _lib.GDN_ERR_NULL       # an input gate without its gradient
    assert bwd() == _lib.GDN_ERR_WORKSPACE
    lib = _lib.load()
    need = lib.gdn_linear_recurrence_bwd_workspace_size(2, 16, 64, 2, 0)
    assert bwd(ws=FAKE, wsb=need - 1) == _lib.GDN_ERR_WORKSPACE
    assert bwd(ws=FAKE + 16, wsb=need) == _lib.GDN_ERR_LAYOUT
    assert lib.gdn_linear_recurrence_carries_size(2, 65, 3) == 5 * 3 * 4
    assert lib.gdn_linear_recurrence_carries_size(2, 65, 0) == NONE
    assert lib.gdn_linear_recurrence_fwd_workspace_size(2, 16, 64, 2) == 0      # one tile a sequence
    long = dict(B=1, T=1 << 20, D=64, px=64, pg=64)                             # a chain that is cut into segments
    need = lib.gdn_linear_recurrence_fwd_workspace_size(1, 1 << 20, 64, 1)
    if need:                                                                    # (not where there is one SM, or none)
        assert fwd(**long) == _lib.GDN_ERR_WORKSPACE
        assert fwd(**long, ws=FAKE, wsb=need - 1) == _lib.GDN_ERR_WORKSPACE
        assert fwd(**long, ws=FAKE + 128, wsb=need) == _lib.GDN_ERR_LAYOUT
    assert lib.gdn_linear_recurrence_fwd_workspace_size(1, 1 << 20, 0, 1) == NONE
    assert lib.gdn_linear_recurrence_bwd_workspace_size(2, -1, 3, 2, 0) == NONE


def test_recurrence_decode():
    assert dec(n=9) == _lib.GDN_ERR_SHAPE
    assert dec(n=-1) == _lib.GDN_ERR_SHAPE
    assert dec(s=None) == _lib.GDN_ERR_NULL
    assert dec(s=FAKE + 2) == _lib.GDN_ERR_LAYOUT
    assert dec(n=0) == _lib.GDN_OK


def qk(back=False, **kw):
    strides = (ctypes.c_longlong * 3)(1 << 10, 64, 32)
    a = dict(q=FAKE, k=FAKE, qs=strides, ks=strides, B=2, T=16, Hq=2, Hk=1, K=32, R=32, io=_lib.GDN_BF16,
             norm=_lib.GDN_NORM_RMS, eps=1e-6, wq=None, wk=None, wd=_lib.GDN_F32, freq=FAKE, pos=None, axes=1,
             sections=None, inter=0, oq=FAKE, ok=FAKE, dwq=None, dwk=None, ws=None, wsb=0, stream=None)
    a.update(kw)
    lib = _lib.load()
    if back:
        return lib.gdn_qk_norm_rotate_bwd(FAKE, a.pop("dk", FAKE), *a.values())
    for n in ("dwq", "dwk", "ws", "wsb"):
        del a[n]
    return lib.gdn_qk_norm_rotate_fwd(*a.values())


@pytest.mark.parametrize("back", [False, True])
def test_qk_calls_reject_bad_arguments(back):
    call = lambda **kw: qk(back, **kw)
    ints = lambda *v: (ctypes.c_int * len(v))(*v)
    assert call(q=None) == _lib.GDN_ERR_NULL
    assert call(ks=None) == _lib.GDN_ERR_NULL
    assert call(freq=None) == _lib.GDN_ERR_NULL
    assert call(ok=None) == _lib.GDN_ERR_NULL
    for bad in (dict(K=0, R=0), dict(K=257), dict(R=31), dict(R=34), dict(R=-2), dict(Hq=0), dict(Hk=-1), dict(B=-1),
                dict(B=1 << 16, T=1 << 15), dict(eps=-1.0), dict(eps=NAN), dict(axes=0), dict(axes=5),
                dict(axes=2, sections=ints(8, 9)), dict(axes=2, sections=ints(8, 7)),
                dict(axes=2, sections=ints(-1, 17)), dict(qs=(ctypes.c_longlong * 3)(-1, 1, 1))):
        assert call(**bad) == _lib.GDN_ERR_SHAPE, bad
    assert call(axes=2) == _lib.GDN_ERR_NULL
    assert call(norm=3) == _lib.GDN_ERR_UNSUPPORTED
    assert call(io=2) == _lib.GDN_ERR_DTYPE
    assert call(io=_lib.GDN_F32, wd=_lib.GDN_BF16) == _lib.GDN_ERR_DTYPE
    assert call(q=FAKE + 1) == _lib.GDN_ERR_LAYOUT
    assert call(wk=FAKE + 2) == _lib.GDN_ERR_LAYOUT
    assert call(pos=FAKE + 2) == _lib.GDN_ERR_LAYOUT
    assert call(oq=FAKE + 1) == _lib.GDN_ERR_LAYOUT
    assert call(B=0) == _lib.GDN_OK
    if back:
        need = _lib.load().gdn_qk_norm_rotate_bwd_workspace_size(2, 16, 2, 1, 32, 1)
        assert call(dwq=FAKE) == _lib.GDN_ERR_WORKSPACE
        assert call(dwq=FAKE, ws=FAKE, wsb=need - 1) == _lib.GDN_ERR_WORKSPACE
        assert call(dwq=FAKE, ws=FAKE + 128, wsb=need) == _lib.GDN_ERR_LAYOUT
        assert call(dwq=FAKE + 2) == _lib.GDN_ERR_LAYOUT
        assert _lib.load().gdn_qk_norm_rotate_bwd_workspace_size(2, 16, 2, 1, 300, 1) == NONE


def test_bindings_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    import chunked_gated_delta_gdn_gb300 as gdn
    x = torch.zeros(1, 4, 8)
    for call in (gdn.gated_linear_recurrence, gdn.gated_linear_recurrence_trainable):
        with pytest.raises(ValueError, match="CUDA"):
            call(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gated_linear_recurrence_fused_gates(x, x, x, x[0, 0])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gated_linear_recurrence_decode(x[0], x[0], x[0])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.qk_norm_rotate(x[None], x[None])
    with pytest.raises(TypeError, match="torch.Tensor"):
        gdn.gated_linear_recurrence(None, x)
    with pytest.raises(TypeError, match="torch.Tensor"):
        gdn.qk_norm_rotate(None, x)


@pytest.mark.parametrize("call", [fwd, bwd, dec])
def test_widest_rows(call):
    """A row's bytes are counted in 32 bits: rows beyond 2^28 channels are refused."""
    wide = (1 << 28) + 1
    assert call(D=wide, px=wide, pg=wide) == _lib.GDN_ERR_SHAPE
    L = _lib.load()
    assert L.gdn_linear_recurrence_carries_size(1, 1, wide) == (1 << 64) - 1
    assert L.gdn_linear_recurrence_fwd_workspace_size(1, 1, wide, 1) == (1 << 64) - 1
    assert L.gdn_linear_recurrence_bwd_workspace_size(1, 1, wide, 1, 1) == (1 << 64) - 1
