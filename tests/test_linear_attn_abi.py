"""Argument checks of the linear attention and group norm entry points, on the host (CPU only)."""
import pytest

from chunked_gated_delta_gdn_gb300 import _lib

FAKE = 1 << 20   # never dereferenced: every call below fails validation first or has nothing to do
NAN = float("nan")


def fwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, B=1, T=64, Hqk=1, Hv=1, K=64, V=64, io=_lib.GDN_F32,
             scale=NAN, init=None, ofs=0, fin=None, cu=None, N=1, si=None, slots=0, o=FAKE, ws=None,
             wsb=0, status=None, stream=None)
    a.update(kw)
    return _lib.load().gdn_linear_attn_chunk_fwd(*a.values())


def bwd(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, B=1, T=64, Hqk=1, Hv=2, K=64, V=64, io=_lib.GDN_F32,
             scale=NAN, init=None, cu=None, N=1, do=FAKE, dfin=None, dq=FAKE, dk=FAKE, dv=FAKE,
             dinit=None, ws=None, wsb=0, status=None, stream=None)
    a.update(kw)
    return _lib.load().gdn_linear_attn_chunk_bwd(*a.values())


def dec(**kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, s=FAKE, slots=8, idx=None, n=4, Hqk=1, Hv=1, K=128,
             V=128, io=_lib.GDN_BF16, scale=NAN, o=FAKE, status=None, stream=None)
    a.update(kw)
    return _lib.load().gdn_linear_attn_decode(*a.values())


@pytest.mark.parametrize("call", [fwd, bwd])
def test_chunk_calls_reject_bad_arguments(call):
    assert call(q=None) == _lib.GDN_ERR_NULL
    assert call(ld=None) == _lib.GDN_ERR_NULL
    assert call(Hv=3, Hqk=2) == _lib.GDN_ERR_SHAPE
    assert call(K=0) == _lib.GDN_ERR_SHAPE
    assert call(V=130) == _lib.GDN_ERR_SHAPE
    assert call(K=6) == _lib.GDN_ERR_SHAPE
    assert call(K=4, io=_lib.GDN_BF16) == _lib.GDN_ERR_SHAPE
    assert call(io=7) == _lib.GDN_ERR_DTYPE
    assert call(B=2, cu=FAKE) == _lib.GDN_ERR_SHAPE
    assert call(cu=FAKE, N=-1) == _lib.GDN_ERR_SHAPE
    assert call(B=1 << 16, T=1 << 16) == _lib.GDN_ERR_SHAPE
    assert call(q=FAKE + 4) == _lib.GDN_ERR_LAYOUT
    assert call(ld=FAKE + 2) == _lib.GDN_ERR_LAYOUT
    assert call(B=0) == _lib.GDN_OK
    assert call(T=0, cu=FAKE, N=0) == _lib.GDN_OK


def test_forward_and_backward_own_arguments():
    lib = _lib.load()
    assert fwd(ofs=1) == _lib.GDN_ERR_NULL
    assert fwd(o=None) == _lib.GDN_ERR_NULL
    assert fwd(si=FAKE) == _lib.GDN_ERR_SHAPE
    assert fwd(init=FAKE + 4) == _lib.GDN_ERR_LAYOUT
    assert bwd(dq=None) == _lib.GDN_ERR_NULL
    assert bwd(do=FAKE + 8) == _lib.GDN_ERR_LAYOUT
    assert bwd(dinit=FAKE + 8) == _lib.GDN_ERR_LAYOUT
    need = lib.gdn_linear_attn_chunk_bwd_workspace_size(1, 64, 1, 2, 64, 64, 1, _lib.GDN_F32)
    assert need >= 64 * 2 * 64 * 4          # two value heads share a query/key head
    assert bwd() == _lib.GDN_ERR_WORKSPACE
    assert bwd(ws=FAKE, wsb=need - 1) == _lib.GDN_ERR_WORKSPACE
    assert bwd(ws=FAKE + 16, wsb=need) == _lib.GDN_ERR_LAYOUT
    for fn in (lib.gdn_linear_attn_chunk_fwd_workspace_size, lib.gdn_linear_attn_chunk_bwd_workspace_size):
        assert fn(1, 64, 2, 3, 64, 64, 1, 0) == (1 << 64) - 1
        assert fn(1, 64, 1, 1, 64, 64, -1, 0) == (1 << 64) - 1


def test_decode_rejects_bad_arguments():
    assert dec(s=None) == _lib.GDN_ERR_NULL
    assert dec(n=9) == _lib.GDN_ERR_SHAPE
    assert dec(n=-1) == _lib.GDN_ERR_SHAPE
    assert dec(Hv=3, Hqk=2) == _lib.GDN_ERR_SHAPE
    assert dec(io=3) == _lib.GDN_ERR_DTYPE
    assert dec(s=FAKE + 8) == _lib.GDN_ERR_LAYOUT
    assert dec(n=0) == _lib.GDN_OK


def test_group_norm_rejects_bad_arguments():
    lib = _lib.load()

    def gf(**kw):
        a = dict(x=FAKE, w=FAKE, b=FAKE, z=None, N=2, L=3, C=32, G=4, io=_lib.GDN_BF16,
                 wb=_lib.GDN_F32, eps=1e-5, act=_lib.GDN_ACT_SILU, y=FAKE, mean=None, rstd=None,
                 ws=None, wsb=0, stream=None)
        a.update(kw)
        return lib.gdn_group_norm_act_fwd(*a.values())

    def gb(**kw):
        a = dict(dy=FAKE, x=FAKE, w=FAKE, b=FAKE, z=None, mean=FAKE, rstd=FAKE, N=2, L=3, C=32, G=4,
                 io=_lib.GDN_BF16, wb=_lib.GDN_F32, act=_lib.GDN_ACT_SILU, dx=FAKE, dz=None, dw=FAKE,
                 db=FAKE, ws=None, wsb=0, stream=None)
        a.update(kw)
        return lib.gdn_group_norm_act_bwd(*a.values())

    for call in (gf, gb):
        assert call(G=5) == _lib.GDN_ERR_SHAPE
        assert call(G=0) == _lib.GDN_ERR_SHAPE
        assert call(N=-1) == _lib.GDN_ERR_SHAPE
        assert call(N=1 << 20, L=1 << 20) == _lib.GDN_ERR_SHAPE
        assert call(io=4) == _lib.GDN_ERR_DTYPE
        assert call(io=_lib.GDN_F32, wb=_lib.GDN_BF16) == _lib.GDN_ERR_DTYPE
        assert call(act=9) == _lib.GDN_ERR_UNSUPPORTED
        assert call(x=None) == _lib.GDN_ERR_NULL
        assert call(x=FAKE + 2) == _lib.GDN_ERR_LAYOUT
        assert call(w=FAKE + 1) == _lib.GDN_ERR_LAYOUT
    assert gf(eps=-1.0) == _lib.GDN_ERR_SHAPE
    assert gf(eps=NAN) == _lib.GDN_ERR_SHAPE
    assert gf(N=0) == _lib.GDN_OK
    assert gb(z=FAKE) == _lib.GDN_ERR_NULL          # a gate without its gradient
    assert gb(N=0, dw=None, db=None) == _lib.GDN_OK
    for fn in (lib.gdn_group_norm_act_fwd_workspace_size, lib.gdn_group_norm_act_bwd_workspace_size):
        assert fn(2, 3, 32, 5, 0) == (1 << 64) - 1


def test_bindings_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    import chunked_gated_delta_gdn_gb300 as gdn
    x = torch.zeros(1, 4, 1, 8)
    ld = torch.zeros(1)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.chunk_linear_attn(x, x, x, ld)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.linear_attn_decode(x[0], x[0], x[0], ld, torch.zeros(4, 1, 8, 8))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.group_norm_act(x, 1)
