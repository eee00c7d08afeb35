"""A call that the CUDA runtime refuses returns its error once: the next call, of any operator, is not
told of it.  The refusals are made on the host, by calls on the legacy stream while another stream
records a graph."""
import ctypes

import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn
from chunked_gated_delta_gdn_gb300 import _lib

pytestmark = pytest.mark.gpu
NAN = float("nan")


def runtime():
    """The CUDA runtime that torch uses (libgdn has its own, linked in)."""
    for line in open("/proc/self/maps"):
        if "libcudart" in line:
            return ctypes.CDLL(line.split()[-1])
    pytest.skip("torch's CUDA runtime is not a shared library")


def refused(call):
    """The status of a call on the legacy stream while a stream that waits for it records a graph."""
    rt, stream, graph = runtime(), ctypes.c_void_p(), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert rt.cudaStreamCreate(ctypes.byref(stream)) == 0
    assert rt.cudaStreamBeginCapture(stream, 0) == 0
    try:
        return call()
    finally:
        rt.cudaStreamEndCapture(stream, ctypes.byref(graph))
        if graph.value:
            rt.cudaGraphDestroy(graph)
        rt.cudaStreamDestroy(stream)
        rt.cudaGetLastError()   # (torch's runtime: the recording has failed)


def norm_without_elements(lib, p):
    return lib.gdn_group_norm_act_bwd(p, p, None, None, None, p, p, 0, 3, 32, 4, _lib.GDN_F32, _lib.GDN_F32,
                                      _lib.GDN_ACT_SILU, p, None, p, p, None, 0, None)


def attention_without_sequences(lib, p):
    return lib.gdn_linear_attn_chunk_fwd(p, p, p, p, 1, 4, 1, 1, 16, 16, _lib.GDN_F32, NAN, None, 0, None, p, 0,
                                         None, 0, p, None, 0, None, None)


def attention_gradients_without_sequences(lib, p):
    return lib.gdn_linear_attn_chunk_bwd(p, p, p, p, 1, 4, 1, 1, 16, 16, _lib.GDN_F32, NAN, None, p, 0, p, None,
                                         p, p, p, None, None, 0, None, None)


def norm(lib, p):
    return lib.gdn_group_norm_act_fwd(p, None, None, None, 2, 3, 32, 4, _lib.GDN_F32, _lib.GDN_F32, 1e-5,
                                      _lib.GDN_ACT_SILU, p, None, None, None, 0, None)


@pytest.mark.parametrize("first", [norm_without_elements, attention_without_sequences,
                                   attention_gradients_without_sequences, norm])
def test_a_refused_call_leaves_nothing_behind(first):
    lib = _lib.load()
    buf = torch.zeros(4096, device="cuda")
    x = torch.randn(4, 64, device="cuda")
    cache = torch.randn(1, 1, 16, 16, device="cuda")
    q = torch.randn(1, 1, 16, device="cuda")
    ld = torch.full((1,), -0.1, device="cuda")
    want = gdn.group_norm_act(x, 8)
    twin = cache.clone()
    o = gdn.linear_attn_decode(q, q, q, ld, twin)
    for call in (lambda: gdn.group_norm_act(x, 8), lambda: gdn.linear_attn_decode(q, q, q, ld, cache)):
        assert refused(lambda: first(lib, buf.data_ptr())) == _lib.GDN_ERR_CUDA
        got = call()
        assert torch.equal(got, want if got.dim() == 2 else o)
    assert torch.equal(cache, twin)
