"""The norm of q and k with rotation where the gradients take the place of those that come in (dq in d_q, dk in
d_k), as the C interface allows: bit for bit what separate tensors get.  The kernel copies heads ahead while it
stores earlier ones; token counts here leave a second, smaller run and groups of lanes with nothing to do."""
import ctypes

import pytest
import torch

from chunked_gated_delta_gdn_gb300 import _lib
from tests.test_gpu_qk_rotate import BF16, F32, freqs, make

pytestmark = pytest.mark.gpu


def backward(d_q, d_k, q, k, freq, wq, wk, interleaved, dq, dk):
    """The C call; (dq_weight, dk_weight)."""
    L = _lib.load()
    B, T, Hq, K = q.shape
    Hk = k.shape[2]
    dt = _lib.GDN_BF16 if q.dtype is BF16 else _lib.GDN_F32
    strides = [(ctypes.c_longlong * 3)(*t.stride()[:3]) for t in (q, k)]
    dwq, dwk = torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    need = L.gdn_qk_norm_rotate_bwd_workspace_size(B, T, Hq, Hk, K, 1)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    rc = L.gdn_qk_norm_rotate_bwd(
        d_q.data_ptr(), d_k.data_ptr(), q.data_ptr(), k.data_ptr(), *strides, B, T, Hq, Hk, K, 2 * freq.numel(), dt,
        _lib.GDN_NORM_RMS, 1e-6, wq.data_ptr(), wk.data_ptr(), _lib.GDN_F32, freq.data_ptr(), None, 1, None, interleaved,
        dq.data_ptr(), dk.data_ptr(), dwq.data_ptr(), dwk.data_ptr(), ws.data_ptr(), need,
        torch.cuda.current_stream().cuda_stream)
    assert rc == _lib.GDN_OK, _lib.status_string(rc)
    return dwq, dwk


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [0, 1])
@pytest.mark.parametrize("B,T,Hq,Hk,K,R", [(1, 9731, 12, 12, 128, 128), (2, 9731, 12, 12, 128, 128), (2, 2501, 32, 8, 128, 64),
                                           (1, 4999, 6, 2, 80, 40), (1, 1, 3, 1, 64, 64), (3, 777, 5, 3, 7, 6),
                                           (1, 1303, 4, 1, 256, 256), (1, 3001, 7, 5, 34, 34)])
def test_gradients_in_the_incoming_ones_place(B, T, Hq, Hk, K, R, interleaved, dtype):
    q, k, wq, wk, d_q, d_k = make(B, T, Hq, Hk, K, dtype)
    freq = freqs(R)
    dq, dk = torch.full_like(d_q, float("nan")), torch.full_like(d_k, float("nan"))
    want = backward(d_q, d_k, q, k, freq, wq, wk, interleaved, dq, dk)
    for _ in range(3):
        a, b = d_q.clone(), d_k.clone()
        got = backward(a, b, q, k, freq, wq, wk, interleaved, a, b)
        assert torch.equal(a, dq) and torch.equal(b, dk)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
