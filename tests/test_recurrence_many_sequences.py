"""The gated linear recurrence counts packed sequences in 32 bits and halves sums of two such counts: more than
2^30 of them are refused, on the host and before anything is launched."""
import pytest

from chunked_gated_delta_gdn_gb300 import _lib
from tests.test_recurrence_abi import FAKE, NONE, bwd, fwd

MOST = 1 << 30


def test_more_sequences_than_the_search_counts():
    # (an output at an odd address is refused later than sizes are, and a missing workspace later still)
    assert fwd(B=1, cu=FAKE, N=MOST + 1, y=FAKE + 1) == _lib.GDN_ERR_SHAPE
    assert fwd(B=1, cu=FAKE, N=(1 << 31) - 2, y=FAKE + 1) == _lib.GDN_ERR_SHAPE
    assert fwd(B=1, cu=FAKE, N=MOST, y=FAKE + 1) == _lib.GDN_ERR_LAYOUT
    assert bwd(B=1, cu=FAKE, N=MOST + 1) == _lib.GDN_ERR_SHAPE
    assert bwd(B=1, cu=FAKE, N=MOST) == _lib.GDN_ERR_WORKSPACE
    # rows are searched by division: there may be more of them
    assert fwd(B=MOST + 1, T=1, y=FAKE + 1) == _lib.GDN_ERR_LAYOUT
    assert bwd(B=MOST + 1, T=1) == _lib.GDN_ERR_WORKSPACE


def test_sizes_of_their_scratch():
    L = _lib.load()
    assert L.gdn_linear_recurrence_fwd_workspace_size(1, 64, 8, MOST + 1) == NONE
    assert L.gdn_linear_recurrence_bwd_workspace_size(1, 64, 8, MOST + 1, 0) == NONE
    assert L.gdn_linear_recurrence_fwd_workspace_size(1, 64, 8, MOST) != NONE
    assert L.gdn_linear_recurrence_fwd_workspace_size(MOST + 1, 1, 8, MOST + 1) != NONE


@pytest.mark.gpu
def test_binding_refuses_them():
    torch = pytest.importorskip("torch")
    import chunked_gated_delta_gdn_gb300 as gdn
    if torch.cuda.mem_get_info()[0] < 6 << 30:
        pytest.skip("not enough free memory")
    x = torch.zeros(1, 4, 8, device="cuda")
    cu = torch.zeros(MOST + 2, dtype=torch.int32, device="cuda")
    for call in (gdn.gated_linear_recurrence, gdn.gated_linear_recurrence_trainable):
        with pytest.raises(ValueError, match="sequences"):
            call(x, x, cu_seqlens=cu)
    with pytest.raises(ValueError, match="sequences"):
        gdn.gated_linear_recurrence_bwd(x, x, x, cu_seqlens=cu)
