"""Group norm's launches are planned for the SMs of the device at hand (none here: one set of rows), and the
scratch that a call asks for says so."""
import pytest

from chunked_gated_delta_gdn_gb300 import _lib


def test_scratch_follows_the_device():
    torch = pytest.importorskip("torch")
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 0
    # a row of 4096 channels in 32 groups of 128: 16 lanes of 8 bf16 channels a group, a CTA holds 16 groups
    # (two CTAs a set of rows), two CTAs an SM; a set's partial sums are two floats a channel
    need = _lib.load().gdn_group_norm_act_bwd_workspace_size(100000, 1, 4096, 32, _lib.GDN_BF16)
    assert need == max(1, 2 * sms // 2) * 2 * 4096 * 4
