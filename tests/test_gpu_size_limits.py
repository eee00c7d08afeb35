"""Sizes that do not fit the C interface's 32-bit integers are refused, not cut down to what fits."""
import pytest
import torch

import chunked_gated_delta_gdn_gb300 as gdn

pytestmark = pytest.mark.gpu


def empty(*shape):
    """bf16 [shape], untouched memory."""
    need = 2
    for s in shape:
        need *= s
    if torch.cuda.mem_get_info()[0] < 2 * need + (1 << 30):
        pytest.skip("not enough free memory")
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda")


def test_group_norm_positions():
    x = empty(1, 65536, 65537, 1)     # 2^32 + 2^16 positions
    for call in (gdn.group_norm_act, gdn.group_norm_act_trainable):
        with pytest.raises(ValueError, match="sizes"):
            call(x, 1)
    s = torch.zeros(1, 1, device="cuda")
    with pytest.raises(ValueError, match="sizes"):
        gdn.group_norm_act_bwd(x, x, s, s, 1)


def test_linear_attention_tokens():
    x = empty(1, (1 << 32) + 64, 1, 8)
    ld = torch.zeros(1, device="cuda")
    with pytest.raises(ValueError, match="sizes"):
        gdn.chunk_linear_attn(x, x, x, ld)
    with pytest.raises(ValueError, match="sizes"):
        gdn.chunk_linear_attn_trainable(x, x, x, ld)
