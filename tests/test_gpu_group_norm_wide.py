"""Groups of 513 to 1024 values at a single position and in small slabs: the forward's widest
register form, in both types, with and without a gate, for each vector width.  Against the plain
64-bit form, with the tolerances of test_gpu_group_norm.py (their reasons hold: more terms a sum than
there are here are tested there)."""
import pytest
import torch

from tests.test_gpu_group_norm import BF16, F32, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("shape,G", [((5, 513), 1), ((5, 514), 1), ((5, 516), 1), ((3, 768), 1),
                                     ((4, 1000), 1), ((700, 1024), 1), ((7, 2048), 2), ((1, 4 * 1024), 4),
                                     ((3, 3, 171), 1), ((2, 6, 86), 1), ((3, 8, 96), 1), ((2, 4, 1024), 4)])
def test_wide_groups(shape, G, gate, dtype):
    check(shape, G, dtype, gate=gate)
