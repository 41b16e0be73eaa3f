"""V2 attention over a paged cache with offsets of sequences that are none: the
status word says so, and nothing but the rows of the output is written."""

import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from test_gpu_paged import BF16, call, i32, make

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("max_new", [0, 1])
@pytest.mark.parametrize("cu", [[5, LOW, HIGH], [0, LOW, LOW], [HIGH, LOW, 3], [HIGH, 0, HIGH], [LOW, HIGH, 0], [7, LOW + 1, -1]],
                         ids=str)
def test_offsets_of_any_value(cu, max_new):
    """Differences of offsets need not fit 32 bits."""
    T = 60
    t = make([30, 30], [200, 150], 16, 4, 2, 128)
    t["cu"], t["sl"] = i32(cu), i32([0, 0])
    big = torch.full((3 * T, 4, 128), 7.0, dtype=BF16, device="cuda")
    out = big[T:2 * T]
    call(t, out=out, max_new=max_new)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    assert bool((big[:T] == 7).all()) and bool((big[2 * T:] == 7).all())
    assert bool(((out == 0) | (out == 7)).all())
    assert bd.diffattn_get_device_status() == bd.DA_OK
