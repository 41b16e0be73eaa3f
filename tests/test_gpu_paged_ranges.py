"""V2 attention over a paged cache at the ends of its ranges: large values."""

import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from test_gpu_paged import BF16, call, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert bd.diffattn_get_device_status() == bd.DA_OK


@pytest.mark.parametrize("rise", [20, 40, 72])
@pytest.mark.parametrize("n,h,d", [(1, 4, 128), (4, 4, 64), (2, 4, 64), (60, 4, 128), (20, 4, 64), (60, 1, 128)])
def test_large_values_under_rising_scores(n, h, d, rise):
    """Values of 2^73 where the scores rise by `rise` powers of two from the first key to the last (half as many for
    every other pair of heads): no sum leaves fp32.  There are as many sequences as keep most items whole, so that a
    maximum of the first tile is that of all the others until it is raised."""
    L = [600] * (2 * torch.cuda.get_device_properties(0).multi_processor_count)
    t = make([n] * len(L), L, 64, h, 1, d, seed=3)
    t["q"][:] = 1.0
    t["q"][:, 2::4] = t["q"][:, 3::4] = 0.5
    j = torch.arange(600, device="cuda")
    at = (t["table"].long()[:, j // 64], (j % 64)[None])
    t["k"][at] = torch.linspace(0.0, rise / (1.4427 * d ** 0.5), 600, device="cuda").to(BF16)[None, :, None, None]
    t["v"][at] = t["v"][at].sign() * 2.0 ** 73
    check(t, call(t, max_new=n), only=(0, 1, 77, len(L) // 2, len(L) - 1))
