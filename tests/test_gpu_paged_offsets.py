"""V2 attention over a paged cache with offsets of sequences that are none: the
status word says so, and nothing but the rows of the output is written."""

import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from test_gpu_paged import BF16, call, check, i32, make

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


@pytest.mark.parametrize("max_new", [0, 1])
@pytest.mark.parametrize("cu,T", [([0, 7, 4, 6], 6), ([0, 5, 3, 9], 9), ([2, 5, 3, 9], 9), ([0, 4, 8, 3], 12), ([0, -1, 3, 9], 9)], ids=str)
def test_offsets_that_fall(cu, T, max_new):
    """Sequences whose rows might be another's too: all rows are zeros, call after call."""
    t = make([4, 4, 4], [200, 150, 90], 16, 4, 2, 128)
    t["q"], t["gate"] = t["q"][:T], t["gate"][:T].contiguous()
    t["cu"] = i32(cu)
    out = torch.empty((T, 4, 128), dtype=BF16, device="cuda")
    for _ in range(20):
        out.fill_(7.0)
        call(t, out=out, max_new=max_new)
        assert not out.any()
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS


@pytest.mark.parametrize("max_new", [0, 1])
def test_offsets_that_fall_among_many(max_new):
    """Behind more sequences than a block has threads, of which each is right."""
    n = [1] * 700
    t = make(n, [9] * 700, 16, 2, 1, 64)
    cu = t["cu"].clone()
    t["cu"][650] = 600
    assert not call(t, max_new=max_new).any()
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    t["cu"] = cu
    check(t, call(t, max_new=max_new))
    assert bd.diffattn_get_device_status() == bd.DA_OK


@pytest.mark.parametrize("n", [[1, 1, 1], [100, 70, 90]])
def test_sequence_before_the_array(n):
    """Rising offsets below 0: the sequences there are out of bounds, those behind them are not."""
    t = make(n, [200, 150, 300], 16, 4, 2, 128)
    t["cu"] = i32([-n[0] - n[1], -n[1], 0, n[2]])
    t["q"] = t["q"].roll(n[2], 0)
    t["gate"] = t["gate"].roll(n[2], 0)
    out = torch.full((sum(n), 4, 128), 7.0, dtype=BF16, device="cuda")
    call(t, out=out)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    check(dict(t, q=t["q"][:n[2]], gate=t["gate"][:n[2]], n=n[2:], L=[300], table=t["table"][2:]), out)
    assert bool((out[n[2]:] == 7).all())


@pytest.mark.parametrize("max_new", [0, 1])
def test_most_sequences_are_empty(max_new):
    """2^20 sequences of which the first, one in between and the last have tokens."""
    B = 2 ** 20
    t = make([2, 3, 1], [300, 150, 90], 16, 4, 2, 128)
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    sl, table = torch.zeros_like(n), torch.zeros((B, t["table"].shape[1]), dtype=torch.int32, device="cuda")
    for i, b in enumerate((0, 12345, B - 1)):
        n[b], sl[b], table[b] = t["n"][i], t["L"][i], t["table"][i]
    cu = torch.cat([n[:1] * 0, n.cumsum(0)]).int()
    out = call(dict(t, cu=cu, sl=sl, table=table), max_new=max_new)
    assert bd.diffattn_get_device_status() == bd.DA_OK
    check(t, out)
