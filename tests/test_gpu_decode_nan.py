"""A NaN in a key or value row inside the sequence of a bf16 cache: the V2
decodes give NaN where the definition does, and nowhere else."""

import pytest
import torch

from differential_attention_diff_gb300 import binding as bd

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("where", ["key", "value"])
@pytest.mark.parametrize("d,L,at", [(64, 1, 0), (64, 700, 699), (128, 100, 40), (128, 3000, 17)])
def test_a_nan_row_reaches_its_kv_head_and_no_other(d, L, at, where):
    """A NaN key makes every weight of its KV head's maps NaN, and so its
    outputs; a NaN value feature reaches that feature of the outputs only, and
    no weight."""
    h, hkv = 4, 2
    g = torch.Generator(device="cuda").manual_seed(31 + d + L)
    k, v = (torch.randn((1, L, hkv, d), generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn((1, 2 * h, d), generator=g, device="cuda").to(BF16)
    gate = torch.rand((1, h), generator=g, device="cuda")
    (k if where == "key" else v)[0, at, 0, 5] = float("nan")
    w = torch.full((1, hkv, L), -2.0, device="cuda")
    weighted = bd.diffattn_v2_decode_weighted(q, k, v, gate=gate, weights_out=w)
    for out in (weighted, bd.diffattn_v2_decode(q, k, v, gate=gate), bd.diffattn_v2_decode_noalloc(q, k, v, gate=gate)):
        nan = torch.isnan(out[0])
        if where == "key":
            assert bool(nan[:2].all())
        else:
            assert bool(nan[:2, 5].all()) and int(nan[:2].sum()) == 2
        assert bool(torch.isfinite(out[0, 2:]).all())
    assert bool(torch.isnan(w[0, 0]).all() if where == "key" else torch.isfinite(w[0, 0]).all())
    assert bool(torch.isfinite(w[0, 1]).all())
    assert bd.diffattn_get_device_status() == bd.DA_OK
