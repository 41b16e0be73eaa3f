"""The V2 decode over a 4-bit cache at the ends of its numbers' ranges, on the
path of a block per head (L 700), of a cluster per head (2200) and of the line
of chunks (8320).

Bars, per half of a value row (u = 2^-24, half an fp32 step; s and m the half's
scale and minimum):
- scores are off by e = 64 u (1 + scale sum_f |q_f| (15 |s| + |m|)) at most, as
  a factor of the weights;
- p s goes to the value product in fp16, 2^-11 relative at most, on codes up to
  15: 2^-11 of the half's largest 15 s.  What falls below fp16's normal numbers
  is off by 2^-25 a key, where the half's largest p s is 2^8 or more: less than
  L 2^-33 of 15 s;
- fp32 steps on s n and m: 64 u (15 s + |m|);
- the output's bf16 rounding, 2^-8 relative."""

import numpy as np
import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from oracle import diffattn_oracle as orc
from oracle import kv_oracle as kvo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.bfloat16
PATHS = (700, 2200, 8320)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert bd.diffattn_get_device_status() == bd.DA_OK


def randn(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def parameters(rec):
    """15 |s| and 15 |s| + |m| of records [..., d + 16]: [..., key / value, half]."""
    d = rec.shape[-1] - 16
    bits = np.ascontiguousarray(rec[..., d:]).view("<u2").astype(np.uint32) << 16
    p = np.abs(bits.view(np.float32).astype(np.float64)).reshape(*rec.shape[:-1], 2, 2, 2)
    return 15 * p[..., 0, :], 15 * p[..., 0, :] + p[..., 1, :]


def check_halves(q, cache, gate, out, scale=None, e=None):
    """Every half row of the output [B, h, d] against the oracle over the
    records; e where the scores' error is known better."""
    rec, got, qf, gf = cache.cpu().numpy(), f64(out), f64(q), f64(gate)
    B, L, hkv, _ = rec.shape
    H2, d = q.shape[1:]
    G = H2 // hkv
    sc = 1.0 / np.sqrt(d) if scale is None else scale
    assert np.all(np.isfinite(got))
    kf, vf = kvo.kv4_values(rec)
    code, mag = parameters(rec)
    ref = orc.v2_decode(qf, kf, vf, [L] * B, gf, scale=sc)["out"]
    for b in range(B):
        for p in range(H2 // 2):
            g, gp = 2 * p // G, abs(gf[b, p])
            if e is None:
                off = 64 * U * (1 + sc * np.abs(qf[b, 2 * p:2 * p + 2]).sum(-1).max() * mag[b, :, g, 0].max())
            else:
                off = e
            for half in (0, 1):
                f = slice(half * d // 2, (half + 1) * d // 2)
                bar = 2.0 ** -8 * np.abs(ref[b, p, f]) + (1 + gp) * (
                    2.0 ** -11 * code[b, :, g, 1, half].max() + (off + 64 * U) * mag[b, :, g, 1, half].max())
                worst = float(np.max(np.abs(got[b, p, f] - ref[b, p, f]) / bar))
                assert worst <= 1.0, (b, p, half, worst)


def cache_of(k, v):
    B, L, hkv, d = k.shape
    cache = torch.zeros((B, hkv, L, d + 16), dtype=torch.uint8, device="cuda").transpose(1, 2)
    return bd.diffattn_kv4_append(k.to(BF16), v.to(BF16), cache)


# ------------------------------------------------ value halves that differ ---
@pytest.mark.parametrize("keys", ["flat", "rising"])
@pytest.mark.parametrize("large", [0, 1])
@pytest.mark.parametrize("ratio", [2.0 ** 30, 2.0 ** 40])
@pytest.mark.parametrize("d,G", [(64, 2), (64, 12), (128, 4), (128, 10)])
@pytest.mark.parametrize("L", PATHS)
def test_value_halves_of_different_size(L, d, G, ratio, large, keys):
    """One half of every value row is larger than the other by 2^30 or 2^40:
    both halves come out, each to its own precision."""
    g = torch.Generator(device="cuda").manual_seed(900 + L + d + G)
    k, v = randn((2, L, 1, d), g), randn((2, L, 1, d), g)
    if keys == "rising":
        k *= torch.linspace(0.05, 4.0, L, device="cuda")[None, :, None, None]
    v[..., large * (d // 2):(large + 1) * (d // 2)] *= ratio
    q, gate = randn((2, G, d), g).to(BF16), torch.rand((2, G // 2), generator=g, device="cuda")
    cache = cache_of(k, v)
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate)
    check_halves(q, cache, gate, out)
