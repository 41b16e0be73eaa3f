"""The V2 decode over a 4-bit cache at the ends of its numbers' ranges, on the
path of a block per head (L 700), of a cluster per head (2200) and of the line
of chunks (8320).

Bars, per half of a value row (u = 2^-24, half an fp32 step; s and m the half's
scale and minimum):
- scores are off by e = 64 u (1 + scale sum_f |q_f| (15 |s| + |m|)) at most, as
  a factor of the weights;
- p s goes to the value product in fp16, 2^-11 relative at most, on codes up to
  15: 2^-11 of the half's largest 15 s.  What falls below fp16's normal numbers
  is off by 2^-25 a key, where the half's largest p s is 2^4 or more: less than
  L 2^-29 of 15 s;
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


@pytest.mark.parametrize("ratio", [2.0 ** 3, 2.0 ** 6, 2.0 ** 30])
@pytest.mark.parametrize("d,G", [(64, 12), (128, 4)])
@pytest.mark.parametrize("L", PATHS)
def test_value_halves_of_different_size_beside_weights(L, d, G, ratio):
    """The same where the keys' weights are gathered, for halves that may share
    a factor and halves that may not; the weights do not depend on the values."""
    g = torch.Generator(device="cuda").manual_seed(920 + L + d)
    k, v = randn((2, L, 1, d), g), randn((2, L, 1, d), g)
    v[1:, ..., :d // 2] *= ratio
    v[:1, ..., d // 2:] *= ratio
    q, gate = randn((2, G, d), g).to(BF16), torch.rand((2, G // 2), generator=g, device="cuda")
    cache, other = cache_of(k, v), cache_of(k, v.flip(0).contiguous())
    w, w2 = torch.zeros((2, 1, L), device="cuda"), torch.zeros((2, 1, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w)
    check_halves(q, cache, gate, out)
    check_halves(q, other, gate, bd.diffattn_v2_decode_kv4(q, other, gate=gate, weights_out=w2))
    rec = cache.cpu().numpy()
    kf, mag = kvo.kv4_values(rec)[0], parameters(rec)[1][..., 0, :].max()
    for b in range(2):
        ref, total = kvo.key_weights(f64(q[b]), kf[b], f64(gate[b]))
        e = 64 * U * (2 + d ** -0.5 * np.abs(f64(q[b])).sum(-1).max() * mag)
        for got in (w, w2):
            assert np.all(np.abs(f64(got[b]) - ref) <= e * total + 4 * U * ref + 1e-37)


# ------------------------------------------------------ the scores' range ---
@pytest.mark.parametrize("heads", ["all", "even"])
@pytest.mark.parametrize("q_size,k_size", [(2.0 ** 119, 2.0 ** -118), (2.0 ** 126, 2.0 ** -126), (2.0 ** -119, 2.0 ** 118),
                                           (2.0 ** -126, 2.0 ** 122)])
@pytest.mark.parametrize("d,G", [(64, 12), (128, 4)])
@pytest.mark.parametrize("L", (33,) + PATHS)
def test_scores_of_huge_and_tiny_queries(L, d, G, q_size, k_size, heads):
    """Queries and keys at the ends of bf16's range whose products are ordinary
    numbers, beside heads (the odd ones, of "even") of ordinary queries."""
    g = torch.Generator(device="cuda").manual_seed(930 + L + d)
    k, v = (torch.rand((2, L, 1, d), generator=g, device="cuda") * 2 - 1 for _ in range(2))
    q = torch.rand((2, G, d), generator=g, device="cuda") * 2 - 1
    if heads == "all":
        q *= q_size
    else:
        q[:, 0::2] *= q_size
        if k_size > 1:
            q[:, 1::2] /= k_size
    q, gate = q.to(BF16), torch.rand((2, G // 2), generator=g, device="cuda")
    cache = cache_of(k * k_size, v)
    w = torch.zeros((2, 1, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w)
    check_halves(q, cache, gate, out)
    assert bool(torch.isfinite(w).all())


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("L", (1, 33) + PATHS)
def test_equal_scores_at_the_end_of_the_range(L, sign):
    """Equal keys whose scores are 0.95 of the least or largest number: every
    weight is 1 / L, as of any equal scores."""
    d, h = 64, 2
    g = torch.Generator(device="cuda").manual_seed(950 + L)
    k, v = torch.full((1, L, 1, d), sign * 2.0 ** 61, device="cuda"), randn((1, L, 1, d), g)
    q = torch.full((1, 2 * h, d), 2.0 ** 60, device="cuda").to(BF16)  # q . k = 2^127
    scale = 0.95 * 2 / 1.4426950408889634  # 0.95 * 2^128 in log2 units
    gate = torch.rand((1, h), generator=g, device="cuda")
    cache = cache_of(k, v)
    w = torch.zeros((1, 1, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w, softmax_scale=scale)
    check_halves(torch.zeros_like(q), cache, gate, out)  # queries of the same weights
    want = float((1 - gate.double()).sum()) / L
    # products rounded before they are subtracted: 64 u of (1 + gate) / L per pair
    assert float((w.double() - want).abs().max()) <= 64 * U * float((1 + gate.double()).sum()) / L


@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 15, 2.0 ** 30])
@pytest.mark.parametrize("d,G", [(64, 12), (128, 4)])
@pytest.mark.parametrize("L", (33,) + PATHS)
def test_scores_far_apart(L, d, G, size):
    """Scores of 2^20 to 2^67: the largest key, ahead of the others by more
    than the scores' error, has all the weight, wherever it stands."""
    g = torch.Generator(device="cuda").manual_seed(960 + L + d)
    signs = torch.where(torch.rand((2, 1, 1, d), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    height = 0.5 + 0.4 * torch.rand((2, L, 1, 1), generator=g, device="cuda")
    best = [L // 3, L - 1]
    height[0, best[0]] = height[1, best[1]] = 1.0
    k, v = size * height * signs, randn((2, L, 1, d), g)
    q = (size * signs[:, 0].expand(2, G, d)).to(BF16)
    gate = torch.rand((2, G // 2), generator=g, device="cuda")
    cache = cache_of(k, v)
    w = torch.zeros((2, 1, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w)
    check_halves(q, cache, gate, out, e=0.0)
    want = torch.zeros_like(w, dtype=torch.float64)
    for b in range(2):
        want[b, 0, best[b]] = (1 - gate[b].double()).sum()
    assert float((w.double() - want).abs().max()) <= 64 * U * 2 * G


# ------------------------------------------------------ the values' range ---
@pytest.mark.parametrize("values", ["equal", "spread"])
@pytest.mark.parametrize("d,G", [(64, 2), (64, 12), (128, 4)])
@pytest.mark.parametrize("B,L", [(24, 1024), (24, 4096), (48, 8320)])
def test_values_near_the_end_of_the_range(B, L, d, G, values):
    """Two chunks or more go to a warp, and every second chunk of 32 keys holds
    one of a score above those before it (by 2^7, or by 2^5 where the values'
    scales bound it too), the others far less; the values are so large that a
    weight of 2^7 or 2^5 of one or two of them passes the largest number, while
    the sum of weights of at most 1 does not."""
    g = torch.Generator(device="cuda").manual_seed(970 + L + d)
    chunks = L // 32
    k = torch.zeros((B, L, 1, d), device="cuda")
    k[..., 0] = -40.0
    for c in range(chunks):
        k[:, 32 * c + (5 * c) % 32, 0, 0] = (7 if values == "equal" else 5) / 1.4426950408889634 if c % 2 else 0.0
    v = 0.6 + 0.4 * torch.rand((B, L, 1, d if values == "spread" else 1), generator=g, device="cuda")
    v = (3.2e38 / (chunks // 2) * v).expand(B, L, 1, d)
    q = torch.zeros((B, G, d), device="cuda")
    q[..., 0] = d ** 0.5
    q[:, 1::2, 0] *= 0.875
    q, gate = q.to(BF16), torch.rand((B, G // 2), generator=g, device="cuda")
    cache = cache_of(k, v)
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate)
    check_halves(q, cache, gate, out)


@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** -105, 2.0 ** -115, 2.0 ** -122])
@pytest.mark.parametrize("keys", ["flat", "rising"])
@pytest.mark.parametrize("L", PATHS)
def test_tiny_values(L, keys, size):
    """Values whose scales are far below 1, down to bf16's least normal numbers."""
    d, G = 128, 4
    g = torch.Generator(device="cuda").manual_seed(990 + L)
    k, v = randn((2, L, 1, d), g), randn((2, L, 1, d), g, size)
    if keys == "rising":
        k *= torch.linspace(0.05, 4.0, L, device="cuda")[None, :, None, None]
    q, gate = randn((2, G, d), g).to(BF16), torch.rand((2, G // 2), generator=g, device="cuda")
    cache = cache_of(k, v)
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate)
    check_halves(q, cache, gate, out)
