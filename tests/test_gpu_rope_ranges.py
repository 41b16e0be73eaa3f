"""Norm and rotation of queries and keys at the ends of their ranges:
frequencies of any size, or none, and infinities.

Bar of a rotated feature (u = 2^-24): a frequency in turns is off by 2^-63, times
a position of up to 2^31; a turn's rest is cut to 2^-34 turns, which is 2^-31
radians, and rounded to fp32 and by two factors (3 u of at most pi / 4); the
series up to x^9 and x^10 are off by 2^-29 and 2^-33, their last steps by 2 u, the
scale by u.  Together below 8 u of the pair's size; with the two products and the
sum 2^-19 scale (|z_u| + |z_v|), and half a step of the output's type."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from oracle import paged_oracle as po

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
LARGE = float(np.nextafter(np.float32(2.0 ** 32), np.float32(0)))  # the largest frequency below 2^32
GOOD = [1.0, -0.3, 12345.678, 1e-30, 0.0, 1e-42, 1e6, -1e9, LARGE, -LARGE, 3.3333e7]
BAD = [float("nan"), float("inf"), -float("inf"), 2.0 ** 32, -3e38]


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert bd.diffattn_get_device_status() == bd.DA_OK


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def two_pi():
    """2 pi to 200 bits: Machin's 16 arctan(1/5) - 4 arctan(1/239)."""
    def arctan(x):
        s, term, k = 0, (1 << 220) // x, 0
        while term:
            s += (-1) ** k * (term // (2 * k + 1))
            term //= x * x
            k += 1
        return s
    return Fraction(2 * (16 * arctan(5) - 4 * arctan(239)), 1 << 220)


def exact_angles(positions, f):
    """position * frequency in radians, reduced to a turn before anything is rounded."""
    turn = two_pi()
    a = [[float((int(p) * Fraction(float(x)) / turn) % 1 * turn) if np.isfinite(x) else np.nan for x in f] for p in positions]
    return np.array(a)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_frequencies(dtype, interleaved):
    """Frequencies below 2^32 turn by what they say at any position; without a finite one, or above, there are no
    angles, and the pair is NaN."""
    f = np.array(GOOD + BAD, np.float32)
    rot, N = 2 * len(f), 5
    g = gen(1)
    x, dy = (torch.randn((1, N, 3, 64), generator=g, device="cuda").to(dtype) for _ in range(2))
    pos = [0, 1, -7, 2 ** 31 - 1, -2 ** 31]
    p = torch.tensor([pos], dtype=torch.int32, device="cuda")
    ft = torch.tensor(f, device="cuda")
    kw = dict(positions=p, rot_dim=rot, interleaved=interleaved, rope_scale=1.25)
    y, _ = bd.diffattn_qk_rope_fwd(x, None, ft, **kw)
    dx = bd.diffattn_qk_rope_bwd(None, None, dy, None, ft, **kw)["dq"]
    ang = exact_angles(pos, f)
    bad = np.arange(len(f)) >= len(GOOD)
    ang[:, bad] = np.nan
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    for got, a, sign in ((y, x, 1), (dx, dy, -1)):
        a, got = (t.double().cpu().numpy()[0] for t in (a, got))
        ref = po.rotate(a, sign * ang, rot, interleaved, 1.25)
        size = np.zeros_like(a)
        size[..., u] = size[..., v] = np.abs(a[..., u]) + np.abs(a[..., v])
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        ok = ~np.isnan(ref)
        bar = 2.0 ** -19 * 1.25 * size + HALF[dtype] * np.abs(ref) * 1.001 + 1e-38
        assert np.all(np.abs(got - ref)[ok] <= bar[ok]), (np.abs(got - ref) / bar)[ok].max()


def test_frequencies_of_an_append():
    g = gen(2)
    k = torch.randn((2, 1, 64), generator=g, device="cuda").to(BF16)
    kp, vp = (torch.zeros((1, 16, 1, 64), dtype=BF16, device="cuda") for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    f = torch.tensor([0.5, float("nan"), 0.25, float("inf")], device="cuda")
    bd.diffattn_paged_append(k, k, kp, vp, i32([[0]]), i32([0, 2]), i32([2]), f)
    nan = torch.isnan(kp[0, :2, 0])
    assert nan[:, [1, 3, 5, 7]].all() and int(nan.sum()) == 8 and torch.equal(vp[0, :2], k)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (128, 8), (128, 64), (16, 8), (64, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_infinity_under_the_norm(interleaved, d, rot, dtype):
    """x / inf: the infinity itself is NaN, and so is its pair's other feature where it is rotated; the rest is 0."""
    x = torch.ones((1, d, 1, d), dtype=dtype, device="cuda")
    x[0, range(d), 0, range(d)] = torch.where(torch.arange(d, device="cuda") % 3 == 0, -torch.inf, torch.inf).to(dtype)
    f = torch.tensor(10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1)), dtype=F32, device="cuda")
    y = bd.diffattn_qk_rope_fwd(x, None, f, norm=True, interleaved=interleaved, rot_dim=rot)[0]
    with np.errstate(all="ignore"):
        ref = po.qk_rope(x.double().cpu().numpy(), f.cpu().numpy(), np.arange(d)[None], rot, interleaved, do_norm=True)
    got = y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.isnan(ref).sum() == d + rot
    assert not got[~np.isnan(ref)].any()
