"""Pins of the 64-bit definitions of the rotation, the norm and the paged
attention: closed forms, invariants, brute force, central differences; and of
the library's host function for frequencies."""

import ctypes as C
import math

import numpy as np
import pytest

from differential_attention_diff_gb300 import binding as bd
from oracle import paged_oracle as po

F = (10000.0 ** (-np.arange(4) / 4)).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_closed_forms(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 12))
    u, v = ([0, 2, 4, 6], [1, 3, 5, 7]) if interleaved else ([0, 1, 2, 3], [4, 5, 6, 7])
    # position 0 and no rotated features: the row itself
    assert np.array_equal(po.qk_rope(x, F, np.zeros(3, int), 8, interleaved), x)
    assert np.array_equal(po.qk_rope(x, F, np.arange(3), 0, interleaved), x)
    # as a product of complex numbers
    pos = np.array([1, 77, 100003])
    y = po.qk_rope(x, F, pos, 8, interleaved, scale=1.25)
    z = (x[..., u] + 1j * x[..., v]) * np.exp(1j * pos[:, None, None] * F.astype(np.float64)) * 1.25
    assert np.allclose(y[..., u], z.real, atol=1e-9) and np.allclose(y[..., v], z.imag, atol=1e-9)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    # products of rotated rows depend on the distance only
    a, b = (po.qk_rope(x[:1], F, [p], 8, interleaved)[0] for p in (5, 1005))
    c, d = (po.qk_rope(x[1:2], F, [p], 8, interleaved)[0] for p in (9, 1009))
    assert np.allclose((a * c).sum(-1), (b * d).sum(-1), atol=1e-9)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("do_norm", [False, True])
def test_backward_against_differences(interleaved, do_norm):
    rng = np.random.default_rng(2)
    x, dy, w = rng.standard_normal((2, 3, 10)), rng.standard_normal((2, 3, 10)), 1 + rng.standard_normal(10) / 5
    kw = dict(rot=8, interleaved=interleaved, scale=1.3, do_norm=do_norm, eps=1e-3)
    pos = np.array([3, 500])
    dx, dw = po.qk_rope_bwd(x, dy, F, pos, w=w, **kw)
    h = 1e-6

    def loss(x, w):
        return (po.qk_rope(x, F, pos, w=w, **kw) * dy).sum()
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    if do_norm:
        for i in range(10):
            e = np.zeros(10)
            e[i] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7
    else:
        assert dw is None


def test_attention_brute_force():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 4, 5)), rng.standard_normal((6, 2, 5)), rng.standard_normal((6, 2, 5))
    gate, seen = rng.random((3, 2)), [4, 5, 6]
    out, size = po.attend(q, k, v, gate, seen, sizes=True)
    for i in range(3):
        for p in range(2):
            o, s = [], []
            for j in (2 * p, 2 * p + 1):
                e = [math.exp(sum(q[i, j, f] * k[m, p, f] for f in range(5)) / math.sqrt(5)) for m in range(seen[i])]
                o.append(sum(e[m] * v[m, p] for m in range(seen[i])) / sum(e))
                s.append(sum(e[m] * abs(v[m, p]) for m in range(seen[i])) / sum(e))
            assert np.allclose(out[i, p], o[0] - gate[i, p] * o[1], atol=1e-12)
            assert np.allclose(size[i, p], s[0] + gate[i, p] * s[1], atol=1e-12)


def test_gather():
    pages = np.arange(4 * 3 * 1 * 2, dtype=float).reshape(4, 3, 1, 2)
    got = po.gather(pages, [2, 9, 0], 8)
    assert np.array_equal(got[:3], pages[2]) and not got[3:6].any() and np.array_equal(got[6:], pages[0, :2])


def test_frequencies():
    """Closed forms of the library's host function: half an fp32 step of the fp64 value, and a little for pow's own
    last bit."""
    def got(*a, **kw):
        f, s = bd.diffattn_rope_inv_freq(*a, device="cpu", **kw)
        return f.numpy().astype(np.float64), s
    plain = 10000.0 ** (-np.arange(32) / 32)
    near = 2.0 ** -24 * 1.001
    for kw, exp, scale in ((dict(), plain, 1.0), (dict(stretch="linear", factor=4.0), plain / 4, 1.0),
                           (dict(stretch="base", factor=4.0), (10000.0 * 4 ** (64 / 62)) ** (-np.arange(32) / 32), 1.0)):
        f, s = got(64, **kw)
        assert np.all(np.abs(f - exp) <= near * exp) and s == scale
    f, s = got(64, stretch="base", factor=4.0)
    assert f[0] == 1 and abs(f[-1] * 4 / plain[-1] - 1) < 1e-6
    f, s = got(64, stretch="ramp", factor=16.0, trained_len=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert np.all(np.abs(f - plain)[turns >= 32] <= near * plain[turns >= 32])
    assert np.all(np.abs(f - plain / 16)[turns <= 1] <= near * plain[turns <= 1] / 16)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all((f < plain)[mid]) and np.all((f > plain / 16)[mid])
    assert abs(s - (0.1 * math.log(16) + 1)) < 1e-6
    assert np.array_equal(got(64, stretch="ramp", factor=1.0, trained_len=4096)[0], got(64)[0])


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=12), dict(base=1.0), dict(base=float("nan")), dict(stretch=4),
                                dict(stretch=1, factor=0.5), dict(stretch=3, factor=2.0, trained=0),
                                dict(stretch=2, factor=float("inf"))])
def test_frequencies_refused(lib, kw):
    f, s = (C.c_float * 64)(), C.c_float()
    a = dict(rot_dim=64, base=10000.0, stretch=0, factor=1.0, trained=4096) | kw
    assert lib.diffattn_rope_inv_freq(a["rot_dim"], a["base"], a["stretch"], a["factor"], a["trained"], f,
                                      C.byref(s)) == bd.DA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        bd.diffattn_rope_inv_freq(64, stretch="no such")
