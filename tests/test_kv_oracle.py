"""Pins of the serving-cache oracle (CPU) and the refusals of the entry points
(argument checks before any launch)."""

import ctypes as C

import numpy as np
import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from oracle import diffattn_oracle as orc
from oracle import kv_oracle as kvo

FAKE = 1 << 20  # never dereferenced: validation fails or stops first


def test_bf16_rounding_matches_torch():
    x = np.random.default_rng(0).standard_normal(4096) * 10.0 ** (np.arange(4096) % 60 - 30)
    x[:4] = [0.0, np.inf, -np.inf, 3.4e38]
    t = torch.from_numpy(x).float().to(torch.bfloat16).double().numpy()
    assert np.array_equal(kvo.round_bf16(x), t)


@pytest.mark.parametrize("d", [64, 128])
def test_quantised_values_are_within_half_a_step(d):
    """|x - value| <= s / 2 inside the codes' range, plus what the top code is
    short of the maximum when s was rounded down (15 s >= range (1 - 2^-8))."""
    x = kvo.round_bf16(np.random.default_rng(d).standard_normal((50, d)) * 3)
    n, s, m = kvo.kv4_quantise(x)
    v = kvo.kv4_values(kvo.kv4_pack(x, -x))
    for got, ref in zip(v, (x, -x)):
        step = np.repeat(kvo.kv4_quantise(ref)[1], d // 2, -1)
        assert np.all(np.abs(got - ref) <= step * (0.5 + 15 * 2.0 ** -8))
    assert n.max() == 15 and n.min() == 0
    assert np.array_equal(kvo.round_bf16(s), s) and np.array_equal(kvo.round_bf16(m), m)


def test_quantise_special_groups():
    x = np.zeros((4, 64))
    x[0, :] = 1.5                   # constant: s = 0, the value itself
    x[1, 3], x[1, 40] = np.nan, 2.0  # NaN in the first group only
    x[2, 33] = -np.inf
    x[3, 0], x[3, 1] = 3.3e38, -3.3e38  # range overflows fp32
    n, s, m = kvo.kv4_quantise(x)
    assert np.all(n[0] == 0) and np.all(s[0] == 0) and np.all(m[0] == 1.5)
    for row, group in ((1, 0), (2, 1), (3, 0)):
        assert np.isnan(s[row, group]) and np.isnan(m[row, group])
        assert np.isfinite(s[row, 1 - group])
    v, _ = kvo.kv4_values(kvo.kv4_pack(x, x))
    assert np.all(v[0] == 1.5) and np.all(np.isnan(v[1, :32]))
    assert v[1, 40] == 15 * kvo.round_bf16(2 / 15)  # the top code, with s rounded to bf16


def test_differences_are_rounded_to_fp32():
    """Over a minimum of -2^-30 and with s = 1, x - m of 0.5, 1.5, .. 14.5 is that
    number in fp32: a tie, which goes to the even code."""
    x = np.zeros((2, 64))
    x[:, :15] = np.arange(15) + 0.5
    x[:, 15], x[:, 16] = 15.0, [-2.0 ** -30, -2.0 ** -18]  # 15 + 2^-18 is an fp32 number, the scale's bf16 still 1
    n, s, _ = kvo.kv4_quantise(x)
    assert np.all(s[:, 0] == 1)
    assert n[0, :15].tolist() == [0, 2, 2, 4, 4, 6, 6, 8, 8, 10, 10, 12, 12, 14, 14]
    assert n[1, :15].tolist() == list(range(1, 16))  # 2^-18 shows in all of these differences


def test_key_weights_of_equal_maps_vanish_and_of_plain_attention_sum_to_one():
    """gate 1 with equal queries gathers nothing; gate 0 is plain attention,
    whose weights sum to one per pair."""
    r = np.random.default_rng(3)
    q, k = r.standard_normal((4, 64)), r.standard_normal((9, 2, 64))
    w, _ = kvo.key_weights(q, k, np.zeros(2))
    assert np.allclose(w.sum(1), 1.0)
    q[1::2] = q[0::2]
    w, _ = kvo.key_weights(q, k, np.ones(2))
    assert np.all(w == 0)


def test_key_weights_bound_the_output():
    """The decode's output is the signed sum that the weights are the absolute
    one of: with V = 1 it is sum_j (A_2p - g A_2p+1) = 1 - g."""
    r = np.random.default_rng(4)
    q, k, g = r.standard_normal((2, 64)), r.standard_normal((7, 1, 64)), r.random(1)
    out = orc.v2_decode(q[None], k[None], np.ones((1, 7, 1, 64)), [7], g[None])["out"]
    w, total = kvo.key_weights(q, k, g)
    assert np.allclose(out, 1 - g[0])
    assert abs(1 - g[0]) <= w.sum() <= total.sum() + 1e-12


def test_evict_small_cases():
    w = [5, 1, 1, 9, 0, 7, 2, 3]
    assert kvo.evict(w, 8) == (8, list(range(8)))
    assert kvo.evict(w, 20) == (8, list(range(8)))
    # 5, 9, 7, 3 stay: slot 0 and 3 in place, 5 and 7 move into 1 and 2
    assert kvo.evict(w, 4) == (4, [0, 5, 7, 3])
    # sinks 2 (slots 0, 1), newest 1 (slot 7) and the best of the rest
    assert kvo.evict(w, 4, sinks=2, recent=1) == (4, [0, 1, 7, 3])
    # ties to the lowest slot; NaN above every number
    assert kvo.evict([1, 1, 1, 1], 2) == (2, [0, 1])
    assert kvo.evict([1, 2, float("nan"), 3], 2) == (2, [2, 3])
    # positions decide what is protected, not slots
    assert kvo.evict([1, 2, 3], 1, recent=1, positions=[9, 4, 5], next_position=10) == (1, [0])


# ------------------------------------------------------------- refusals ------
def _with(p, **kw):
    q = type(p).from_buffer_copy(p)
    for k, v in kw.items():
        setattr(q, k, v)
    return C.byref(q)


def test_null_params_rejected(lib):
    for name in ("diffattn_kv4_append", "diffattn_kv4_read", "diffattn_v2_decode_kv4",
                 "diffattn_v2_decode_weighted", "diffattn_kv_evict"):
        assert getattr(lib, name)(None, None) == bd.DA_ERR_INVALID_ARG, name


def test_record_bytes(lib):
    assert [bd.diffattn_kv4_record_bytes(d) for d in (64, 128, 96, 0, -1)] == [80, 144, 0, 0, 0]


def test_append_and_read_argument_checks(lib):
    row, rec = bd.da_t4(FAKE, 8 * 4 * 128, 4 * 128, 128), bd.da_t4(FAKE, 64 * 4 * 144, 4 * 144, 144)
    ap = bd.da_kv4_append_params(2, 8, 4, 128, 64, row, row, rec, FAKE, FAKE)
    rd = bd.da_kv4_read_params(2, 8, 4, 128, 64, rec, FAKE, FAKE, row, row)
    for f, p, names in ((lib.diffattn_kv4_append, ap, ("k", "v")), (lib.diffattn_kv4_read, rd, ("k_out", "v_out"))):
        for bad in (dict(B=-1), dict(N=-1), dict(h_kv=0), dict(L_max=0), dict(d=0), dict(start=FAKE + 2),
                    dict(counts=FAKE + 1), dict(cache=bd.da_t4(None, 0, 0, 0)),
                    dict(cache=bd.da_t4(FAKE + 8, 144, 144, 144)), dict(cache=bd.da_t4(FAKE, 144, 72, 144)),
                    dict(cache=bd.da_t4(FAKE, 144, -144, 144))):
            assert f(_with(p, **bad), None) == bd.DA_ERR_INVALID_ARG, bad
        for n in names:
            assert f(_with(p, **{n: bd.da_t4(None, 0, 0, 0)}), None) == bd.DA_ERR_INVALID_ARG
            assert f(_with(p, **{n: bd.da_t4(FAKE, 64, 60, 64)}), None) == bd.DA_ERR_INVALID_ARG
            assert f(_with(p, **{n: bd.da_t4(FAKE + 2, 64, 64, 64)}), None) == bd.DA_ERR_INVALID_ARG
        assert f(_with(p, d=96), None) == bd.DA_ERR_UNSUPPORTED
        assert f(_with(p, N=1 << 28), None) == bd.DA_ERR_UNSUPPORTED  # more rows than 32 bits count
        assert f(_with(p, B=0), None) == bd.DA_OK
        assert f(_with(p, N=0), None) == bd.DA_OK
    for n in ("key_weights", "positions", "first_position"):
        assert lib.diffattn_kv4_append(_with(ap, **{n: FAKE + 2}), None) == bd.DA_ERR_INVALID_ARG


def test_decode_kv4_argument_checks(lib):
    rec = bd.da_t4(FAKE, 1024 * 8 * 144, 144, 1024 * 144)
    p = bd.da_v2_decode_kv4_params(B=2, h=32, h_kv=8, d=128, L_max=1024, q=FAKE, cache=rec, gate=FAKE, out=FAKE)
    f = lib.diffattn_v2_decode_kv4
    for bad in (dict(B=0), dict(L_max=0), dict(h_kv=3), dict(h=4), dict(q=None), dict(q=FAKE + 2), dict(out=None),
                dict(gate=None), dict(gate=FAKE + 2), dict(seqlens=FAKE + 2),
                dict(cache=bd.da_t4(FAKE + 8, 144, 144, 144)), dict(cache=bd.da_t4(FAKE, 144, 72, 144)),
                dict(weights_out=FAKE + 2), dict(weights_in=FAKE),  # gathered weights need somewhere to go
                dict(weights_in=FAKE + 2, weights_out=FAKE),
                dict(gate=None, x=FAKE + 2, w_lambda=FAKE, d_model=64)):
        assert f(_with(p, **bad), None) == bd.DA_ERR_INVALID_ARG, bad
    for bad in (dict(d=96), dict(h=128), dict(gate=None, x=FAKE, w_lambda=FAKE, d_model=100), dict(B=65536),
                dict(L_max=(1 << 30) + 1)):
        assert f(_with(p, **bad), None) == bd.DA_ERR_UNSUPPORTED, bad
    size = lib.diffattn_v2_decode_kv4_workspace_size
    p.L_max = 16384
    need = size(2, 32, 8, 128, 16384, 1, 0)
    assert f(_with(p), None) == bd.DA_ERR_WORKSPACE
    assert f(_with(p, workspace=FAKE, workspace_bytes=need - 1), None) == bd.DA_ERR_WORKSPACE
    assert f(_with(p, workspace=FAKE + 128, workspace_bytes=need), None) == bd.DA_ERR_WORKSPACE
    # gathering needs room for a score per query head and key
    assert size(2, 32, 8, 128, 16384, 1, 1) - need >= 2 * 64 * 16384 * 4
    assert f(_with(p, weights_out=FAKE, workspace=FAKE, workspace_bytes=need), None) == bd.DA_ERR_WORKSPACE
    # few short heads need room for the scores and the gate only
    assert size(2, 32, 8, 128, 1024, 1, 0) == 0
    assert size(2, 32, 8, 128, 1024, 0, 0) == 2 * 32 * 4 and size(2, 32, 8, 128, 1024, 1, 1) == 2 * 64 * 1024 * 4
    p.L_max = 1024
    assert f(_with(p, weights_out=FAKE), None) == bd.DA_ERR_WORKSPACE
    assert f(_with(p, gate=None, x=FAKE, w_lambda=FAKE, d_model=64), None) == bd.DA_ERR_WORKSPACE
    assert lib.diffattn_v2_decode_kv4_workspace_size(0, 32, 8, 128, 1024, 1, 0) == 0


def test_decode_weighted_argument_checks(lib):
    cache = bd.da_t4(FAKE, 1024 * 8 * 128, 8 * 128, 128)
    dec = bd.da_v2_decode_params(B=2, h=32, h_kv=8, d=128, L_max=1024, q=FAKE, k_cache=cache, v_cache=cache,
                                 gate=FAKE, out=FAKE)
    p = bd.da_v2_decode_weighted_params(dec, None, FAKE)
    f = lib.diffattn_v2_decode_weighted
    assert f(_with(p, weights_out=None), None) == bd.DA_ERR_INVALID_ARG
    assert f(_with(p, weights_out=FAKE + 2), None) == bd.DA_ERR_INVALID_ARG
    assert f(_with(p, weights_in=FAKE + 2), None) == bd.DA_ERR_INVALID_ARG
    p.decode.h_kv = 3
    assert f(_with(p), None) == bd.DA_ERR_INVALID_ARG
    p.decode.h_kv, p.decode.d = 8, 96
    assert f(_with(p), None) == bd.DA_ERR_UNSUPPORTED
    p.decode.d, p.decode.num_splits = 128, 70000
    assert f(_with(p), None) == bd.DA_ERR_INVALID_ARG
    p.decode.num_splits, p.decode.L_max = 4, (1 << 30) + 1
    assert f(_with(p), None) == bd.DA_ERR_UNSUPPORTED
    p.decode.L_max = 1024
    plain = lib.diffattn_v2_decode_workspace_size(2, 32, 8, 128, 1024, 4, 1)
    need = lib.diffattn_v2_decode_weighted_workspace_size(2, 32, 8, 128, 1024, 4, 1)
    assert need - plain >= 2 * 64 * 1024 * 4
    p.decode.workspace, p.decode.workspace_bytes = FAKE, plain
    assert f(_with(p), None) == bd.DA_ERR_WORKSPACE


def test_evict_argument_checks(lib):
    p = bd.da_kv_evict_params(B=2, h_kv=4, L_max=64, keep=32, sinks=4, recent=8, seqlens=FAKE, seqlens_out=FAKE,
                              weights_in=FAKE, weights_out=FAKE, n_rows=2)
    for i in range(2):
        p.rows[i] = bd.da_t4(FAKE, 64 * 4 * 256, 4 * 256, 256)
        p.row_bytes[i] = 256
    f = lib.diffattn_kv_evict
    for bad in (dict(B=-1), dict(h_kv=0), dict(L_max=0), dict(keep=0), dict(sinks=-1), dict(recent=-1),
                dict(sinks=25), dict(recent=0x7fffffff), dict(n_rows=0), dict(n_rows=4), dict(n_rows=3),
                dict(weights_in=None), dict(weights_out=None), dict(seqlens_out=None), dict(positions_in=FAKE),
                dict(weights_in=FAKE + 2), dict(positions_out=FAKE + 2), dict(next_position=FAKE + 1),
                dict(seqlens=FAKE + 2)):
        assert f(_with(p, **bad), None) == bd.DA_ERR_INVALID_ARG, bad
    for field, value in (("rows", bd.da_t4(FAKE + 8, 256, 256, 256)), ("rows", bd.da_t4(FAKE, 256, 8, 256)),
                         ("row_bytes", 0), ("row_bytes", 24)):
        q = type(p).from_buffer_copy(p)
        getattr(q, field)[1] = value
        assert f(C.byref(q), None) == bd.DA_ERR_INVALID_ARG, (field, value)
    assert f(_with(p), None) == bd.DA_ERR_WORKSPACE
    need = lib.diffattn_kv_evict_workspace_size(2, 4, 64, 32)
    assert need >= 2 * 4 * 32 * 2 * 4
    assert f(_with(p, workspace=FAKE, workspace_bytes=need - 1), None) == bd.DA_ERR_WORKSPACE
    assert f(_with(p, B=0), None) == bd.DA_OK
    for bad in (dict(L_max=(1 << 20) + 1), dict(B=1 << 28)):  # more slots, or more heads, than are counted
        assert f(_with(p, **bad), None) == bd.DA_ERR_UNSUPPORTED, bad
    # keeping everything needs no lists
    assert lib.diffattn_kv_evict_workspace_size(2, 4, 64, 64) < need


def test_binding_refuses_wrong_tensors():
    """The binding checks types, shapes and contiguity before the library sees
    a pointer (CPU tensors are refused for not being on a GPU)."""
    k = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16)
    cache = torch.zeros((1, 4, 1, 80), dtype=torch.uint8)
    with pytest.raises(ValueError):
        bd.diffattn_kv4_append(k, k, cache)
    with pytest.raises(ValueError):
        bd.diffattn_kv4_read(cache, 2, k_out=k, v_out=k)
    with pytest.raises(ValueError):
        bd.diffattn_v2_decode_kv4(torch.zeros((1, 2, 64), dtype=torch.bfloat16), cache, gate=torch.zeros((1, 1)))
    with pytest.raises(ValueError):
        bd.diffattn_kv_evict([], torch.zeros((1, 1, 4)), 2)
