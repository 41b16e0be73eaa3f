"""The 4-bit KV cache on the GPU: append and read back bit for bit against the
fp64 definition, and the V2 decode over it.

Bars, derived from the arithmetic (u = 2^-24, half an fp32 step):
- records are compared bit for bit (the definition fixes every rounding);
- values read back: one bf16 rounding, 2^-8 |v|, after fp32 steps on s n and m;
- decode: the scores carry fp32 accumulation over the features,
  e = 64 u (1 + scale sum_f |q_f| (15 |s| + |m|)) at most, which moves every
  weight A by A e; probabilities reach the value product in 16 bits with at
  least 11 bits of mantissa (2^-11 relative, on codes of range 15 s); the
  output is rounded to bf16 (2^-8 relative);
- gathered weights: e (A_2p + |g| A_2p+1) summed over pairs, and the fp32
  rounding of the sum."""

import numpy as np
import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from oracle import diffattn_oracle as orc
from oracle import kv_oracle as kvo
from ratio_log import record

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.bfloat16


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def new_cache(B, L, hkv, d, layout="head", fill=0xFF):
    """A cache whose records hold NaN parameters until they are written."""
    if layout == "head":
        return torch.full((B, hkv, L, d + 16), fill, dtype=torch.uint8, device="cuda").transpose(1, 2)
    if layout == "token":
        return torch.full((B, L, hkv, d + 16), fill, dtype=torch.uint8, device="cuda")
    # records 32 bytes further apart than they are long, base offset by one record
    big = torch.full((B, L + 1, hkv, d + 48), fill, dtype=torch.uint8, device="cuda")
    return big[:, 1:, :, 16:d + 32]


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert bd.diffattn_get_device_status() == bd.DA_OK


# ------------------------------------------------------- append and read ----
def test_append_special_values_bit_for_bit():
    """Constants, zeros of both signs, subnormals, outliers, huge ranges,
    infinities and NaN, in either group."""
    for d in (64, 128):
        x = torch.zeros((1, 12, 1, d))
        g = torch.Generator().manual_seed(d)
        x[0, 0] = 1.5
        x[0, 1, 0, ::2] = -0.0
        x[0, 2] = torch.randn((1, d), generator=g) * 1e-39
        x[0, 3] = torch.randn((1, d), generator=g)
        x[0, 3, 0, 5] = 300.0
        x[0, 4, 0, 0], x[0, 4, 0, 1] = 3e38, -3e38
        x[0, 5, 0, d - 1] = float("nan")
        x[0, 6, 0, 2] = float("inf")
        x[0, 7, 0, d // 2] = float("-inf")
        x[0, 8] = float("nan")
        x[0, 9] = float("inf")
        x[0, 10] = torch.arange(d).float() / 8 - 3  # quotients that fall on ties
        x[0, 11] = torch.randn((1, d), generator=g) * 1e30
        k, v = x.to(BF16).cuda(), x.flip(1).to(BF16).cuda()
        cache = new_cache(1, 12, 1, d)
        bd.diffattn_kv4_append(k, v, cache)
        ref = kvo.kv4_pack(f64(k), f64(v))
        assert np.array_equal(cache.cpu().numpy(), ref)
        kb, vb = bd.diffattn_kv4_read(cache, 12)
        for got, exp in zip((kb, vb), kvo.kv4_values(ref)):
            got = f64(got)
            assert np.array_equal(np.isnan(got), np.isnan(exp))
            ok = ~np.isnan(exp)
            assert np.all(np.abs(got - exp)[ok] <= 2.0 ** -8 * (1 + 2.0 ** -12) * np.abs(exp[ok]) + 2.0 ** -134)


@pytest.mark.parametrize("d", [64, 128])
def test_append_ties_of_rounded_differences(d):
    """Differences x - m that are ties of two codes in fp32 and not in more
    bits, in either group, at scales from 2^-115 to 2^120; a minimum of
    -2^-18 s beside one of -2^-30 s shows in the differences."""
    x = torch.zeros((1, 16, 1, d), dtype=torch.float64)
    for i, e in enumerate((0, 40, 100, 120, -40, -99, -101, -115)):
        for j, low in enumerate((2.0 ** -30, 2.0 ** -18)):
            for half in (0, 1):
                part = x[0, 2 * i + j, 0, half * d // 2:]
                part[:15] = torch.arange(15) + 0.5
                part[15], part[16 + half] = 15.0, -low
            x[0, 2 * i + j] *= 2.0 ** e
    x = x.to(BF16).cuda()
    cache = new_cache(1, 16, 1, d)
    bd.diffattn_kv4_append(x, x.flip(1), cache)
    assert np.array_equal(cache.cpu().numpy(), kvo.kv4_pack(f64(x), f64(x.flip(1))))


@pytest.mark.parametrize("layout", ["head", "token", "padded"])
@pytest.mark.parametrize("B,N,hkv,d,L,ragged", [(1, 1, 1, 64, 1, False), (3, 1, 8, 128, 40, False),
                                                 (2, 37, 3, 128, 64, True), (4, 130, 2, 64, 131, True),
                                                 (2, 300, 5, 64, 1000, True)])
def test_append_read_parity(B, N, hkv, d, L, ragged, layout):
    g = gen(100 + B + N + d)
    x = randn((B, N, 3 * hkv, d), g, 2.0)  # strided views of a packed projection
    k, v = x[:, :, hkv:2 * hkv], x[:, :, 2 * hkv:]
    counts = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if ragged else None
    n = [N] * B if counts is None else counts.tolist()
    start = torch.tensor([int(s) for s in np.random.default_rng(B + N).integers(0, L - N + 1, B)], dtype=torch.int32,
                         device="cuda")
    cache = new_cache(B, L, hkv, d, layout)
    before = cache.cpu().numpy().copy()
    w = torch.full((B, hkv, L), 7.0, device="cuda")
    pos = torch.full((B, hkv, L), -5, dtype=torch.int32, device="cuda")
    first = torch.arange(B, dtype=torch.int32, device="cuda") * 1000 + 11
    bd.diffattn_kv4_append(k, v, cache, start=start, counts=counts, key_weights=w, positions=pos,
                           first_position=first)
    k_out, v_out = (torch.full((B, N, hkv, d), 9.0, dtype=BF16, device="cuda") for _ in range(2))
    bd.diffattn_kv4_read(cache, N, start=start, counts=counts, k_out=k_out, v_out=v_out)
    exp_w, exp_p = np.full((B, hkv, L), 7.0), np.full((B, hkv, L), -5)
    exp_out = [np.full((B, N, hkv, d), 9.0) for _ in range(2)]
    for b in range(B):
        s, c = int(start[b]), n[b]
        before[b, s:s + c] = kvo.kv4_pack(f64(k[b, :c]), f64(v[b, :c]))
        exp_w[b, :, s:s + c] = 0
        exp_p[b, :, s:s + c] = 1000 * b + 11 + np.arange(c)
        for e, r in zip(exp_out, kvo.kv4_values(before[b, s:s + c])):
            e[b, :c] = r
    assert np.array_equal(cache.cpu().numpy(), before)  # records that no row goes to are as they were
    assert np.array_equal(w.cpu().numpy(), exp_w) and np.array_equal(pos.cpu().numpy(), exp_p)
    for got, exp in zip((k_out, v_out), exp_out):
        assert np.all(np.abs(f64(got) - exp) <= 2.0 ** -8 * (1 + 2.0 ** -12) * np.abs(exp) + 2.0 ** -20)


def test_append_bad_rows_are_recorded_and_not_written():
    B, N, hkv, d, L = 5, 4, 2, 64, 16
    k = randn((B, N, hkv, d), gen(1))
    cache = new_cache(B, L, hkv, d)
    start = torch.tensor([0, -1, 13, 0, 12], dtype=torch.int32, device="cuda")
    counts = torch.tensor([4, 2, 4, 5, 4], dtype=torch.int32, device="cuda")
    bd.diffattn_kv4_append(k, k, cache, start=start, counts=counts)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    got = cache.cpu().numpy()
    for b, written in ((0, True), (1, False), (2, False), (3, False), (4, True)):
        assert bool(np.any(got[b] != 0xFF)) == written, b
    out = bd.diffattn_kv4_read(cache, N, start=start, counts=counts)[0]
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    assert float(out[1:4].abs().max()) == 0.0 and float(out[0].abs().max()) > 0
    # no rows at all: nothing to do, nothing recorded
    bd.diffattn_kv4_append(k[:, :0], k[:, :0], cache)
    bd.diffattn_kv4_append(k[:0], k[:0], cache[:0])


# ---------------------------------------------------------------- decode ----
def check_decode(q, kf, vf, rng_k, rng_v, lens, gate, out, w=None, w_in=None, w_before=None, scale=None, heads=None,
                 p_bits=11):
    """Compare with the oracle: kf, vf [B, L, hkv, d] fp64 values; rng_k, rng_v:
    largest |s| * 15 + |m| and |s| * 15 per [B, L, hkv] (the arithmetic's magnitudes)."""
    B, H2, d = q.shape
    hkv = kf.shape[2]
    G = H2 // hkv
    sc = 1.0 / np.sqrt(d) if scale is None else scale
    qf, got = f64(q), f64(out)
    worst, worst_w = 0.0, 0.0
    for b in range(B):
        n = lens[b]
        kb, vb = kf[b, :n], vf[b, :n]
        ref = orc.v2_decode(qf[b:b + 1], kb[None], vb[None], [n], gate[b:b + 1], scale=sc)["out"][0]
        e = np.zeros(H2)
        for j in range(H2):
            e[j] = 64 * U * (1 + sc * np.abs(qf[b, j]).sum() * rng_k[b, :n, j // G].max())
        for p in range(H2 // 2):
            g, gp = 2 * p // G, abs(gate[b, p])
            v_max = np.abs(vb[:, g]).max()
            bar = 2.0 ** -8 * np.abs(ref[p]) + (1 + gp) * (2.0 ** -p_bits * rng_v[b, :n, g].max() +
                                                          (max(e[2 * p], e[2 * p + 1]) + 64 * U) * v_max)
            worst = max(worst, float(np.max(np.abs(got[b, p] - ref[p]) / bar)))
        if w is not None:
            dw, total = kvo.key_weights(qf[b], kb, gate[b], sc)
            base = np.zeros((hkv, n)) if w_in is None else f64(w_in[b, :, :n])
            em = e.reshape(hkv, G).max(1)[:, None] + 64 * U
            bar = em * total + 4 * U * np.abs(base + dw) + 1e-37
            worst_w = max(worst_w, float(np.max(np.abs(f64(w[b, :, :n]) - base - dw) / bar)))
            assert torch.equal(w[b, :, n:], w_before[b, :, n:])  # behind the sequence: as it was
    record({"out": worst, "weights": worst_w})
    assert worst <= 1.0 and worst_w <= 1.0, (worst, worst_w)


def ranges(rec):
    """kv4_values plus the magnitudes that check_decode takes."""
    kf, vf = kvo.kv4_values(rec)
    d = rec.shape[-1] - 16
    par = np.ascontiguousarray(rec[..., d:]).view("<u2").astype(np.uint32) << 16
    par = np.abs(par.view(np.float32).astype(np.float64)).reshape(*rec.shape[:-1], 2, 2, 2)  # row, s / m, group
    return kf, vf, (15 * par[..., 0, 0, :] + par[..., 0, 1, :]).max(-1), 15 * par[..., 1, 0, :].max(-1)


def make(B, L, h, hkv, d, lens, seed, layout="head", k_std=1.0, v_std=1.0):
    g = gen(seed)
    cache = new_cache(B, L, hkv, d, layout)
    for b in range(B):
        n = lens[b]
        rows = [randn((1, n, hkv, d), g, s) for s in (k_std, v_std)]
        bd.diffattn_kv4_append(*rows, cache[b:b + 1])
    q = randn((B, 2 * h, d), g)
    gate = torch.rand((B, h), generator=g, device="cuda")
    return g, cache, q, gate, torch.tensor(lens, dtype=torch.int32, device="cuda")


def clean(cache, lens):
    """The records as numpy, with those behind each sequence (NaN parameters) zeroed for the oracle."""
    rec = cache.cpu().numpy().copy()
    for b, n in enumerate(lens):
        rec[b, n:] = 0
    return rec


@pytest.mark.parametrize("layout", ["head", "token", "padded"])
@pytest.mark.parametrize("B,L,h,hkv,d,lens", [
    (1, 1, 1, 1, 128, [1]), (1, 1, 1, 1, 64, [1]), (3, 70, 4, 2, 128, [70, 1, 33]), (2, 129, 8, 1, 64, [129, 64]),
    (4, 1000, 16, 4, 128, [1000, 17, 999, 256]), (2, 777, 3, 1, 128, [500, 777]), (2, 2100, 6, 2, 64, [31, 2100]),
    (1, 5003, 8, 2, 128, [5003])])
def test_decode_kv4_parity(B, L, h, hkv, d, lens, layout):
    """Ragged lengths, one to sixteen query heads per KV head, every layout;
    the records behind each sequence hold NaN."""
    g, cache, q, gate, sl = make(B, L, h, hkv, d, lens, 200 + L + h, layout)
    w_in = torch.rand((B, hkv, L), generator=g, device="cuda")
    w = torch.full((B, hkv, L), -3.0, device="cuda")
    before = w.clone()
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w_in, weights_out=w)
    plain = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate)
    torch.cuda.synchronize()
    assert torch.equal(out, plain)  # gathering weights does not change the output
    kf, vf, rk, rv = ranges(clean(cache, lens))
    check_decode(q, kf, vf, rk, rv, lens, f64(gate), out, w, w_in, before)


@pytest.mark.parametrize("d,G", [(d, G) for d in (64, 128) for G in (2, 4, 6, 8, 10, 12, 14, 16)])
def test_decode_kv4_every_group_size(d, G):
    lens = [201, 64]
    g, cache, q, gate, sl = make(2, 201, G, 2, d, lens, 300 + G + d)
    w = torch.zeros((2, 2, 201), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=w)
    kf, vf, rk, rv = ranges(clean(cache, lens))
    check_decode(q, kf, vf, rk, rv, lens, f64(gate), out, w, None, torch.zeros_like(w))


@pytest.mark.parametrize("case", ["rising", "sink", "tiny_v", "huge_v", "mixed_v", "sharp", "big_q"])
def test_decode_kv4_magnitudes(case):
    """Scores that keep rising, a dominant first key, value scales from 1e-6 to
    1e6 in one sequence, a near one-hot softmax, large queries."""
    B, L, h, hkv, d = 1, 700, 4, 1, 128
    g = gen(400 + len(case))
    k, v, q = randn((B, L, hkv, d), g), randn((B, L, hkv, d), g), randn((B, 2 * h, d), g)
    scale = 0.0
    if case == "rising":
        k *= torch.linspace(0.05, 6.0, L, device="cuda").to(BF16)[None, :, None, None]
    elif case == "sink":
        k[:, 0] = q[:, :1] * 3
        v[:, 0] = 0.001
    elif case == "tiny_v":
        v *= 1e-6
    elif case == "huge_v":
        v *= 1e6
    elif case == "mixed_v":
        v *= torch.logspace(-6, 6, L, device="cuda").flip(0).to(BF16)[None, :, None, None]
    elif case == "sharp":
        scale = 3.0
    elif case == "big_q":
        q *= 40.0
    cache = new_cache(B, L, hkv, d)
    bd.diffattn_kv4_append(k, v, cache)
    gate = torch.rand((B, h), generator=g, device="cuda")
    w = torch.zeros((B, hkv, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w, softmax_scale=scale)
    kf, vf, rk, rv = ranges(cache.cpu().numpy())
    check_decode(q, kf, vf, rk, rv, [L], f64(gate), out, w, None, torch.zeros_like(w), scale=scale or None)


def test_decode_kv4_gate_from_x_and_strided_views():
    """The gate computed from x is the one that diffattn_v2_gate gives; caches
    that are slices of a larger allocation."""
    lens = [90, 64]
    g, big, q, _, sl = make(2, 90, 4, 4, 128, lens, 500, "token")
    x, wl = randn((2, 256), g), randn((256, 4), g, 0.02)
    gate = bd.diffattn_v2_gate(x, wl)
    a = bd.diffattn_v2_decode_kv4(q, big, seqlens=sl, x=x, w_lambda=wl)
    b = bd.diffattn_v2_decode_kv4(q, big, seqlens=sl, gate=gate)
    assert torch.equal(a, b)
    half = big[:, :, 1:3]  # KV heads 1 and 2
    c = bd.diffattn_v2_decode_kv4(q[:, 2:6].contiguous(), half, seqlens=sl, gate=gate[:, 1:3].contiguous())
    # other heads beside them cut the work elsewhere: equal up to the order of fp32 sums
    kf, vf, rk, rv = ranges(clean(half, lens))
    check_decode(q[:, 2:6], kf, vf, rk, rv, lens, f64(gate[:, 1:3]), c)
    check_decode(q[:, 2:6], kf, vf, rk, rv, lens, f64(gate[:, 1:3]), b[:, 1:3])


def test_decode_kv4_exact_cancellation_and_repeats():
    """Equal even and odd queries with gate 1: zero output and no weight
    gathered; a repeated call gives the same bits."""
    g, cache, q, gate, _ = make(2, 3000, 8, 2, 128, [3000, 3000], 510)
    q[:, 1::2] = q[:, 0::2]
    one = torch.ones_like(gate)
    w = torch.zeros((2, 2, 3000), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=one, weights_out=w)
    assert torch.count_nonzero(out).item() == 0 and torch.count_nonzero(w).item() == 0
    a = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w)
    w2 = torch.zeros_like(w)
    b = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w2)
    assert torch.equal(a, b) and torch.equal(w, w2)


def test_decode_kv4_accumulates_in_place():
    g, cache, q, gate, sl = make(2, 300, 4, 2, 64, [300, 150], 520)
    w = torch.rand((2, 2, 300), generator=g, device="cuda")
    apart = torch.full_like(w, 5.0)
    bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w, weights_out=apart)
    w0 = w.clone()
    bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w, weights_out=w)
    assert torch.equal(w[0], apart[0]) and torch.equal(w[1, :, :150], apart[1, :, :150])
    assert torch.equal(w[1, :, 150:], w0[1, :, 150:]) and float(apart[1, :, 150:].min()) == 5.0


def test_decode_kv4_bad_lengths_are_recorded():
    g, cache, q, gate, _ = make(3, 64, 2, 1, 64, [64, 64, 64], 530)
    sl = torch.tensor([0, 65, 64], dtype=torch.int32, device="cuda")
    w = torch.full((3, 1, 64), 2.0, device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=w)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    assert torch.count_nonzero(out[:2]).item() == 0 and torch.count_nonzero(out[2]).item() > 0
    assert float(w[:2].min()) == float(w[:2].max()) == 2.0 and float(w[2].max()) < 2.0


def test_decode_kv4_nan_record_gives_nan():
    """A NaN row inside the sequence reaches its KV head's outputs and weights
    and no other head's."""
    g, cache, q, gate, _ = make(1, 100, 4, 2, 128, [100], 540)
    bad = torch.full((1, 1, 2, 128), float("nan"), dtype=BF16, device="cuda")
    ok = randn((1, 1, 2, 128), g)
    bad[:, :, 1] = ok[:, :, 1]
    bd.diffattn_kv4_append(bad, ok, cache, start=torch.tensor([40], dtype=torch.int32, device="cuda"))
    w = torch.zeros((1, 2, 100), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w)
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isfinite(out[0, 2:]).all())
    assert bool(torch.isnan(w[0, 0]).all()) and bool(torch.isfinite(w[0, 1]).all())


@pytest.mark.parametrize("d", [64, 128])
def test_decode_kv4_nan_beside_growing_values(d):
    """A NaN in one half of a value row leaves the other half's features right,
    also where the value scales grow by orders of magnitude in the same keys."""
    B, L, h, hkv = 1, 96, 2, 1
    g = gen(545)
    k, v, q = randn((B, L, hkv, d), g, 0.1), randn((B, L, hkv, d), g), randn((B, 2 * h, d), g)
    v[:, 40:] *= 1000.0
    v[0, 40:64:3, 0, 3] = float("nan")  # keys of the first group only
    cache = new_cache(B, L, hkv, d)
    bd.diffattn_kv4_append(k, v, cache)
    gate = torch.rand((B, h), generator=g, device="cuda")
    w = torch.zeros((B, hkv, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w)
    assert bool(torch.isnan(out[..., :d // 2]).all()) and bool(torch.isfinite(w).all())
    kf, vf, rk, rv = ranges(cache.cpu().numpy())
    half = slice(d // 2, d)
    ref = orc.v2_decode(f64(q), kf, np.nan_to_num(vf), [L], f64(gate))["out"][0][:, half]
    got = f64(out)[0][:, half]
    # as check_decode: the output's rounding, and 2^-11 of the values' range
    v_range = 15 * np.abs(kvo.kv4_quantise(f64(v)[..., half].repeat(2, -1))[1]).max()
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * 2.0 ** -11 * v_range + 1e-4 * np.abs(vf[..., half]).max())


def test_decode_kv4_many_sequences():
    """More (sequence, head) units than SMs, short and ragged."""
    B = 70
    lens = [int(x) for x in np.random.default_rng(8).integers(1, 97, B)]
    g, cache, q, gate, sl = make(B, 96, 4, 4, 128, lens, 550)
    w = torch.zeros((B, 4, 96), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=w)
    kf, vf, rk, rv = ranges(clean(cache, lens))
    check_decode(q, kf, vf, rk, rv, lens, f64(gate), out, w, None, torch.zeros_like(w))


@pytest.mark.parametrize("d,G,layout", [(64, 2, "head"), (64, 12, "token"), (128, 4, "padded")])
def test_decode_kv4_more_sequences_than_threads(d, G, layout):
    """1300 sequences of 0 to 45 keys: every block sums the lengths in tiles of
    its 512 or 256 threads and finds its part in one of them.  Lengths of 0 are
    recorded and their rows zero; the others are right."""
    B, L = 1300, 45
    lens = [int(x) for x in np.random.default_rng(d + G).integers(0, L + 1, B)]
    g, cache, q, gate, sl = make(B, L, G // 2, 1, d, lens, 552, layout)
    w = torch.zeros((B, 1, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=w)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    zero = [b for b in range(B) if lens[b] == 0]
    full = [b for b in range(B) if lens[b]]
    assert zero and torch.count_nonzero(out[zero]).item() == 0 and torch.count_nonzero(w[zero]).item() == 0
    some = full[::7] + full[-3:]
    kf, vf, rk, rv = ranges(clean(cache[some], [lens[b] for b in some]))
    check_decode(q[some], kf, vf, rk, rv, [lens[b] for b in some], f64(gate[some]), out[some], w[some], None,
                 torch.zeros_like(w[some]))


def test_append_more_sequences_than_a_grid_dimension():
    """70000 sequences, a row each: blocks walk the sequences behind the first 65535."""
    B, d = 70_000, 64
    k, v = randn((B, 1, 1, d), gen(7)), randn((B, 1, 1, d), gen(8))
    cache = new_cache(B, 1, 1, d)
    bd.diffattn_kv4_append(k, v, cache)
    for part in (slice(0, 300), slice(65_400, 65_700), slice(69_900, B)):
        assert np.array_equal(cache[part].cpu().numpy(), kvo.kv4_pack(f64(k[part]), f64(v[part])))
    kb, _ = bd.diffattn_kv4_read(cache, 1)
    err = (kb.double() - k.double()).abs().amax(-1)
    assert float(err.max()) < 1.0  # every row came back


def test_decode_kv4_two_streams_at_once():
    """Two calls in flight on two streams, each with a workspace of its own."""
    made = [make(2, 4000, 4, 2, 128, [4000, 2500], 590 + i) for i in range(2)]
    want = [bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate) for _, cache, q, gate, sl in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, (_, cache, q, gate, sl) in enumerate(made):
            got[i].append(bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_decode_kv4_shared_prefix_and_views():
    """One cache read by every sequence of a batch (batch stride 0), and a
    contiguous run of positions of a longer cache."""
    g, cache, q, gate, _ = make(1, 300, 4, 2, 64, [300], 595)
    qs, gates = randn((3, 8, 64), g), torch.rand((3, 4), generator=g, device="cuda")
    both = bd.diffattn_v2_decode_kv4(qs, cache.expand(3, 300, 2, 80), gate=gates)
    same = bd.diffattn_v2_decode_kv4(qs, cache.repeat(3, 1, 1, 1).contiguous(), gate=gates)
    kf, vf, rk, rv = ranges(cache.expand(3, 300, 2, 80).cpu().numpy())
    for out in (both, same):
        check_decode(qs, kf, vf, rk, rv, [300] * 3, f64(gates), out)
    part = cache[:, 100:250]
    out = bd.diffattn_v2_decode_kv4(q, part, gate=gate)
    kf, vf, rk, rv = ranges(part.cpu().numpy())
    check_decode(q, kf, vf, rk, rv, [150], f64(gate), out)


def test_decode_kv4_long_sums_lose_nothing():
    """Over 16.8 million records (some 220 chunks of 32 keys per warp) the
    output's RMS error against 64 bits stays at its own rounding.  A bf16 value
    x in [1, 2) is off by 2^-8 / sqrt(3) in the mean square, 1.63e-3 of x after
    the mean of 1 / x^2 = 1/2 over values spread evenly in a binade (1.66e-3
    where their logarithm is).  P s in 16 bits is off by 2^-11 / sqrt(3) at
    most, and a code's mean square, 8.7 s, is 2.6 to 2.9 of the values' own:
    8e-4 of the output.  Together 1.9e-3; fp32 steps add 1e-5 of it.  Sums that
    lose bits at every step add what grows with the length (chained through the
    tensor cores' accumulators they gave 2.8e-3)."""
    B, L, hkv, d = 32, 32768, 16, 64
    g = gen(565)
    cache = new_cache(B, L, hkv, d)
    for b in range(B):
        bd.diffattn_kv4_append(randn((1, L, hkv, d), g), randn((1, L, hkv, d), g), cache[b:b + 1])
    q, gate = randn((B, 2 * hkv, d), g), torch.rand((B, hkv), generator=g, device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate)
    num = den = 0.0
    for b in (0, 13, 31):
        rec = cache[b].transpose(0, 1).contiguous()  # [hkv, L, d + 16]
        rows = []
        for i in (0, 1):
            c = rec[..., i * (d // 2):(i + 1) * (d // 2)]
            n = torch.stack((c & 15, c >> 4), -1).flatten(-2).double().unflatten(-1, (2, -1))
            p = rec[..., d + 8 * i:d + 8 * i + 8].contiguous().view(BF16).double()
            rows.append((n * p[..., 0:2, None] + p[..., 2:4, None]).flatten(-2))
        a = torch.softmax(q[b].double().reshape(hkv, 2, d) @ rows[0].transpose(1, 2) * d ** -0.5, -1)
        ref = (a @ rows[1])[:, 0] - gate[b].double()[:, None] * (a @ rows[1])[:, 1]
        num += float((out[b].double() - ref).square().sum())
        den += float(ref.square().sum())
    record({"rms": (num / den) ** 0.5 / 2e-3})
    assert (num / den) ** 0.5 <= 2e-3
    del cache
    torch.cuda.empty_cache()


def test_decode_kv4_long_cache_offsets():
    """A cache whose byte offsets pass 2^32: two sequences 4.5 GB apart."""
    L, hkv, d = 5000, 2, 128
    big = torch.zeros((4_600_000_000,), dtype=torch.uint8, device="cuda")
    cache = big.as_strided((2, L, hkv, d + 16), (4_500_000_000 // 16 * 16, d + 16, L * (d + 16), 1))
    g = gen(560)
    bd.diffattn_kv4_append(randn((2, L, hkv, d), g), randn((2, L, hkv, d), g), cache)
    q, gate = randn((2, 8, d), g), torch.rand((2, 4), generator=g, device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate)
    same = bd.diffattn_v2_decode_kv4(q, cache.contiguous(), gate=gate)
    assert torch.equal(out, same)
    kf, vf, rk, rv = ranges(cache.cpu().numpy())
    check_decode(q, kf, vf, rk, rv, [L, L], f64(gate), out)


def test_decode_kv4_other_stream_and_graph():
    """On a side stream, and captured with the append of the step's token:
    replays follow the inputs."""
    g, cache, q, gate, _ = make(2, 256, 4, 2, 128, [200, 100], 570)
    k, v = randn((2, 1, 2, 128), g), randn((2, 1, 2, 128), g)
    start = torch.tensor([200, 100], dtype=torch.int32, device="cuda")
    sl = start + 1
    w = torch.zeros((2, 2, 256), device="cuda")
    ws = torch.empty((bd.diffattn_v2_decode_kv4_workspace_size(2, 4, 2, 128, 256, True, True),), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty((2, 4, 128), dtype=BF16, device="cuda")

    def step():
        bd.diffattn_kv4_append(k, v, cache, start=start)
        bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=w, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    assert torch.equal(out, first)
    for seed in (571, 572):
        for t in (k, v, q):
            t.copy_(randn(tuple(t.shape), gen(seed + t.dim())))
        graph.replay()
        torch.cuda.synchronize()
        got, gw = out.clone(), w.clone()
        step()
        assert torch.equal(out, got) and torch.equal(w, gw)


def test_decode_kv4_gate_from_x_in_a_graph():
    """The gate's projection, the decode that runs beside it and the weights,
    captured: replays follow the inputs, also back to back, where one replay's
    gate must not start on the workspace before the last one's merge is done."""
    g, cache, q, _, _ = make(3, 700, 8, 2, 128, [700, 300, 512], 575)
    x, wl = randn((3, 512), g), randn((512, 8), g, 0.05)
    sl = torch.tensor([700, 300, 512], dtype=torch.int32, device="cuda")
    w = torch.zeros((3, 2, 700), device="cuda")
    ws = torch.empty((bd.diffattn_v2_decode_kv4_workspace_size(3, 8, 2, 128, 700, False, True),), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty((3, 8, 128), dtype=BF16, device="cuda")

    def step():
        bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, x=x, w_lambda=wl, weights_out=w, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(576, 582):
        x.copy_(randn((3, 512), gen(seed)))
        q.copy_(randn((3, 16, 128), gen(seed + 100)))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        got, gw = out.clone(), w.clone()
        gate = bd.diffattn_v2_gate(x, wl)
        want_w = torch.zeros_like(w)
        # the gate given: cut for all SMs, so the fp32 sums may associate otherwise
        want = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=want_w)
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(w, gw)
        assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max())
        assert float((gw - want_w).abs().max()) <= 1e-5 * float(want_w.max())


def _sweep(seed):
    r = np.random.default_rng(seed)
    d, hkv, G = int(r.choice([64, 128])), int(r.choice([1, 2, 3, 8])), 2 * int(r.integers(1, 9))
    B, L = int(r.integers(1, 6)), int(np.exp(r.uniform(0, np.log(3000))))
    lens = [int(x) for x in r.integers(1, L + 1, B)]
    return dict(B=B, L=L, h=hkv * G // 2, hkv=hkv, d=d, lens=lens, layout=str(r.choice(["head", "token", "padded"])),
                scale=float(r.choice([0.0, 0.05, 0.4])), k_std=float(r.choice([0.3, 1.0, 2.0])),
                v_std=float(r.choice([1e-3, 1.0, 50.0])), from_x=bool(r.random() < 0.3), weights=bool(r.random() < 0.7))


@pytest.mark.parametrize("seed", range(24))
def test_decode_kv4_swept_shapes(seed):
    c = _sweep(9000 + seed)
    g, cache, q, gate, sl = make(c["B"], c["L"], c["h"], c["hkv"], c["d"], c["lens"], 9100 + seed, c["layout"],
                                 c["k_std"], c["v_std"])
    kw = dict(gate=gate)
    if c["from_x"] and c["h"] <= 64:
        kw = dict(x=randn((c["B"], 192), g), w_lambda=randn((192, c["h"]), g, 0.1))
        gate = bd.diffattn_v2_gate(kw["x"], kw["w_lambda"])
    w = w_in = before = None
    if c["weights"]:
        w_in = torch.rand((c["B"], c["hkv"], c["L"]), generator=g, device="cuda")
        w = torch.full_like(w_in, -2.0)
        before = w.clone()
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, softmax_scale=c["scale"], weights_in=w_in, weights_out=w, **kw)
    kf, vf, rk, rv = ranges(clean(cache, c["lens"]))
    check_decode(q, kf, vf, rk, rv, c["lens"], f64(gate), out, w, w_in, before, scale=c["scale"] or None)


# A cache that can hold more keys than the short path takes sends the same
# short sequences through the line of chunks and the merge after it; one that
# cannot gives every head a block or a cluster of them.  LINE is past the
# longest short cache.
LINE = 8200


@pytest.mark.parametrize("layout", ["head", "token", "padded"])
@pytest.mark.parametrize("d,G", [(d, G) for d in (64, 128) for G in (2, 4, 8, 10, 16)])
def test_decode_kv4_short_sequences_in_a_long_cache(d, G, layout):
    lens = [201, 64, 1, 33]
    g, cache, q, gate, sl = make(4, LINE, G, 2, d, lens, 610 + G + d, layout)
    w_in = torch.rand((4, 2, LINE), generator=g, device="cuda")
    w = torch.full_like(w_in, -3.0)
    before = w.clone()
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w_in, weights_out=w)
    kf, vf, rk, rv = ranges(clean(cache, lens))
    check_decode(q, kf, vf, rk, rv, lens, f64(gate), out, w, w_in, before)
    short = cache[:, :201]  # the same records, a block per head
    w2 = torch.full((4, 2, 201), -3.0, device="cuda")
    out2 = bd.diffattn_v2_decode_kv4(q, short, seqlens=sl, gate=gate, weights_in=w_in[..., :201].contiguous(),
                                     weights_out=w2)
    check_decode(q, kf, vf, rk, rv, lens, f64(gate), out2, w2, w_in, torch.full_like(w, -3.0)[..., :201])


@pytest.mark.parametrize("layout", ["head", "padded"])
@pytest.mark.parametrize("d,G", [(64, 2), (64, 16), (128, 8), (128, 10)])
@pytest.mark.parametrize("B,hkv,L,lens", [(1, 1, 8192, [8191]), (3, 1, 8000, [1, 4100, 31]), (2, 8, 2048, [2048, 1025]),
                                          (4, 8, 4096, [33, 4096, 1, 500]), (5, 8, 1100, [1100, 512, 64, 1099, 2]),
                                          (12, 4, 2048, [2048, 7] * 6), (2, 2, 1025, [1025, 32])])
def test_decode_kv4_clusters(B, hkv, L, lens, d, G, layout):
    """A cluster of two, four or eight blocks per head: full heads, heads with
    fewer chunks than warps or than blocks; a repeated call gives the same bits."""
    g, cache, q, gate, sl = make(B, L, hkv * G // 2, hkv, d, lens, 680 + G + L, layout)
    w_in = torch.rand((B, hkv, L), generator=g, device="cuda")
    w = torch.full_like(w_in, -3.0)
    before = w.clone()
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w_in, weights_out=w)
    assert torch.equal(out, bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate))
    w2 = w_in.clone()
    assert torch.equal(out, bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w2, weights_out=w2))
    for b, n in enumerate(lens):
        assert torch.equal(w2[b, :, :n], w[b, :, :n]) and torch.equal(w2[b, :, n:], w_in[b, :, n:])
    kf, vf, rk, rv = ranges(clean(cache, lens))
    check_decode(q, kf, vf, rk, rv, lens, f64(gate), out, w, w_in, before)


@pytest.mark.parametrize("B,L", [(33, 2048), (34, 2048), (38, 2048), (39, 1025), (76, 1025), (77, 2048), (9, 8192),
                                 (10, 8192), (33, 4096)])
def test_decode_kv4_as_many_clusters_as_fit(B, L):
    lens = [1 + (131 * b) % L for b in range(B)]
    lens[-1] = L
    g, cache, q, gate, sl = make(B, L, 2, 1, 64, lens, 695)
    w = torch.zeros((B, 1, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=w)
    kf, vf, rk, rv = ranges(clean(cache, lens))
    check_decode(q, kf, vf, rk, rv, lens, f64(gate), out, w, None, torch.zeros_like(w))


def test_decode_kv4_clusters_bad_lengths_and_nan():
    L = 2000
    g, cache, q, gate, _ = make(4, L, 4, 2, 128, [100, 100, 100, L], 690)
    sl = torch.tensor([0, L + 1, -5, L], dtype=torch.int32, device="cuda")
    w = torch.full((4, 2, L), 2.0, device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=w)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    assert torch.count_nonzero(out[:3]).item() == 0 and torch.count_nonzero(out[3]).item() > 0
    assert float(w[:3].min()) == float(w[:3].max()) == 2.0 and float(w[3].max()) < 2.0
    bad = torch.full((1, 1, 2, 128), 0.5, dtype=BF16, device="cuda")
    bad[:, :, 0] = float("nan")
    bd.diffattn_kv4_append(bad, bad, cache[3:], start=torch.tensor([L - 1], dtype=torch.int32, device="cuda"))
    out = bd.diffattn_v2_decode_kv4(q[3:], cache[3:], seqlens=sl[3:], gate=gate[3:], weights_out=w[3:])
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isfinite(out[0, 2:]).all())
    assert bool(torch.isnan(w[3, 0]).all()) and bool(torch.isfinite(w[3, 1]).all())


def test_decode_kv4_long_cache_bad_lengths_nan_and_in_place():
    """The line's own refusals: lengths of 0, below 0 and past the cache beside
    a good one, a NaN record, weights taken in place."""
    lens = [0, LINE + 1, -1, 100]
    g, cache, q, gate, _ = make(4, LINE, 4, 2, 128, [100] * 4, 630)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w = torch.rand((4, 2, LINE), generator=g, device="cuda")
    w0 = w.clone()
    apart = torch.full_like(w, 5.0)
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w, weights_out=apart)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    again = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w, weights_out=w)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    assert torch.equal(out, again) and torch.count_nonzero(out[:3]).item() == 0
    assert torch.equal(w[:3], w0[:3]) and torch.equal(w[3, :, 100:], w0[3, :, 100:])
    assert torch.equal(w[3, :, :100], apart[3, :, :100]) and float(apart[:3].min()) == float(apart[:3].max()) == 5.0
    bad = torch.full((1, 1, 2, 128), float("nan"), dtype=BF16, device="cuda")
    bad[:, :, 1] = 0.5
    bd.diffattn_kv4_append(bad, bad[:, :, 1:].expand(1, 1, 2, 128).contiguous(), cache[3:],
                           start=torch.tensor([40], dtype=torch.int32, device="cuda"))
    out = bd.diffattn_v2_decode_kv4(q[3:], cache[3:], seqlens=sl[3:], gate=gate[3:], weights_out=w[3:])
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isfinite(out[0, 2:]).all())
    assert bool(torch.isnan(w[3, 0, :100]).all()) and bool(torch.isfinite(w[3, 1]).all())


@pytest.mark.parametrize("case", ["rising", "mixed_v", "sharp"])
@pytest.mark.parametrize("L", [700, 2200, LINE + 120])
def test_decode_kv4_magnitudes_on_either_path(case, L):
    """References that must move within a warp's part and between parts, d = 64
    and two head tiles."""
    h, hkv, d = 6, 1, 64
    g = gen(640 + len(case))
    k, v, q = randn((1, L, hkv, d), g), randn((1, L, hkv, d), g), randn((1, 2 * h, d), g)
    if case == "rising":
        k *= torch.linspace(0.05, 6.0, L, device="cuda").to(BF16)[None, :, None, None]
    elif case == "mixed_v":
        v *= torch.logspace(-6, 6, L, device="cuda").flip(0).to(BF16)[None, :, None, None]
    scale = 3.0 if case == "sharp" else 0.0
    cache = new_cache(1, L, hkv, d)
    bd.diffattn_kv4_append(k, v, cache)
    gate = torch.rand((1, h), generator=g, device="cuda")
    w = torch.zeros((1, hkv, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w, softmax_scale=scale)
    kf, vf, rk, rv = ranges(cache.cpu().numpy())
    check_decode(q, kf, vf, rk, rv, [L], f64(gate), out, w, None, torch.zeros_like(w), scale=scale or None)


@pytest.mark.parametrize("more", [-1, 0, 1])
@pytest.mark.parametrize("L", [1024, 1025, 2048, 2049])
def test_decode_kv4_where_the_paths_meet(more, L):
    """As many heads as there are SMs, one more and one fewer, at caches of the
    lengths where the path changes; most sequences short, the last ones full."""
    B = torch.cuda.get_device_properties(0).multi_processor_count + more
    lens = [1 + (7 * b) % 41 for b in range(B)]
    lens[-1], lens[-2], lens[0] = L, L - 1, 1
    g, cache, q, gate, sl = make(B, L, 2, 1, 64, lens, 650 + more)
    w = torch.zeros((B, 1, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_out=w)
    some = list(range(0, B, 9)) + [B - 2, B - 1]
    n = [lens[b] for b in some]
    kf, vf, rk, rv = ranges(clean(cache[some], n))
    check_decode(q[some], kf, vf, rk, rv, n, f64(gate[some]), out[some], w[some], None, torch.zeros_like(w[some]))


@pytest.mark.parametrize("L", [700, 2000, LINE])
def test_decode_kv4_gate_from_x_captured_on_either_path(L):
    g, cache, q, _, sl = make(2, L, 4, 2, 128, [300, 555], 660)
    x, wl = randn((2, 256), g), randn((256, 4), g, 0.05)
    w, w2 = torch.zeros((2, 2, L), device="cuda"), torch.zeros((2, 2, L), device="cuda")
    ws = torch.empty((bd.diffattn_v2_decode_kv4_workspace_size(2, 4, 2, 128, L, False, True),), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty((2, 4, 128), dtype=BF16, device="cuda")

    def step():
        bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, x=x, w_lambda=wl, weights_out=w, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (661, 662):
        x.copy_(randn((2, 256), gen(seed)))
        q.copy_(randn((2, 8, 128), gen(seed + 10)))
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        kf, vf, rk, rv = ranges(clean(cache, [300, 555]))
        check_decode(q, kf, vf, rk, rv, [300, 555], f64(bd.diffattn_v2_gate(x, wl)), out, w, None, w2)


@pytest.mark.parametrize("lens,d,G", [([80000] * 4, 64, 2), ([80000, 79999, 70001, 80000], 64, 12),
                                      ([80000, 1, 33, 64], 64, 4), ([80000, 79000, 80000, 78001], 128, 8)])
def test_decode_kv4_gate_from_x_over_long_caches(lens, d, G):
    """Parts of unequal length beside the gate's projection: every key is taken
    once.  The workspace holds NaN before, so a key that was passed over leaves
    one in its weight."""
    B, L, hkv = 4, 80000, 8
    g, cache, q, _, sl = make(B, L, hkv * G // 2, hkv, d, lens, 670 + G)
    x, wl = randn((B, 256), g), randn((256, hkv * G // 2), g, 0.05)
    need = bd.diffattn_v2_decode_kv4_workspace_size(B, hkv * G // 2, hkv, d, L, False, True)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    w, want_w = torch.zeros((B, hkv, L), device="cuda"), torch.zeros((B, hkv, L), device="cuda")
    out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, x=x, w_lambda=wl, weights_out=w, workspace=ws)
    want = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=bd.diffattn_v2_gate(x, wl), weights_out=want_w)
    for b, n in enumerate(lens):
        assert bool(torch.isfinite(w[b, :, :n]).all()) and torch.count_nonzero(w[b, :, n:]).item() == 0
        top = float(want[b].float().abs().max())
        # other cuts: fp32 sums associate otherwise; then one bf16 rounding each
        assert float((out[b].float() - want[b].float()).abs().max()) <= 2.0 ** -7 * top
        assert float((w[b] - want_w[b]).abs().max()) <= 1e-5 * float(want_w[b].max())


def test_prefix_read_back_feeds_the_forward():
    """A cached prefix read back and attended by diffattn_v2_fwd gives, for the
    last position, the decode's result over the same records."""
    B, N, h, hkv, d = 1, 200, 4, 2, 128
    g, cache, _, gate, _ = make(B, N, h, hkv, d, [N], 580)
    k, v = bd.diffattn_kv4_read(cache, N)
    q = randn((B, N, 2 * h, d), g)
    full = bd.diffattn_v2_fwd(q, k, v, gate=gate[:, None].expand(B, N, h).contiguous())
    out = bd.diffattn_v2_decode_kv4(q[:, -1].contiguous(), cache, gate=gate)
    # k and v rounded to bf16, P in bf16: the forward's parity bar
    rms = float(v.float().pow(2).mean().sqrt())
    assert float((full[:, -1].float() - out.float()).abs().max()) <= 2e-2 * rms
