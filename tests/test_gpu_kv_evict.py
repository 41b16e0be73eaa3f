"""Gathered key weights over a bf16 cache, eviction by gathered weight, and the
operators together as a serving loop uses them.  Eviction moves bytes, so its
results are compared exactly."""

import numpy as np
import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from differential_attention_diff_gb300 import synth
from oracle import kv_oracle as kvo
from test_gpu_kv4 import BF16, check_decode, clean, f64, gen, make, new_cache, randn, ranges

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert bd.diffattn_get_device_status() == bd.DA_OK


# ---------------------------------------------- gathered weights, bf16 ------
@pytest.mark.parametrize("B,L,h,hkv,d,lens,splits", [
    (1, 1, 1, 1, 128, [1], 0), (2, 300, 4, 2, 64, [300, 1], 0), (3, 1000, 16, 2, 128, [1000, 127, 640], 0),
    (1, 4097, 8, 8, 128, [4097], 0), (2, 900, 3, 1, 64, [900, 333], 7), (1, 3000, 32, 8, 128, [3000], 2)])
def test_decode_weighted_parity(B, L, h, hkv, d, lens, splits):
    t = synth.decode_inputs(B, L, h, hkv, d, 128, seed=600 + L, device="cuda", seqlens=lens)
    for b, n in enumerate(lens):  # behind each sequence: NaN
        t["k_cache"][b, n:] = float("nan")
    g = gen(601)
    gate = torch.rand((B, h), generator=g, device="cuda")
    w_in = torch.rand((B, hkv, L), generator=g, device="cuda")
    w = torch.full((B, hkv, L), -1.0, device="cuda")
    before = w.clone()
    kw = dict(seqlens=t["seqlens"], gate=gate, num_splits=splits)
    out = bd.diffattn_v2_decode_weighted(t["q"], t["k_cache"], t["v_cache"], weights_in=w_in, weights_out=w, **kw)
    plain = bd.diffattn_v2_decode(t["q"], t["k_cache"], t["v_cache"], **kw)
    assert torch.equal(out, plain)
    kf, vf = f64(t["k_cache"]), f64(t["v_cache"])
    for b, n in enumerate(lens):
        kf[b, n:] = 0
    rk, rv = np.abs(kf).max(-1), np.abs(vf).max(-1)
    # P is bf16 here: 8 bits
    check_decode(t["q"], kf, vf, rk, rv, lens, f64(gate), out, w, w_in, before, p_bits=8)


def test_decode_weighted_gate_from_x_and_bad_length():
    t = synth.decode_inputs(3, 200, 4, 2, 128, 128, seed=620, device="cuda", seqlens=[200, 0, 201])
    w = torch.full((3, 2, 200), 2.0, device="cuda")
    out = bd.diffattn_v2_decode_weighted(t["q"], t["k_cache"], t["v_cache"], seqlens=t["seqlens"], x=t["x"],
                                         w_lambda=t["w_lambda"], weights_out=w)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    assert torch.count_nonzero(out[1:]).item() == 0 and float(w[1:].min()) == float(w[1:].max()) == 2.0
    gate = bd.diffattn_v2_gate(t["x"], t["w_lambda"])
    w2 = torch.zeros((1, 2, 200), device="cuda")
    one = bd.diffattn_v2_decode_weighted(t["q"][:1], t["k_cache"][:1], t["v_cache"][:1], gate=gate[:1], weights_out=w2)
    assert torch.equal(one[0], out[0]) and torch.equal(w2[0], w[0])


# -------------------------------------------------------------- eviction ----
def run_evict(B, hkv, L, keep, lens, *, sinks=0, recent=0, weights, positions=None, nxt=None, widths=((64, BF16),),
              inplace=False, layout="head", seed=0):
    """Runs the eviction on random rows and checks every output and every slot."""
    g = gen(seed)
    rows = []
    for width, dt in widths:
        shape = (B, hkv, L, width) if layout == "head" else (B, L, hkv, width)
        bits = torch.randint(0, 256, (*shape[:-1], width * torch.empty((), dtype=dt).element_size()), generator=g,
                             device="cuda", dtype=torch.uint8)
        t = bits.view(dt)
        rows.append(t.transpose(1, 2) if layout == "head" else t)
    raw = [r.contiguous().view(torch.uint8).cpu().numpy().copy() for r in rows]
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w_np = weights.cpu().numpy().copy()
    p_np = None if positions is None else positions.cpu().numpy().copy()
    if inplace:
        kw = dict(seqlens=sl, positions=positions)
        exp_w = w_np.copy()
        exp_p = None if p_np is None else p_np.copy()
    else:
        kw = dict(seqlens=sl, positions=positions, weights_out=torch.full_like(weights, -9.0),
                  positions_out=torch.full((B, hkv, L), -9, dtype=torch.int32, device="cuda"),
                  seqlens_out=torch.full_like(sl, -9))
        exp_w, exp_p = np.full_like(w_np, -9.0), np.full((B, hkv, L), -9)
    r = bd.diffattn_kv_evict(rows, weights, keep, sinks=sinks, recent=recent,
                             next_position=None if nxt is None else torch.tensor(nxt, dtype=torch.int32, device="cuda"),
                             **kw)
    exp = [x.copy() for x in raw]
    for b in range(B):
        n = lens[b]
        for h in range(hkv):
            pos = None if p_np is None else p_np[b, h, :n]
            m, source = kvo.evict(w_np[b, h, :n], keep, sinks=sinks, recent=recent, positions=pos,
                                  next_position=None if nxt is None else nxt[b])
            exp_w[b, h, :m] = w_np[b, h, source]
            if exp_p is not None:
                exp_p[b, h, :m] = np.asarray(source) if pos is None else pos[source]
            for x, o in zip(exp, raw):
                x[b, :m, h] = o[b, source, h]
    assert r["seqlens"].tolist() == [min(n, keep) for n in lens]
    assert np.array_equal(r["key_weights"].cpu().numpy(), exp_w, equal_nan=True)
    if exp_p is not None:
        assert np.array_equal(r["positions"].cpu().numpy(), exp_p)
    for x, t in zip(exp, rows):
        assert np.array_equal(t.contiguous().view(torch.uint8).cpu().numpy(), x)
    if not inplace:
        assert np.array_equal(weights.cpu().numpy(), w_np, equal_nan=True) and sl.tolist() == lens
    return r


def spread(shape, seed, ties=True):
    g = gen(seed)
    w = torch.randn(shape, generator=g, device="cuda").mul_(2).exp_()
    if ties:
        w = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.3, w.round(), w)
    return w


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,hkv,L,keep,lens,sinks,recent", [
    (1, 1, 1, 1, [1], 0, 0), (1, 1, 2, 1, [2], 0, 1), (2, 3, 100, 50, [100, 51], 4, 10), (2, 2, 100, 99, [100, 7], 0, 0),
    (3, 2, 1025, 64, [1025, 1024, 0], 1, 63), (1, 2, 5000, 2500, [5000], 4, 256), (1, 1, 3000, 1, [2999], 0, 0),
    (2, 1, 40, 64, [40, 13], 4, 32), (1, 1, 70000, 30000, [70000], 16, 1000)])
def test_evict_parity(B, hkv, L, keep, lens, sinks, recent, inplace):
    run_evict(B, hkv, L, keep, lens, sinks=sinks, recent=recent, weights=spread((B, hkv, L), 700 + L),
              widths=((64, BF16), (64, BF16)), inplace=inplace, seed=L)


@pytest.mark.parametrize("layout", ["head", "token"])
def test_evict_with_positions_and_row_kinds(layout):
    """Slots in no order of position; K1, K2 and V of different widths; records."""
    B, hkv, L, seen = 2, 2, 600, 900
    pos = torch.rand((B, hkv, seen), generator=gen(1), device="cuda").argsort(-1)[..., :L].int().contiguous()
    for widths in (((128, BF16), (128, BF16), (256, BF16)), ((144, torch.uint8),), ((80, torch.uint8),)):
        for inplace in (False, True):
            run_evict(B, hkv, L, 200, [600, 350], sinks=5, recent=100, weights=spread((B, hkv, L), 710),
                      positions=pos.clone(), nxt=[seen, seen - 100], widths=widths, inplace=inplace, layout=layout)


@pytest.mark.parametrize("kind", ["zeros", "equal", "two", "nan", "inf", "negative", "subnormal", "close"])
def test_evict_weights_that_tie_or_are_not_numbers(kind):
    B, hkv, L = 1, 2, 3000
    w = spread((B, hkv, L), 720, ties=False)
    r = torch.rand((B, hkv, L), generator=gen(721), device="cuda")
    if kind == "zeros":
        w = torch.where(r < 0.5, 0.0, -0.0)  # one value, of either sign
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "two":
        w = torch.where(r < 0.5, 1.0, 2.0)
    elif kind == "nan":
        w = torch.where(r < 0.2, float("nan"), w)
    elif kind == "inf":
        w = torch.where(r < 0.2, float("inf"), torch.where(r > 0.9, float("-inf"), w))
    elif kind == "negative":
        w = w * torch.where(r < 0.5, -1.0, 1.0)
    elif kind == "subnormal":
        w = w * 1e-40
    elif kind == "close":
        w = 1.0 + (r * 64).floor() * 2.0 ** -23
    for keep in (1, 777, 2999):
        run_evict(B, hkv, L, keep, [L], sinks=1 if keep > 1 else 0, weights=w.clone(), seed=keep)


@pytest.mark.parametrize("kind", ["equal", "two", "few"])
def test_evict_ties_across_a_cluster(kind):
    """Slots that tie spread over the slices of one head's cluster: the lowest
    of them stay, whichever slice holds them."""
    L = 70_001
    r = torch.rand((1, 2, L), generator=gen(722), device="cuda")
    w = {"equal": torch.full_like(r, 3.0), "two": torch.where(r < 0.5, 1.0, 2.0), "few": (r * 5).floor()}[kind]
    for keep in (1, 9_000, 35_123, 70_000):
        run_evict(1, 2, L, keep, [L], sinks=min(keep, 3), recent=min(keep // 2, 500), weights=w.clone(),
                  widths=((8, BF16),), seed=keep)


@pytest.mark.parametrize("seed", range(24))
def test_evict_swept(seed):
    r = np.random.default_rng(9500 + seed)
    B, hkv, L = int(r.integers(1, 5)), int(r.choice([1, 2, 3, 8])), int(np.exp(r.uniform(0, np.log(12_000))))
    keep = int(r.integers(1, L + 3))
    sinks = int(r.integers(0, min(keep, 6) + 1))
    recent = int(r.integers(0, keep - sinks + 1))
    lens = [int(x) for x in r.integers(0, L + 1, B)]
    w = spread((B, hkv, L), 9600 + seed)
    if r.random() < 0.3:
        w = w.floor()
    positions = nxt = None
    if r.random() < 0.5:
        seen = L + int(r.integers(0, 50))
        positions = torch.rand((B, hkv, seen), generator=gen(seed), device="cuda").argsort(-1)[..., :L].int().contiguous()
        nxt = [seen - int(x) for x in r.integers(0, 10, B)]
    kinds = [((64, BF16),), ((64, BF16), (64, BF16)), ((80, torch.uint8),), ((8, torch.float32), (16, BF16), (144, torch.uint8))]
    run_evict(B, hkv, L, keep, lens, sinks=sinks, recent=recent, weights=w, positions=positions, nxt=nxt,
              widths=kinds[int(r.integers(0, 4))], inplace=bool(r.random() < 0.5), layout=str(r.choice(["head", "token"])),
              seed=seed)


def test_weighted_decode_and_eviction_in_a_graph():
    """A decode over bf16 caches that gathers weights, with the gate from x, and
    the eviction that follows, captured together and replayed on new inputs."""
    t = synth.decode_inputs(2, 600, 4, 2, 128, 256, seed=790, device="cuda")
    k0, v0 = t["k_cache"].clone(), t["v_cache"].clone()
    w, sl = torch.zeros((2, 2, 600), device="cuda"), torch.tensor([600, 450], dtype=torch.int32, device="cuda")
    wo, po, so = torch.zeros_like(w), torch.zeros((2, 2, 600), dtype=torch.int32, device="cuda"), torch.zeros_like(sl)
    ws = torch.empty((max(bd.diffattn_v2_decode_weighted_workspace_size(2, 4, 2, 128, 600),
                          bd.diffattn_kv_evict_workspace_size(2, 2, 600, 200)),), dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 4, 128), dtype=BF16, device="cuda")

    def step():
        bd.diffattn_v2_decode_weighted(t["q"], t["k_cache"], t["v_cache"], seqlens=sl, x=t["x"], w_lambda=t["w_lambda"],
                                       weights_out=w, out=out, workspace=ws)
        bd.diffattn_kv_evict([t["k_cache"], t["v_cache"]], w, 200, sinks=4, recent=32, seqlens=sl, weights_out=wo,
                             positions_out=po, seqlens_out=so, workspace=ws)

    def restore():
        t["k_cache"].copy_(k0)
        t["v_cache"].copy_(v0)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (791, 792):
        t["q"].copy_(randn((2, 8, 128), gen(seed)))
        restore()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, w, wo, po, so, t["k_cache"], t["v_cache"])]
        restore()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, w, wo, po, so, t["k_cache"], t["v_cache"])))
        for b, n in enumerate((600, 450)):
            for i in range(2):
                m, src = kvo.evict(w[b, i, :n].cpu().numpy(), 200, sinks=4, recent=32)
                assert po[b, i, :m].tolist() == src and torch.equal(t["k_cache"][b, :m, i], k0[b, src, i])


def test_evict_without_positions_or_lengths():
    w = spread((1, 2, 64), 730)
    rows = [randn((1, 64, 2, 64), gen(731))]
    r = bd.diffattn_kv_evict(rows, w.clone(), 16)
    assert r["positions"] is None and r["seqlens"].tolist() == [16]


def test_evict_more_protected_than_kept_stays_in_bounds():
    """Positions that repeat (a caller's mistake) can protect more slots than
    are kept: the lowest of them stay."""
    pos = torch.zeros((1, 1, 50), dtype=torch.int32, device="cuda")
    run_evict(1, 1, 50, 10, [50], sinks=1, weights=spread((1, 1, 50), 740), positions=pos)


def test_evict_bad_length_is_recorded_and_left():
    rows = [randn((3, 32, 1, 64), gen(750))]
    before = rows[0].clone()
    w = spread((3, 1, 32), 751)
    w0 = w.clone()
    sl = torch.tensor([-1, 33, 32], dtype=torch.int32, device="cuda")
    r = bd.diffattn_kv_evict(rows, w, 8, seqlens=sl, seqlens_out=torch.zeros_like(sl))
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    assert r["seqlens"].tolist() == [-1, 33, 8]
    assert torch.equal(rows[0][:2], before[:2]) and torch.equal(w[:2], w0[:2])


def test_evict_many_heads_in_place():
    """Heads enough for every SM, lengths updated where the other heads of a
    sequence read them; rows of several kinds."""
    B, hkv = 44, 8
    for L, widths in ((97, ((80, torch.uint8),)), (2500, ((64, BF16), (16, BF16)))):
        lens = [int(x) for x in np.random.default_rng(L).integers(0, L + 1, B)]
        pos = torch.rand((B, hkv, L + 9), generator=gen(L), device="cuda").argsort(-1)[..., :L].int().contiguous()
        run_evict(B, hkv, L, L // 2 + 1, lens, sinks=2, recent=L // 9, weights=spread((B, hkv, L), 761), positions=pos,
                  nxt=[L + 9] * B, widths=widths, inplace=True, layout="token")


@pytest.mark.parametrize("more", [-1, 0, 1])
@pytest.mark.parametrize("L,keep,widths", [(1000, 900, ((128, BF16), (256, BF16))), (6200, 6000, ((16, BF16),)),
                                           (8192, 4096, ((8, BF16),)), (8193, 4097, ((8, BF16),))])
def test_evict_as_many_heads_as_sms(more, L, keep, widths):
    """One head per SM, one more, one fewer: rows moved by the head's own block
    or by a launch of their own."""
    B = torch.cuda.get_device_properties(0).multi_processor_count + more
    lens = [L - (b % 5) * (L // 6) for b in range(B)]
    run_evict(B, 1, L, keep, lens, sinks=4, recent=50, weights=spread((B, 1, L), 765), widths=widths, inplace=True)


@pytest.mark.parametrize("keep", [99, 100, 350])
@pytest.mark.parametrize("inplace", [False, True])
def test_evict_few_heads_with_few_and_many_rows(keep, inplace):
    """Three heads whose rows to move are just below and above what their own
    blocks take; several sequences with the lengths updated in place."""
    B, hkv, L = 3, 2, 700
    pos = torch.rand((B, hkv, 900), generator=gen(5), device="cuda").argsort(-1)[..., :L].int().contiguous()
    run_evict(B, hkv, L, keep, [700, 351, 90], sinks=3, recent=20, weights=spread((B, hkv, L), 766), positions=pos,
              nxt=[900] * B, widths=((256, BF16), (256, BF16), (512, BF16)), inplace=inplace)


@pytest.mark.parametrize("B,hkv,L,keep", [(2, 2, 700, 400), (40, 8, 130, 60), (23, 7, 300, 250), (18, 9, 300, 250),
                                          (160, 1, 97, 40), (3, 1, 5000, 2500), (70, 2, 3001, 2900)])
@pytest.mark.parametrize("out", ["lengths", "next", "both", "apart"])
def test_evict_lengths_that_others_read(B, hkv, L, keep, out):
    """New lengths written over the array that every head of the sequence reads
    its length or its newest position from."""
    lens = [max(1, L - (i * 37) % L) for i in range(B)]
    w = spread((B, hkv, L), 768)
    rows = [randn((B, L, hkv, 8), gen(6))]
    raw = rows[0].cpu().view(torch.uint8).numpy().copy()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    nxt = sl if out == "both" else sl + 5
    pos = (torch.arange(L, dtype=torch.int32, device="cuda") + (0 if out == "both" else 5)).expand(B, hkv, L).contiguous()
    so = {"lengths": sl, "both": sl, "next": nxt, "apart": torch.full_like(sl, -9)}[out]
    w_np, p_np, n_np = w.cpu().numpy().copy(), pos.cpu().numpy().copy(), nxt.tolist()
    r = bd.diffattn_kv_evict(rows, w, keep, sinks=0, recent=20, seqlens=sl, positions=pos, next_position=nxt,
                             seqlens_out=so)
    assert so.tolist() == [min(n, keep) for n in lens]
    got = rows[0].cpu().view(torch.uint8).numpy()
    for b in range(B):
        for h in range(hkv):
            m, source = kvo.evict(w_np[b, h, :lens[b]], keep, sinks=0, recent=20, positions=p_np[b, h, :lens[b]],
                                  next_position=n_np[b])
            assert np.array_equal(r["positions"][b, h, :m].cpu().numpy(), p_np[b, h, source])
            assert np.array_equal(got[b, :m, h], raw[b, source, h])


def test_evict_many_heads():
    B, hkv, L = 40, 8, 130
    lens = [int(x) for x in np.random.default_rng(9).integers(0, L + 1, B)]
    run_evict(B, hkv, L, 60, lens, sinks=2, recent=20, weights=spread((B, hkv, L), 760), widths=((80, torch.uint8),))


def test_evict_more_slots_than_shared_memory_holds():
    """Half a million slots of one head: each CTA of the cluster keeps the
    first 49152 ranks of its slice and reads the others again."""
    L = 500_001
    for keep, ties in ((200_000, True), (499_000, False)):
        run_evict(1, 1, L, keep, [L], sinks=4, recent=1000, weights=spread((1, 1, L), 780, ties), widths=((8, BF16),))


def test_evict_does_not_change_what_a_decode_over_the_kept_keys_gives():
    """A decode over the compacted cache equals one over the kept keys in their
    own order, up to the order of fp32 sums."""
    B, L, h, hkv, d, keep = 1, 900, 4, 2, 128, 300
    g, cache, q, gate, sl = make(B, L, h, hkv, d, [L], 770)
    w = torch.zeros((B, hkv, L), device="cuda")
    bd.diffattn_v2_decode_kv4(q, cache, gate=gate, weights_out=w)
    kept = [sorted(kvo.evict(w[0, i].cpu().numpy(), keep)[1]) for i in range(hkv)]
    apart = torch.stack([cache[0, kept[i], i] for i in range(hkv)], 1)[None].contiguous()
    r = bd.diffattn_kv_evict([cache], w, keep, seqlens=sl)
    a = bd.diffattn_v2_decode_kv4(q, cache, seqlens=r["seqlens"], gate=gate)
    kf, vf, rk, rv = ranges(apart.cpu().numpy())
    check_decode(q, kf, vf, rk, rv, [keep], f64(gate), a)


# -------------------------------------------------- as a serving loop -------
def test_serving_loop_against_the_definitions():
    """Prompts appended, decode steps that gather weights, the cache cut to its
    budget whenever it is full, tokens appended into the freed slots: every
    step against the fp64 definitions run on their own bookkeeping."""
    B, hkv, h, d, cap, keep, sinks, recent, steps = 2, 2, 4, 128, 96, 64, 2, 16, 50
    g = gen(800)
    lens = [90, 40]
    cache = new_cache(B, cap, hkv, d)
    w = torch.full((B, hkv, cap), 123.0, device="cuda")
    pos = torch.full((B, hkv, cap), -1, dtype=torch.int32, device="cuda")
    k, v = randn((B, 90, hkv, d), g), randn((B, 90, hkv, d), g)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    bd.diffattn_kv4_append(k, v, cache, counts=sl, key_weights=w, positions=pos)
    nxt = sl.clone()
    ref_w = [np.zeros((hkv, n)) for n in lens]
    ref_p = [np.tile(np.arange(n), (hkv, 1)) for n in lens]
    err = np.zeros(B)  # what the gathered weights may be off by now
    evictions = 0
    for step in range(steps):
        if int(sl.max()) == cap:
            w_np = w.cpu().numpy()
            r = bd.diffattn_kv_evict([cache], w, keep, sinks=sinks, recent=recent, seqlens=sl, positions=pos,
                                     next_position=nxt)
            evictions += 1
            for b in range(B):
                n = ref_w[b].shape[1]
                src = [kvo.evict(w_np[b, i, :n], keep, sinks=sinks, recent=recent, positions=ref_p[b][i],
                                 next_position=int(nxt[b]))[1] for i in range(hkv)]
                ref_w[b] = np.stack([ref_w[b][i, src[i]] for i in range(hkv)])
                ref_p[b] = np.stack([ref_p[b][i, src[i]] for i in range(hkv)])
            assert r["seqlens"] is sl and sl.tolist() == [x.shape[1] for x in ref_w]
        kn, vn, q = randn((B, 1, hkv, d), g), randn((B, 1, hkv, d), g), randn((B, 2 * h, d), g)
        gate = torch.rand((B, h), generator=g, device="cuda")
        bd.diffattn_kv4_append(kn, vn, cache, start=sl, key_weights=w, positions=pos, first_position=nxt)
        sl += 1
        nxt += 1
        before = w.clone()
        out = bd.diffattn_v2_decode_kv4(q, cache, seqlens=sl, gate=gate, weights_in=w, weights_out=w)
        n = sl.tolist()
        rec = clean(cache, n)
        kf, vf, rk, rv = ranges(rec)
        check_decode(q, kf, vf, rk, rv, n, f64(gate), out, w, before, before)
        for b in range(B):
            ref_p[b] = np.concatenate([ref_p[b], np.full((hkv, 1), int(nxt[b]) - 1)], 1)
            assert np.array_equal(pos[b, :, :n[b]].cpu().numpy(), ref_p[b])
            dw, total = kvo.key_weights(f64(q[b]), kf[b, :n[b]], f64(gate[b]))
            ref_w[b] = np.concatenate([ref_w[b], np.zeros((hkv, 1))], 1) + dw
            err[b] += 1e-4 * total.max()
            assert np.max(np.abs(f64(w[b, :, :n[b]]) - ref_w[b])) <= err[b]
    assert evictions >= 1
