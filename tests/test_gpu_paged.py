"""V2 attention of new tokens over a paged cache on the GPU, against the 64-bit
definition.

Bars (u = 2^-24): the scores carry fp32 accumulation over the features, e = 64 u
(1 + scale sum_f |q_f| |k_f|) at most, which moves every weight A by A e (twice:
the sum too); the weights reach the value product as bf16 (2^-8 relative); the
rest of the arithmetic is fp32 (2^-16 for the exponentials, joined parts and
sums); the output is rounded to bf16 (2^-8).  So an output is within
(2^-8 + 2^-16 + 2 e) (sum A_2p |v| + gate sum A_2p+1 |v|) + 2^-8 |out|."""

import numpy as np
import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from oracle import paged_oracle as po
from ratio_log import record

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert bd.diffattn_get_device_status() == bd.DA_OK


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(n, L, page, h, hkv, d, layout="token", extra=0, seed=0, std=1.0, max_pages=None):
    """A batch with n[b] new tokens of L[b] cached ones; what no position of a sequence lives in holds NaN."""
    g = gen(seed + sum(L) + 7 * len(n))
    B, T = len(n), sum(n) + extra
    P = max_pages or max(1, -(-max(L) // page))
    count = B * P + 2
    table = torch.randperm(count, generator=g, device="cuda")[:B * P].reshape(B, P)
    shape = (count, hkv, page, d) if layout == "head" else (count, page, hkv, d)
    pages = []
    for _ in range(2):
        t = torch.full(shape, float("nan"), dtype=BF16, device="cuda")
        t = t.transpose(1, 2) if layout == "head" else t
        for b in range(B):
            j = torch.arange(L[b], device="cuda")
            t[table[b, j // page], j % page] = randn((L[b], hkv, d), g, std)
        pages.append(t)
    table = table.int()
    for b in range(B):  # entries behind the length are not looked at
        table[b, -(-L[b] // page):] = -12345
    q = randn((T, 2 * h, d), g, std)
    gate = torch.rand((T, h), generator=g, device="cuda")
    return dict(q=q, k=pages[0], v=pages[1], table=table, cu=i32(np.cumsum([0] + n)), sl=i32(L), gate=gate, n=n, L=L)


def call(t, **kw):
    kw.setdefault("gate", t["gate"] if "x" not in kw else None)
    return bd.diffattn_v2_paged_fwd(t["q"], t["k"], t["v"], t["table"], t["cu"], t["sl"], **kw)


def check(t, out, gate=None, scale=None, only=None, tag=""):
    gate = f64(t["gate"]) if gate is None else gate
    q, table, worst = f64(t["q"]), t["table"].cpu().numpy(), 0.0
    d = q.shape[-1]
    s = d ** -0.5 if scale is None else scale
    t0 = 0
    for b, (n, L) in enumerate(zip(t["n"], t["L"])):
        if n and (only is None or b in only):
            used = t["table"][b, :-(-L // t["k"].shape[1])].long()
            k, v = (f64(t[x][used].flatten(0, 1)[:L]) for x in ("k", "v"))
            ref, size = po.attend(q[t0:t0 + n], k, v, gate[t0:t0 + n], np.arange(L - n, L) + 1, s, sizes=True)
            most = np.abs(k).max(0)  # per KV head and feature
            G = q.shape[1] // k.shape[1]
            e = 64 * U * (1 + s * (np.abs(q[t0:t0 + n]) * np.repeat(most, G, 0)).sum(-1))  # [n, 2h]
            e = np.maximum(e[:, 0::2], e[:, 1::2])[..., None]
            bar = (2.0 ** -8 + 2.0 ** -16 + 2 * e) * size + 2.0 ** -8 * np.abs(ref) + 1e-30
            err = np.abs(f64(out[t0:t0 + n]) - ref)
            assert not np.isnan(err).any(), (b, np.argwhere(np.isnan(err))[:4])
            worst = max(worst, (err / bar).max())
            assert (err <= bar).all(), (b, (err / bar).max(), np.argwhere(err > bar)[:4])
        t0 += n
    record({"out": worst}, tag)


CASES = [  # counts, lengths, page, h, h_kv, d, layout, extra rows
    ([1], [1], 16, 2, 1, 128, "token", 0),
    ([1], [1000], 16, 32, 8, 128, "token", 0),
    ([1, 1, 1, 1], [5, 128, 129, 700], 32, 4, 2, 64, "head", 3),
    ([1, 0, 1], [1, 0, 257], 16, 8, 1, 128, "token", 0),
    ([4, 4, 4], [4, 300, 513], 16, 8, 2, 64, "token", 1),
    ([3, 1], [130, 4000], 64, 6, 2, 128, "head", 0),
    ([200], [200], 128, 4, 1, 128, "head", 0),
    ([129, 1, 64], [129, 900, 1500], 48, 4, 2, 64, "token", 5),
    ([300, 17], [1100, 17], 256, 3, 1, 128, "token", 0),  # 6 heads per KV head
    ([77], [400], 16, 12, 2, 64, "head", 0),              # 12
    ([90, 2, 0], [333, 222, 111], 16, 10, 2, 128, "token", 2),  # 10
    ([40, 1], [41, 260], 32, 64, 1, 128, "token", 0),     # 128: one token to a tile
    ([50], [60], 16, 2, 2, 128, "token", 0),              # 2: 64 tokens to a tile
    ([1] * 40, list(range(1, 2000, 50)), 16, 4, 2, 128, "token", 0),
]


@pytest.mark.parametrize("max_new", [0, 1])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0][:4]}-{c[1][:4]}-p{c[2]}-{c[3]}-{c[4]}-{c[5]}-{c[6]}")
def test_parity(case, max_new):
    """Whatever the number of new tokens is said to be, the result is right."""
    t = make(*case)
    out = torch.full((t["q"].shape[0], case[3], case[5]), 7.0, dtype=BF16, device="cuda")
    call(t, out=out, max_new=max_new)
    check(t, out)
    assert bool((out[sum(t["n"]):] == 7).all())
    again = torch.zeros_like(out)
    call(t, out=again, max_new=max_new)
    assert torch.equal(again[:sum(t["n"])], out[:sum(t["n"])])


def test_swept_shapes():
    rng = np.random.default_rng(11)
    for i in range(24):
        B = int(rng.integers(1, 7))
        L = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), B)).astype(int)]
        mode = i % 3
        n = [1 if mode == 0 else int(rng.integers(0, min(x, 5 if mode == 1 else 400) + 1)) for x in L]
        if sum(n) == 0:
            n[0] = 1
        d, hkv = int(rng.choice([64, 128])), int(rng.choice([1, 2, 3]))
        G = int(rng.choice([2, 4, 6, 8, 10, 14, 16, 24]))
        t = make(n, L, int(rng.choice([16, 32, 48, 64, 112, 128, 256])), hkv * G // 2, hkv, d,
                 str(rng.choice(["token", "head"])), extra=int(rng.integers(0, 3)), seed=i, std=float(rng.choice([1.0, 3.0])))
        scale = float(rng.choice([0.0, 0.05, 0.2]))
        out = call(t, max_new=int(rng.choice([0, 1, max(n)])), softmax_scale=scale)
        check(t, out, scale=scale or None, tag=str(i))


@pytest.mark.parametrize("max_new", [2, 0])
def test_more_sequences_than_threads(max_new):
    rng = np.random.default_rng(5)
    L = [int(x) for x in rng.integers(0, 300, 700)]
    n = [min(x, int(rng.integers(0, 3))) for x in L]
    n[650], L[650] = 70, 270
    t = make(n, L, 16, 2, 1, 64)
    check(t, call(t, max_new=max_new))


def test_turns_of_the_shares():
    """Keys that do not fit L2, read for many items: the CTAs take several shares each, whose parts are joined."""
    t = make([260, 150, 300], [9000, 12000, 10000], 128, 16, 8, 128, layout="head", seed=4)
    P = 400  # room for 51200 positions a sequence: 3.7 GB of keys and values at most
    table = torch.full((3, P), -1, dtype=torch.int32, device="cuda")
    table[:, :t["table"].shape[1]] = t["table"]
    t["table"] = table
    out = call(t)
    t0 = 0
    for n, L in zip(t["n"], t["L"]):  # one sequence by itself, its first and last tokens
        one = dict(t, q=t["q"][t0:t0 + n], gate=t["gate"][t0:t0 + n], n=[n], L=[L], cu=i32([0, n]), sl=i32([L]),
                   table=t["table"][t["L"].index(L)][None].contiguous())
        alone = call(one)
        assert float((alone.float() - out[t0:t0 + n].float()).abs().max()) <= 2.0 ** -6 * float(alone.float().abs().max())
        few = [0, 1, n // 2, n - 1]
        k, v = (f64(one[x][one["table"][0, :-(-L // 128)].long()].flatten(0, 1)[:L]) for x in ("k", "v"))
        ref, size = po.attend(f64(one["q"][few]), k, v, f64(one["gate"][few]), np.array(few) + L - n + 1, sizes=True)
        got = f64(out[t0:t0 + n][few])
        assert np.all(np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * np.abs(ref))
        t0 += n


def test_scores_that_grow():
    """Scores far above the first tile's: the running maximum is raised, O rescaled; and the reverse."""
    for n, L in (([1], [1500]), ([300], [1500]), ([60], [1500])):
        for up in (True, False):
            t = make(n, L, 64, 4, 1, 128, seed=3)
            ramp = torch.linspace(0.0, 40.0, L[0], device="cuda")
            ramp = ramp if up else ramp.flip(0)
            for j in range(L[0]):
                p, s = int(t["table"][0, j // 64]), j % 64
                t["k"][p, s] = t["k"][p, s] * ramp[j].item()
            check(t, call(t), tag=str((n, up)))


def test_partial_last_tiles_call_after_call():
    """Many sequences of few tokens, each with a last tile that ends inside a page, on the kernel for chunks: the stage
    whose values are zeroed behind the end may hold nothing of the tile before, whatever the copies' order."""
    for n, L, h, hkv, page in (([1, 9, 3, 15, 5, 12, 1, 2] * 5, list(range(1203, 9203, 200)), 16, 8, 256),
                               ([1, 2, 3, 1] * 8, list(range(333, 8333, 250)), 64, 4, 128)):
        t = make(n, L, page, h, hkv, 128, layout="head")
        out = call(t, max_new=1000)
        check(t, out, only=(0, 7, 20, len(n) - 1))
        other = torch.randn(1 << 25, device="cuda")
        for i in range(150):
            if i % 3 == 0:
                other.add_(1.0)  # the caches' contents differ from call to call
            assert torch.equal(call(t, max_new=1000), out), i


def test_equal_heads_cancel():
    """Heads 2p and 2p + 1 alike and gate 1: exactly nothing is left, whole or joined."""
    for n, L in (([1], [5000]), ([200], [900]), ([1] * 30, [300] * 30)):
        t = make(n, L, 32, 4, 2, 128)
        t["q"][:, 1::2] = t["q"][:, 0::2]
        t["gate"].fill_(1.0)
        assert not call(t).any()


def test_gate_from_x_and_strided_views():
    g = gen(4)
    for n, L in (([1, 1, 1], [50, 600, 77]), ([200, 1, 37], [300, 600, 37])):
        t = make(n, L, 16, 6, 2, 64, seed=1)
        T = sum(n)
        x, w = randn((T, 256), g), randn((256, 6), g, 0.05)
        gate = 1 / (1 + np.exp(-(f64(x) @ f64(w))))
        big = torch.full((T, 20, 64), float("nan"), dtype=BF16, device="cuda")
        big[:, 4:16] = t["q"]
        t["q"] = big[:, 4:16]
        res = torch.full((T, 8, 128), 7.0, dtype=BF16, device="cuda")
        out = res[:, 1:7, :64]
        call(t, x=x, w_lambda=w, out=out)
        check(t, out, gate=gate)
        assert bool((res[:, [0, 7]] == 7).all()) and bool((res[..., 64:] == 7).all())


def test_shared_pages():
    """Two sequences over the same pages of a prefix."""
    t = make([1, 1, 40], [200, 130, 190], 16, 4, 2, 128)
    t["table"][1, :8] = t["table"][0, :8]
    t["table"][2, :8] = t["table"][0, :8]
    check(t, call(t))


@pytest.mark.parametrize("n", [1, 70])
def test_far_pages(n):
    """Pages that lie more than 2^32 elements and bytes behind the first."""
    page, hkv, d = 64, 8, 128
    count = 2 ** 32 // (page * hkv * d) + 5  # 8.6 GB each of K and V
    t = make([n], [200], page, 16, hkv, d)
    far = torch.tensor([count - 1, 3, count - 4, count - 2], device="cuda")
    pages = []
    for x in ("k", "v"):
        big = torch.empty((count, page, hkv, d), dtype=BF16, device="cuda")
        big[far] = t[x][t["table"][0].long()]
        pages.append(big)
    near = call(t)
    t.update(k=pages[0], v=pages[1], table=far.int()[None])
    assert torch.equal(call(t), near)
    check(t, near)
    # and appended to
    k, v = randn((n, hkv, d), gen(1)), randn((n, hkv, d), gen(2))
    bd.diffattn_paged_append(k, v, *pages, t["table"], t["cu"], t["sl"], None)
    j = torch.arange(200 - n, 200, device="cuda")
    assert torch.equal(pages[0][far[j // page], j % page], k) and torch.equal(pages[1][far[j // page], j % page], v)


@pytest.mark.parametrize("n", [[1, 1, 1], [100, 70, 90]])
@pytest.mark.parametrize("what", ["short", "long", "rows", "below"])
def test_sequence_out_of_bounds(what, n):
    t = make(n, [200, 150, 300], 16, 4, 2, 128, max_pages=20)
    cu, sl = t["cu"].tolist(), t["sl"].tolist()
    bad = 1
    if what == "short":
        sl[1] = n[1] - 1
    elif what == "long":
        sl[1] = 321
    elif what == "rows":
        cu[3] += 1
        bad = 2
    else:
        cu[0], bad = -1, 0
    t["cu"], t["sl"] = i32(cu), i32(sl)
    out = torch.full((sum(n), 4, 128), 7.0, dtype=BF16, device="cuda")
    call(t, out=out)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    check(t, out, only=[b for b in range(3) if b != bad])
    t0 = sum(n[:bad])
    assert not out[t0:t0 + n[bad]].any()


@pytest.mark.parametrize("n", [1, 90])
def test_page_out_of_bounds(n):
    """Its keys and values are zeros, and the status word says so."""
    t = make([n, 1], [200, 50], 16, 4, 2, 128)
    pages = t["k"].shape[0]
    for bad in (-1, pages, 2 ** 31 - 1):
        t["table"][0, 3] = bad
        out = call(t)
        assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
        k, v = (po.gather(f64(t[x]), t["table"][0].tolist(), 200) for x in ("k", "v"))
        ref, size = po.attend(f64(t["q"][:n]), k, v, f64(t["gate"][:n]), np.arange(200 - n, 200) + 1, sizes=True)
        assert np.all(np.abs(f64(out[:n]) - ref) <= (2.0 ** -8 + 2.0 ** -10) * size + 2.0 ** -8 * np.abs(ref))
        check(t, out, only=[1])


def test_nan_query_and_key_reach_what_they_may():
    """A NaN query makes its pair's output NaN and no other; a NaN key every token that sees it."""
    for n in (1, 100):
        t = make([n, n], [300, 300], 16, 4, 2, 128)
        t["q"][n - 1, 0] = float("nan")
        out = call(t)
        nan = torch.isnan(out).any(-1)
        assert bool(nan[n - 1, 0]) and int(nan.sum()) == 1
        t = make([n, n], [300, 300], 16, 4, 2, 128, seed=2)
        t["k"][int(t["table"][0, 299 // 16]), 299 % 16, 0] = float("nan")  # the last token's own key
        nan = torch.isnan(call(t)).any(-1)
        assert bool(nan[n - 1, :2].all()) and int(nan.sum()) == 2


def test_graph_and_streams():
    """Captured and replayed after the inputs changed; two calls on two streams at once, each with its workspace."""
    t, o = make([1, 30, 1], [700, 200, 90], 16, 8, 2, 128), make([90], [400], 16, 8, 2, 128, seed=5)
    out = torch.zeros((32, 8, 128), dtype=BF16, device="cuda")
    ws = torch.empty(bd.diffattn_v2_paged_fwd_workspace_size(32, 3, 30, 8, 2, 128, gate_given=True), dtype=torch.uint8, device="cuda")
    call(t, out=out, workspace=ws, max_new=30)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(t, out=out, workspace=ws, max_new=30)
    t["q"].copy_(randn(t["q"].shape, gen(8)))
    t["sl"].copy_(i32([650, 150, 1]))
    t["L"] = [650, 150, 1]
    graph.replay()
    check(t, out)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    res = [[call(x, stream=s) for _ in range(5)] for x, s in zip((t, o), streams)]
    torch.cuda.synchronize()
    for x, r in zip((t, o), res):
        check(x, r[0])
        assert all(torch.equal(r[0], y) for y in r)


@pytest.mark.parametrize("n", [[1, 1, 2], [150, 1, 40]])
def test_graph_with_the_gate_from_x(n):
    """The gate's kernel, the attention that starts beside it and the join, captured and replayed after x changed; and
    a step of append and attention."""
    t = make(n, [200, 700, 333], 32, 8, 2, 64, seed=9)
    g, T = gen(10), sum(n)
    x, w = randn((T, 512), g), randn((512, 8), g, 0.05)
    k, v, q = randn((T, 2, 64), g), randn((T, 2, 64), g), randn((T, 16, 64), g)
    f, _ = bd.diffattn_rope_inv_freq(64)
    out = torch.zeros((T, 8, 64), dtype=BF16, device="cuda")
    ws = torch.empty(bd.diffattn_v2_paged_fwd_workspace_size(T, 3, max(n), 8, 2, 64), dtype=torch.uint8, device="cuda")

    def step():
        bd.diffattn_paged_append(k, v, t["k"], t["v"], t["table"], t["cu"], t["sl"], f, q=q, q_out=t["q"])
        call(t, x=x, w_lambda=w, out=out, workspace=ws, max_new=max(n))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x.copy_(randn(x.shape, g))
        k.copy_(randn(k.shape, g))
        graph.replay()
        check(t, out, gate=1 / (1 + np.exp(-(f64(x) @ f64(w)))))


def test_serving_steps():
    """A run as a serving loop makes it: prompts in chunks, then single tokens, each appended (normed, rotated) and
    attended; against the definition over everything that was appended."""
    g = gen(6)
    h, hkv, d, page = 4, 2, 128, 16
    P, count = 20, 50
    kp, vp = (torch.full((count, page, hkv, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.randperm(count, generator=g, device="cuda")[:2 * P].reshape(2, P).int()
    f, scale = bd.diffattn_rope_inv_freq(d, stretch="ramp", factor=4.0, trained_len=64)
    w = 1 + torch.rand(d, generator=g, device="cuda")
    L = [0, 0]
    for n in ([150, 37], [100, 1], [1, 1], [1, 60], [1, 1]):
        T = sum(n)
        L = [a + b for a, b in zip(L, n)]
        cu, sl = i32(np.cumsum([0] + n)), i32(L)
        x = randn((T, 2 * h + 2 * hkv, d), g)
        q = bd.diffattn_paged_append(x[:, 2 * h:2 * h + hkv], x[:, 2 * h + hkv:], kp, vp, table, cu, sl, f,
                                     q=x[:, :2 * h], rope_scale=scale, norm=True, q_weight=w, k_weight=w)
        t = dict(q=q, k=kp, v=vp, table=table, cu=cu, sl=sl, gate=torch.rand((T, h), generator=g, device="cuda"), n=n, L=L)
        check(t, call(t, max_new=max(n)))
        pos = np.concatenate([np.arange(b - a, b) for a, b in zip(n, L)])
        exp = po.qk_rope(f64(x[:, :2 * h]), f64(f), pos, d, False, scale, True, 1e-5, f64(w))
        assert np.all(np.abs(f64(q) - exp) <= 2.0 ** -8 * np.abs(exp) * 1.01 + 1e-4)


def test_matches_the_contiguous_decode_and_forward():
    """Pages in a row are a contiguous cache: the V2 decode and forward give the same within both bars."""
    B, L, h, hkv, d = 3, 512, 8, 2, 128
    t = make([1] * B, [L] * B, 64, h, hkv, d)
    k, v = (t[x][t["table"].long()].flatten(1, 2).contiguous() for x in ("k", "v"))
    a, b = call(t), bd.diffattn_v2_decode(t["q"], k, v, gate=t["gate"])
    assert float((a.float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.float().abs().max())
    t = make([L] * B, [L] * B, 64, h, hkv, d)
    k, v = (t[x][t["table"].long()].flatten(1, 2).contiguous() for x in ("k", "v"))
    a = call(t).reshape(B, L, h, d)
    b = bd.diffattn_v2_fwd(t["q"].reshape(B, L, 2 * h, d), k, v, gate=t["gate"].reshape(B, L, h))
    assert float((a.float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.float().abs().max())
