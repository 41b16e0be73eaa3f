"""Norm and rotation of queries and keys on the GPU, forward and backward, and the
append of new tokens to a paged cache.

Bars (u = 2^-24, half an fp32 step; h = half a step of the output's type):
- z: the sum of d squares in fp32 (8 in a row, then a tree of at most 4), rsqrt
  (2 steps) and two products: within 32 u;
- cos, sin: the angle within 2 u, sincospi 2 steps, the scale: within 8 u;
- so y is within 2^-19 scale (|z_u| + |z_v|), then h |y|;
- dz likewise from dy; dx = r (g - xh m) within 2^-18 r (A + |xh| mean(A |xh|)) for
  A = |w| scale (|dy_u| + |dy_v|), then h |dx|;
- dw: 2^-18 sum A' |xh| over the rows, A' = A without w: a lane adds up few rows."""

import numpy as np
import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from oracle import paged_oracle as po

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, g, dtype=BF16, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert bd.diffattn_get_device_status() == bd.DA_OK


def pair_sum(a, rot, interleaved):
    """|a_u| + |a_v| of each feature's pair, |a| behind rot."""
    y = np.abs(a)
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    s = y[..., u] + y[..., v]
    y[..., u], y[..., v] = s, s
    return y


def check_fwd(y, x, f, pos, kw, w):
    rot, inter, scale = kw["rot_dim"], kw["interleaved"], kw["rope_scale"]
    x = f64(x)
    ref = po.qk_rope(x, f64(f), pos, rot, inter, scale, kw["norm"], kw["norm_eps"], w)
    z = po.norm(x, w, kw["norm_eps"]) if kw["norm"] else x
    bar = 2.0 ** -19 * max(scale, 1) * pair_sum(z, rot, inter) + HALF[y.dtype] * np.abs(ref) * 1.001 + 1e-38
    err = np.abs(f64(y) - ref)
    assert np.all(err <= bar), (err / bar).max()


def check_bwd(dx, x, dy, f, pos, kw, w):
    rot, inter, scale = kw["rot_dim"], kw["interleaved"], kw["rope_scale"]
    x, dy = f64(x), f64(dy)
    ref, dw = po.qk_rope_bwd(x, dy, f64(f), pos, rot, inter, scale, kw["norm"], kw["norm_eps"], w)
    A = max(scale, 1) * pair_sum(dy, rot, inter)
    if kw["norm"]:
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + kw["norm_eps"])
        xh, Aw = np.abs(x * r), A if w is None else A * np.abs(w)
        bar = 2.0 ** -18 * r * (Aw + xh * (Aw * xh).mean(-1, keepdims=True))
        dw_bar = 2.0 ** -18 * (A * xh).reshape(-1, x.shape[-1]).sum(0)
    else:
        bar, dw_bar = 2.0 ** -19 * A, None
    err, bar = np.abs(f64(dx) - ref), bar + HALF[dx.dtype] * np.abs(ref) * 1.001 + 1e-38
    assert np.all(err <= bar), (err / bar).max()
    return dw, dw_bar


CASES = [  # B, N, h_q, h_k, d, rot, interleaved, norm, dtype, positions, scale, strided
    (1, 1, 64, 8, 128, 128, False, True, BF16, "far", 1.0, False),
    (2, 37, 6, 2, 128, 64, True, True, BF16, "given", 1.25, True),
    (3, 5, 3, 1, 64, 64, False, False, BF16, None, 1.0, True),
    (1, 700, 4, 4, 64, 16, True, True, F32, "far", 1.0, False),
    (2, 9, 7, 3, 32, 24, False, True, F32, "given", 1.3, True),
    (2, 3, 2, 2, 16, 16, False, True, BF16, "given", 1.0, False),
    (1, 4, 5, 2, 16, 8, True, False, F32, "far", 1.0, True),
    (2, 6, 3, 2, 128, 0, False, True, BF16, None, 1.0, False),
    (4, 1500, 8, 2, 128, 128, False, True, BF16, None, 1.0, True),
    (1, 3, 0, 5, 64, 64, False, True, BF16, "far", 1.0, False),
    (1, 3, 5, 0, 64, 64, True, True, BF16, "far", 1.0, False),
]


def make(B, N, h_q, h_k, d, rot, dtype, positions, strided, g):
    if strided:  # views of a fused projection, heads in front of tokens
        x = randn((B, h_q + h_k + 1, N, d), g, dtype, 1.5).transpose(1, 2)
        q, k = x[:, :, :h_q], x[:, :, h_q + 1:]
    else:
        q, k = randn((B, N, h_q, d), g, dtype, 1.5), randn((B, N, h_k, d), g, dtype, 1.5)
    f = torch.tensor(10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1)), dtype=F32, device="cuda")
    if positions == "far":
        p = torch.randint(900000, 2 ** 31 - 1, (B, N), generator=g, device="cuda").int()
    elif positions == "given":  # any value: below zero too
        p = torch.randint(-5000, 5000, (B, N), generator=g, device="cuda").int()
    else:
        p = None
    pos = np.broadcast_to(np.arange(N), (B, N)) if p is None else p.cpu().numpy()
    return q if h_q else None, k if h_k else None, f, p, pos


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_fwd_and_bwd(case):
    B, N, h_q, h_k, d, rot, inter, norm, dtype, positions, scale, strided = case
    g = gen(B * 1000 + N + d)
    q, k, f, p, pos = make(B, N, h_q, h_k, d, rot, dtype, positions, strided, g)
    w = [1 + randn((d,), g, F32, 0.3) for _ in range(2)] if norm else [None, None]
    wn = [None if x is None else f64(x) for x in w]
    kw = dict(rot_dim=rot, interleaved=inter, rope_scale=scale, norm=norm, norm_eps=1e-5)
    y = bd.diffattn_qk_rope_fwd(q, k, f, positions=p, q_weight=w[0], k_weight=w[1], **kw)
    dy = [None if t is None else randn(t.shape, g, dtype) for t in (q, k)]
    r = bd.diffattn_qk_rope_bwd(q, k, *dy, f, positions=p, q_weight=w[0], k_weight=w[1], **kw)
    again = bd.diffattn_qk_rope_bwd(q, k, *dy, f, positions=p, q_weight=w[0], k_weight=w[1], **kw)
    for i, (x, name) in enumerate(((q, "q"), (k, "k"))):
        if x is None:
            assert y[i] is None and r["d" + name] is None
            continue
        check_fwd(y[i], x, f, pos, kw, wn[i])
        dw, bar = check_bwd(r["d" + name], x, dy[i], f, pos, kw, wn[i])
        if norm:
            assert np.all(np.abs(f64(r[f"d{name}_weight"]) - dw) <= bar + HALF[F32] * np.abs(dw))
        for n in ("d" + name, f"d{name}_weight"):
            assert r[n] is None or torch.equal(r[n], again[n])


def test_in_place_and_unit_weights():
    """Outputs that are the inputs; a norm without weights is one with ones."""
    g = gen(7)
    q, k, f, _, pos = make(2, 33, 6, 2, 128, 128, BF16, None, True, g)
    kw = dict(norm=True, rope_scale=1.5)
    ones = torch.ones(128, device="cuda")
    exp = bd.diffattn_qk_rope_fwd(q, k, f, q_weight=ones, k_weight=ones, **kw)
    dy = [randn(t.shape, g) for t in (q, k)]
    ge = bd.diffattn_qk_rope_bwd(q, k, *dy, f, **kw)
    dx = [t.clone() for t in dy]
    gi = bd.diffattn_qk_rope_bwd(q, k, *dx, f, dq=dx[0], dk=dx[1], **kw)
    assert gi["dq"] is dx[0] and all(torch.equal(ge[n], gi[n]) for n in ge)
    got = bd.diffattn_qk_rope_fwd(q, k, f, q_out=q, k_out=k, **kw)
    assert got[0] is q and torch.equal(exp[0], q) and torch.equal(exp[1], k)


def test_rows_of_zeros_and_nan():
    """A row of zeros gives zeros (and finite gradients with norm_eps); a NaN stays within its row."""
    x = torch.ones((1, 4, 1, 64), device="cuda").to(BF16)
    x[0, 1] = 0
    x[0, 2, 0, 5] = float("nan")
    f = torch.ones(32, device="cuda")
    y, _ = bd.diffattn_qk_rope_fwd(x, None, f, norm=True)
    assert not y[0, 1].any() and torch.isnan(y[0, 2]).any() and not torch.isnan(y[0, [0, 1, 3]]).any()
    r = bd.diffattn_qk_rope_bwd(x, None, torch.ones_like(x), None, f, norm=True)
    assert torch.isnan(r["dq"][0, 2]).any() and not torch.isnan(r["dq"][0, [0, 1, 3]]).any()


def test_empty_and_refused():
    f = torch.ones(32, device="cuda")
    q = torch.zeros((2, 0, 4, 64), dtype=BF16, device="cuda")
    y, _ = bd.diffattn_qk_rope_fwd(q, None, f)
    assert y.shape == q.shape
    w = torch.full((64,), 3.0, device="cuda")
    bd.diffattn_qk_rope_bwd(q, None, q, None, f, norm=True, dq_weight=w)
    assert not w.any()  # a sum over no rows
    x = torch.zeros((1, 2, 4, 64), dtype=BF16, device="cuda")
    for bad in (dict(positions=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(q_weight=f), dict(rot_dim=32),
                dict(q_out=x[:, :, :2])):
        with pytest.raises(ValueError):
            bd.diffattn_qk_rope_fwd(x, None, f, norm=True, **bad)
    with pytest.raises(bd.DiffAttnError):
        bd.diffattn_qk_rope_fwd(x, None, f[:30])  # 60 features: not whole groups of eight
    with pytest.raises(ValueError):
        bd.diffattn_qk_rope_fwd(x.cpu(), None, f)


def test_graph_and_other_stream():
    g = gen(9)
    q, k, f, p, pos = make(2, 70, 8, 2, 128, 128, BF16, "given", False, g)
    w = torch.rand(128, device="cuda")
    kw = dict(norm=True, q_weight=w, k_weight=w, positions=p)
    exp = bd.diffattn_qk_rope_fwd(q, k, f, **kw)
    dexp = bd.diffattn_qk_rope_bwd(q, k, *exp, f, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bd.diffattn_qk_rope_fwd(q, k, f, stream=s, **kw)
    dgot = bd.diffattn_qk_rope_bwd(q, k, *got, f, stream=s, **kw)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = bd.diffattn_qk_rope_fwd(q, k, f, **kw)
        dcap = bd.diffattn_qk_rope_bwd(q, k, *cap, f, **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in [(exp[i], got[i], cap[i]) for i in (0, 1)] + [(dexp[n], dgot[n], dcap[n]) for n in dexp]:
        assert torch.equal(a, b) and torch.equal(a, c)


# --------------------------------------------------------------- paged append ---
def paged(B, L_max, page, hkv, d, layout, g, spare=3):
    """Pages of NaN, and a table that names them in no order."""
    P = -(-L_max // page)
    n = B * P + spare
    table = torch.randperm(n, generator=g, device="cuda")[:B * P].reshape(B, P).int()
    pages = []
    for _ in range(2):
        if layout == "head":
            t = torch.full((n, hkv, page, d), float("nan"), dtype=BF16, device="cuda").transpose(1, 2)
        elif layout == "token":
            t = torch.full((n, page, hkv, d), float("nan"), dtype=BF16, device="cuda")
        else:  # K and V of a slot side by side
            t = torch.full((n, page, hkv, 2, d), float("nan"), dtype=BF16, device="cuda")[:, :, :, 1]
        pages.append(t)
    return pages, table


@pytest.mark.parametrize("case", [  # counts, lengths, page, h_q, h_kv, d, rot, interleaved, norm, layout, extra rows
    ([1, 1, 1], [1, 40, 33], 16, 8, 2, 128, 128, False, True, "token", 0),
    ([5, 0, 130, 1], [5, 0, 200, 64], 16, 0, 3, 64, 32, True, False, "head", 7),
    ([64, 33], [100, 33], 48, 6, 1, 128, 64, False, True, "apart", 3),
    ([1] * 70, list(range(1, 71)), 1, 4, 2, 64, 64, True, True, "token", 2),
    ([1200], [1300], 256, 16, 8, 128, 0, False, True, "head", 0),
])
def test_paged_append(case):
    n, L, page, h_q, hkv, d, rot, inter, norm, layout, extra = case
    g = gen(sum(L))
    B, T = len(n), sum(n) + extra
    (kp, vp), table = paged(B, max(L), page, hkv, d, layout, g)
    x = randn((T, h_q + 2 * hkv, d), g, BF16, 1.5)
    q, k, v = (x[:, :h_q] if h_q else None), x[:, h_q:h_q + hkv], x[:, h_q + hkv:]
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda")
    sl = torch.tensor(L, dtype=torch.int32, device="cuda")
    f = torch.tensor(500000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1)), dtype=F32, device="cuda")
    w = 1 + randn((d,), g, F32, 0.3) if norm else None
    kw = dict(rot_dim=rot, interleaved=inter, rope_scale=1.0, norm=norm, norm_eps=1e-5)
    q_out = None if q is None else torch.full((T, h_q, d), 7.0, dtype=BF16, device="cuda")
    bd.diffattn_paged_append(k, v, kp, vp, table, cu, sl, f, q=q, q_out=q_out, q_weight=w, k_weight=w, **kw)
    pos = np.concatenate([np.arange(b - a, b) for a, b in zip(n, L)])
    m = sum(n)
    wn = None if w is None else f64(w)
    t = table.cpu().numpy()
    where = torch.tensor([t[b, p // page] for b in range(B) for p in range(L[b] - n[b], L[b])]), torch.tensor(pos % page)
    check_fwd(kp[where], k[:m], f, pos, kw, wn)
    assert torch.equal(vp[where], v[:m])
    if q is not None:
        check_fwd(q_out[:m], q[:m], f, pos, kw, wn)
        assert bool((q_out[m:] == 7).all())
    for pages in (kp, vp):  # nothing else was written
        seen = torch.ones(pages.shape[:2], dtype=torch.bool, device="cuda")
        seen[where] = False
        assert bool(torch.isnan(pages[seen]).all())


def test_paged_append_positions_and_values_as_they_are():
    """Rotation positions of their own; values keep every bit, NaN among them; queries in place."""
    g = gen(3)
    (kp, vp), table = paged(1, 32, 16, 2, 64, "token", g)
    k, q = randn((3, 2, 64), g), randn((3, 4, 64), g)
    v = torch.randint(-2 ** 15, 2 ** 15, (3, 2, 64), generator=g, device="cuda").to(torch.int16).view(BF16)
    cu, sl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [20]))
    p = torch.tensor([5, 900000, -3], dtype=torch.int32, device="cuda")
    f = torch.tensor(10000.0 ** (-np.arange(32) / 32), dtype=F32, device="cuda")
    kw = dict(rot_dim=64, interleaved=False, rope_scale=1.0, norm=False, norm_eps=0.0)
    q0 = q.clone()
    bd.diffattn_paged_append(k, v, kp, vp, table, cu, sl, f, q=q, q_out=q, positions=p)
    page = table[0, 1].long()
    check_fwd(kp[page, 1:4], k, f, p.cpu().numpy(), kw, None)
    check_fwd(q, q0, f, p.cpu().numpy(), kw, None)
    assert torch.equal(vp[page, 1:4].view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("what", ["short", "long", "rows", "falling", "page"])
def test_paged_append_out_of_bounds(what):
    """The status word says so, that sequence (or token) is not written, the others are."""
    g = gen(5)
    (kp, vp), table = paged(3, 32, 16, 2, 64, "token", g)
    cu, sl = [0, 2, 4, 6], [10, 12, 14]
    if what == "short":
        sl[1] = 1
    elif what == "long":
        sl[1] = 33
    elif what == "rows":
        cu[3] = 7
    elif what == "falling":
        cu[3] = 3
    else:
        table[1, 0] = -1
    cu, sl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, sl))
    k, v, q = randn((6, 2, 64), g), randn((6, 2, 64), g), randn((6, 4, 64), g)
    q_out = bd.diffattn_paged_append(k, v, kp, vp, table, cu, sl, None, q=q)
    assert bd.diffattn_get_device_status() == bd.DA_ERR_BOUNDS
    bad = 2 if what in ("rows", "falling") else 1
    for b in range(3):
        rows = kp[table[b, 0].long(), int(sl[b]) - 2:int(sl[b])] if b != bad else None
        if b != bad:
            assert torch.equal(rows, k[2 * b:2 * b + 2]) and torch.equal(q_out[2 * b:2 * b + 2], q[2 * b:2 * b + 2])
        elif what != "falling":
            assert not q_out[2 * b:2 * b + 2].any() or what == "page"
    assert int(torch.isnan(kp[..., 0, 0]).logical_not().sum()) == 4
    if what == "page":
        assert torch.equal(q_out, q)


# ------------------------------------------------------------- a training step ---
@pytest.mark.parametrize("interleaved", [False, True])
def test_training_step_with_the_v2_attention(interleaved):
    """Raw queries and keys normed, rotated, attended, and all the way back: gradients of the raw rows, of the values
    and of the norms' weights against the 64-bit chain, with the attention's own bars (1.5e-2 of a tensor's norm for
    its backward, as much again for the bf16 rows in between)."""
    g = gen(31)
    B, N, h, hkv, d = 2, 130, 4, 2, 64
    q, k, v = randn((B, N, 2 * h, d), g), randn((B, N, hkv, d), g), randn((B, N, hkv, d), g)
    dout, gate = randn((B, N, h, d), g), torch.rand((B, N, h), generator=g, device="cuda")
    w = [1 + randn((d,), g, F32, 0.2) for _ in range(2)]
    f, _ = bd.diffattn_rope_inv_freq(32)
    kw = dict(interleaved=interleaved, norm=True, q_weight=w[0], k_weight=w[1])
    qr, kr = bd.diffattn_qk_rope_fwd(q, k, f, **kw)
    _, saves = bd.diffattn_v2_fwd(qr, kr, v, gate=gate, save=True)
    a = bd.diffattn_v2_bwd(qr, kr, v, dout, saves, gate=gate)
    r = bd.diffattn_qk_rope_bwd(q, k, a["dq"], a["dk"], f, **kw)

    pos = np.broadcast_to(np.arange(N), (B, N))
    rk = dict(rot=32, interleaved=interleaved, do_norm=True)
    q64, k64, w64 = f64(q), f64(k), [f64(x) for x in w]
    q1, k1 = po.qk_rope(q64, f64(f), pos, w=w64[0], **rk), po.qk_rope(k64, f64(f), pos, w=w64[1], **rk)
    gz = f64(gate)
    dq1, dk1, dv1 = np.zeros_like(q1), np.zeros_like(k1), np.zeros_like(k1)
    for b in range(B):  # the chain rule of the attention, head by head
        for j in range(2 * h):
            c = j // (2 * h // hkv)
            t = q1[b, :, j] @ k1[b, :, c].T * d ** -0.5
            t[np.triu_indices(N, 1)] = -np.inf
            A = np.exp(t - t.max(-1, keepdims=True))
            A /= A.sum(-1, keepdims=True)
            do = f64(dout)[b, :, j // 2] * (1.0 if j % 2 == 0 else -gz[b, :, j // 2, None])
            dP = do @ f64(v)[b, :, c].T
            dS = A * (dP - (A * dP).sum(-1, keepdims=True)) * d ** -0.5
            dq1[b, :, j] += dS @ k1[b, :, c]
            dk1[b, :, c] += dS.T @ q1[b, :, j]
            dv1[b, :, c] += A.T @ do
    dq, dqw = po.qk_rope_bwd(q64, dq1, f64(f), pos, w=w64[0], **rk)
    dk, dkw = po.qk_rope_bwd(k64, dk1, f64(f), pos, w=w64[1], **rk)
    for got, exp in ((r["dq"], dq), (r["dk"], dk), (a["dv"], dv1), (r["dq_weight"], dqw), (r["dk_weight"], dkw)):
        assert np.linalg.norm(f64(got) - exp) <= 3e-2 * np.linalg.norm(exp)
