"""Measured cases of the operators around a paged V2 cache: the norm and the
position rotation of queries and keys (with gradients), the append of new
tokens to a cache kept in pages, and the V2 attention of a chunk of new tokens
over those pages.

``run`` computes an operator either in its plain form (elementary torch
operations in 32 bits, rounded once at the end; the angles in 64) or, with
``own`` true, by the calls that a user's program makes.  ``exact`` restates
the definitions in 64 bits.

Norm and rotation of one head's row x, with w and eps where there is a norm:
    z = w x / sqrt(mean x^2 + eps)          (z = x without it)
    a_i = position * inv_freq[i],  i < rot_dim / 2
    (y_u, y_v) = s (z_u cos a_i - z_v sin a_i, z_v cos a_i + z_u sin a_i)
with (u, v) = (i, i + rot_dim / 2) or, interleaved, (2i, 2i + 1); the other
features are z.  Sequence b's new tokens are rows cu_seqlens[b] ..
cu_seqlens[b + 1] - 1 of the packed arrays and the last n of its seqlens[b]
positions; position j lives in slot j % page_size of page
block_table[b, j // page_size].  A new token sees the positions up to its own,
    out[t, p] = A_2p V - gate[t, p] A_2p+1 V.
"""

import math
import random

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # one new token of one conversation: queries and keys normed and rotated, launch latency
        dict(name="rope one token", op="rope", B=1, N=1, h_q=64, h_k=8, d=128, rot=128, layout="half", norm=True,
             dtype="bf16", strided=False, backward=False, far=True),
        # a training step at the library's V2 forward workload: forward and backward of the norm and the rotation
        dict(name="rope training", op="rope", B=2, N=8192, h_q=64, h_k=8, d=128, rot=128, layout="half", norm=True,
             dtype="bf16", strided=False, backward=True, far=False),
        # head dim 64, pairs side by side, half of each head rotated, straight out of a fused projection; odd length
        dict(name="rope partial strided", op="rope", B=3, N=1777, h_q=32, h_k=4, d=64, rot=32, layout="interleaved",
             norm=False, dtype="bf16", strided=True, backward=True, far=False),
        # one new token for each of a serving batch goes into the pages, its queries rotated beside it
        dict(name="append one token", op="append", B=64, N=1, ragged=False, h_q=64, h_kv=8, d=128, L_max=4096, page=16,
             rot=128, layout="half", norm=True, pages="token"),
        # a ragged batch of prompts goes into the pages, positions far beyond the trained context
        dict(name="append prompts", op="append", B=6, N=4096, ragged=True, h_q=64, h_kv=8, d=128, L_max=32768, page=64,
             rot=128, layout="half", norm=False, pages="head"),
        # a single conversation of ordinary length: latency of one decode step
        dict(name="attend one sequence", op="attend", B=1, N=1, ragged=False, h=32, h_kv=8, d=128, L_max=1000, page=16,
             full=True, d_model=0, pages="token"),
        # the library's decode workload over pages (64 sequences, up to 32768, 64 query / 8 KV heads), gate from x
        dict(name="attend decode batch", op="attend", B=64, N=1, ragged=False, h=32, h_kv=8, d=128, L_max=32768, page=64,
             full=True, d_model=4096, pages="head"),
        # four drafted tokens per sequence to verify, ragged lengths, head dim 64
        dict(name="attend drafted tokens", op="attend", B=32, N=4, ragged=False, h=16, h_kv=4, d=64, L_max=8192, page=32,
             full=False, d_model=0, pages="token"),
        # the first chunk of one long prompt: every key is a new token's
        dict(name="attend first chunk", op="attend", B=1, N=8192, ragged=False, h=32, h_kv=8, d=128, L_max=8192, page=128,
             full=True, d_model=4096, pages="head"),
        # later chunks of a ragged batch of long prompts
        dict(name="attend later chunks", op="attend", B=4, N=2048, ragged=True, h=32, h_kv=8, d=128, L_max=32768, page=64,
             full=False, d_model=0, pages="token"),
        # a mixed batch of a serving loop: most sequences decode one token, every eighth brings part of a prompt
        dict(name="attend mixed batch", op="attend", B=48, N=1000, ragged="mixed", h=16, h_kv=4, d=128, L_max=6000,
             page=16, full=False, d_model=0, pages="token"),
        # a layer's whole step of such a loop: tokens rotated and appended, then attended
        dict(name="append and attend", op="step", B=16, N=1, ragged=False, h=32, h_kv=8, d=128, L_max=8192, page=32,
             full=False, d_model=0, pages="token", rot=64, layout="half", norm=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "attend", "attend", "attend", "step"])
    d = rng.choice([64, 128])
    layout, norm = rng.choice(["half", "interleaved"]), rng.random() < 0.6
    rot = rng.choice([d, d, d // 2, d // 4])
    B = _log(rng, 1, 64)
    if op == "rope":
        N = max(1, min(_log(rng, 1, 16384), 16384 // B))
        h_k = rng.choice([1, 2, 4, 8])
        return dict(op=op, B=B, N=N, h_q=h_k * rng.choice([2, 4, 6, 8]), h_k=h_k, d=d, rot=rot, layout=layout, norm=norm,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), strided=rng.random() < 0.4,
                    backward=rng.random() < 0.6, far=rng.random() < 0.4)
    h_kv, page, pages = rng.choice([1, 2, 4, 8]), rng.choice([16, 16, 32, 48, 64, 128, 256]), rng.choice(["token", "head"])
    G = rng.choice([2, 4, 6, 8, 12, 16])
    ragged = rng.choice([False, True, "mixed"])
    if op == "append":
        N = max(1, min(_log(rng, 1, 8192), 16384 // B))
        return dict(op=op, B=B, N=N, ragged=ragged, h_q=rng.choice([0, h_kv * G]), h_kv=h_kv, d=d,
                    L_max=N + _log(rng, 1, max(2, 65536 // B)), page=page, rot=rot, layout=layout, norm=norm, pages=pages)
    L = max(1, min(_log(rng, 1, 131072), (131072 if op == "step" else 524288) // B))
    most = int(3e12 / (B * L * h_kv * G * d * 4))  # the largest listed case's products
    N = 1 if rng.random() < 0.4 else max(1, min(L, _log(rng, 1, 4096), 8192 // B, most))
    c = dict(op=op, B=B, N=N, ragged=ragged, h=h_kv * G // 2, h_kv=h_kv, d=d, L_max=L, page=page, full=rng.random() < 0.3,
             d_model=rng.choice([0, 0, 256, 4096]), pages=pages)
    if op == "step":
        c.update(rot=rot, layout=layout, norm=norm)
    return c


def _counts(c):
    """New tokens of each sequence: a function of the case."""
    rng = random.Random(c["B"] * 131 + c["N"])
    B, N = c["B"], c["N"]
    if c["ragged"] == "mixed":
        return [N - b if b % 8 == 0 and N > b else 1 for b in range(B)]
    if c["ragged"]:
        return [N] + [rng.randint(N // 4, N) for _ in range(B - 1)]
    return [N] * B


# ---------------------------------------------------------------- prepare ---
def _randn(shape, g, std=1.0, dtype=BF16):
    x = torch.randn(shape, generator=g, device=DEV, dtype=dtype)
    return x if std == 1.0 else x * std


def _frequencies(rot, far):
    """Radians per position and the factor s: as trained, or stretched 16-fold where one turn is longer than 4096
    positions, with the frequencies in between ramped and a factor for the attention's spread."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2 * i / rot)
    if not far:
        return f.float().to(DEV), 1.0
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return (f * keep + f / 16 * (1 - keep)).float().to(DEV), 0.1 * math.log(16) + 1


def _table(s, c, g):
    """Pages in no order for B sequences of up to L_max positions, and a few that nobody has."""
    P = -(-c["L_max"] // c["page"])
    n = c["B"] * P + 3
    s["table"] = torch.randperm(n, generator=g, device=DEV)[:c["B"] * P].reshape(c["B"], P).int()
    h_kv, d, page = c["h_kv"], c["d"], c["page"]
    for x in ("k_pages", "v_pages"):
        if c["op"] == "append":
            t = torch.zeros((n, h_kv, page, d) if c["pages"] == "head" else (n, page, h_kv, d), dtype=BF16, device=DEV)
        else:
            t = _randn((n, h_kv, page, d) if c["pages"] == "head" else (n, page, h_kv, d), g)
        s[x] = t.transpose(1, 2) if c["pages"] == "head" else t


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, d = c["op"], c["d"]
    s = dict(op=op, case=c)
    if op == "rope":
        B, N, h_q, h_k = c["B"], c["N"], c["h_q"], c["h_k"]
        dt = BF16 if c["dtype"] == "bf16" else torch.float32
        if c["strided"]:
            x = _randn((B, N, h_q + 2 * h_k, d), g, 1.5, dt)
            s["q"], s["k"] = x[:, :, :h_q], x[:, :, h_q:h_q + h_k]
        else:
            s["q"], s["k"] = _randn((B, N, h_q, d), g, 1.5, dt), _randn((B, N, h_k, d), g, 1.5, dt)
        if c["backward"]:
            s["dq"], s["dk"] = _randn((B, N, h_q, d), g, 1.0, dt), _randn((B, N, h_k, d), g, 1.0, dt)
        s["inv_freq"], s["factor"] = _frequencies(c["rot"], c["far"])
        start = torch.randint(0, 100000 if c["far"] else 1, (B, 1), generator=g, device=DEV)
        s["positions"] = (start + torch.arange(N, device=DEV)).int()
        s["wq"] = s["wk"] = None
        if c["norm"]:
            s["wq"], s["wk"] = (1 + _randn((d,), g, 0.2, torch.float32) for _ in range(2))
        s["workspace"] = None  # a training loop keeps one: made by the first pass
        return s
    n = _counts(c)
    T, B, h_kv = sum(n), c["B"], c["h_kv"]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s["n"], s["cu"] = n, torch.tensor(cu, dtype=torch.int32, device=DEV)
    low = torch.tensor(n, dtype=torch.int32, device=DEV)
    if c.get("full"):
        s["seqlens"] = torch.full((B,), c["L_max"], dtype=torch.int32, device=DEV)
    else:
        s["seqlens"] = low + (torch.rand((B,), generator=g, device=DEV) * (c["L_max"] - low + 1)).int().clamp(max=c["L_max"] - low)
    _table(s, c, g)
    h_q = c["h_q"] if op == "append" else 2 * c["h"]
    if op in ("append", "step"):
        x = _randn((T, h_q + 2 * h_kv, d), g, 1.5)  # a fused projection
        s["q"] = x[:, :h_q] if h_q else None
        s["k"], s["v"] = x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
        s["q_out"] = torch.zeros((T, h_q, d), dtype=BF16, device=DEV) if h_q else None
        s["inv_freq"], s["factor"] = _frequencies(c["rot"], c["L_max"] > 8192)
        s["wq"] = s["wk"] = None
        if c["norm"]:
            s["wq"], s["wk"] = (1 + _randn((d,), g, 0.2, torch.float32) for _ in range(2))
    else:
        s["q"] = _randn((T, h_q, d), g)
    if op in ("attend", "step"):
        h = c["h"]
        if c["d_model"]:
            s["gate"], s["x"], s["w_lambda"] = None, _randn((T, c["d_model"]), g), _randn((c["d_model"], h), g, 0.02)
        else:
            s["gate"], s["x"], s["w_lambda"] = torch.rand((T, h), generator=g, device=DEV), None, None
        s["out"] = torch.zeros((T, h, d), dtype=BF16, device=DEV)
        s["workspace"] = None  # a serving loop keeps one: made by the first pass
    return s


# ------------------------------------------------------------- plain forms --
def _angles(s, positions):
    """cos and sin of every position and frequency, fp32 from 64-bit angles."""
    a = positions.double()[..., None] * s["inv_freq"].double()
    return torch.cos(a).float()[..., None, :], torch.sin(a).float()[..., None, :]


def _turn(x, cos, sin, c, factor):
    """The rotation of rows x [..., heads, d] (fp32) by angles [..., 1, rot / 2]."""
    rot = c["rot"]
    if c["layout"] == "half":
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        u, v = x[..., :rot:2], x[..., 1:rot:2]
    u, v = factor * (u * cos - v * sin), factor * (v * cos + u * sin)
    y = torch.cat((u, v), -1) if c["layout"] == "half" else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


EPS = 1e-5


def _norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_rope(s):
    c = s["case"]
    cos, sin = _angles(s, s["positions"])
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        out.append(_turn(_norm(x, w), cos, sin, c, s["factor"]).to(x.dtype))
    if not c["backward"]:
        return out
    dw = []
    for x, w, dy in ((s["q"], s["wq"], s["dq"]), (s["k"], s["wk"], s["dk"])):
        dz = _turn(dy.float(), cos, -sin, c, s["factor"])
        if w is None:
            out.append(dz.to(x.dtype))
            continue
        r = torch.rsqrt((x.float() ** 2).mean(-1, keepdim=True) + EPS)
        xh = x.float() * r
        dw.append((dz * xh).sum((0, 1, 2), dtype=torch.float64).float())
        dz = dz * w
        out.append((r * (dz - xh * (dz * xh).mean(-1, keepdim=True))).to(x.dtype))
    return out + dw


def _new_positions(s):
    """(sequence, position) of every packed token."""
    n = torch.diff(s["cu"])
    b = torch.repeat_interleave(torch.arange(len(s["n"]), device=DEV), n.long(), output_size=sum(s["n"]))
    i = torch.arange(sum(s["n"]), device=DEV) - s["cu"][b]
    return b, (s["seqlens"] - n)[b] + i


def _plain_append(s):
    c = s["case"]
    b, pos = _new_positions(s)
    cos, sin = _angles(s, pos)
    where = (s["table"][b, pos // c["page"]].long(), pos % c["page"])
    s["k_pages"][where] = _turn(_norm(s["k"], s["wk"]), cos, sin, c, s["factor"]).to(BF16)
    s["v_pages"][where] = s["v"]
    if s["q"] is None:
        return s["k_pages"], s["v_pages"]
    s["q_out"].copy_(_turn(_norm(s["q"], s["wq"]), cos, sin, c, s["factor"]))
    return s["q_out"], s["k_pages"], s["v_pages"]


def _plain_attend(s, q):
    c = s["case"]
    h, h_kv, d = c["h"], c["h_kv"], c["d"]
    G = 2 * h // h_kv
    gate = s["gate"]
    if gate is None:
        gate = 1 / (1 + torch.exp(-(s["x"].float() @ s["w_lambda"].float())))
    t0 = 0
    for b, n in enumerate(s["n"]):
        if n == 0:
            continue
        # keys behind the sequence's end are masked like those behind a token, so no length comes to the host
        k, v = (s[x][s["table"][b].long()].flatten(0, 1)[:c["L_max"]].transpose(0, 1).float() for x in ("k_pages", "v_pages"))
        pos = s["seqlens"][b] - n + torch.arange(n, device=DEV)
        hidden = (torch.arange(k.shape[1], device=DEV) > pos[:, None])[None, :, None]
        qb = q[t0:t0 + n].float().reshape(n, h_kv, G, d).transpose(0, 1) / math.sqrt(d)
        step = max(1, 2 ** 30 // (n * G * k.shape[1]))  # KV heads at a time
        for g in range(0, h_kv, step):
            e = min(h_kv, g + step)
            a = torch.matmul(qb[g:e].reshape(e - g, n * G, d), k[g:e].transpose(-1, -2)).reshape(e - g, n, G, -1)
            a = a.masked_fill_(hidden, -torch.inf)
            a = a.sub_(a.amax(-1, keepdim=True)).exp_()
            a = a.div_(a.sum(-1, keepdim=True))
            o = torch.matmul(a.reshape(e - g, n * G, -1), v[g:e]).reshape(e - g, n, G // 2, 2, d)
            del a
            gg = gate[t0:t0 + n].reshape(n, h_kv, G // 2, 1)[:, g:e].transpose(0, 1)
            s["out"][t0:t0 + n, g * G // 2:e * G // 2] = (o[..., 0, :] - gg * o[..., 1, :]).transpose(0, 1).flatten(1, 2).to(BF16)
        t0 += n
    return s["out"]


# -------------------------------------------------------------------- run ---
def run(state):
    s = state
    c, op = s["case"], s["op"]
    if not own:
        if op == "rope":
            return _plain_rope(s)
        got = _plain_append(s) if op != "attend" else None
        if op == "append":
            return got
        out = _plain_attend(s, s["q"] if op == "attend" else s["q_out"])
        return out if op == "attend" else (out, *got)
    import differential_attention_diff_gb300 as da
    if op == "rope":
        kw = dict(positions=s["positions"], rot_dim=c["rot"], interleaved=c["layout"] == "interleaved",
                  rope_scale=s["factor"], norm=c["norm"], norm_eps=EPS, q_weight=s["wq"], k_weight=s["wk"])
        out = list(da.diffattn_qk_rope_fwd(s["q"], s["k"], s["inv_freq"], **kw))
        if c["backward"]:
            if s["workspace"] is None:
                size = da.diffattn_qk_rope_bwd_workspace_size(c["B"], c["N"], c["h_q"], c["h_k"], c["d"])
                s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
            g = da.diffattn_qk_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["inv_freq"], workspace=s["workspace"], **kw)
            out += [g["dq"], g["dk"]]
            if c["norm"]:
                out += [g["dq_weight"], g["dk_weight"]]
        return out
    got = []
    where = (s["k_pages"], s["v_pages"], s["table"], s["cu"], s["seqlens"])
    if op != "attend":
        da.diffattn_paged_append(s["k"], s["v"], *where, s["inv_freq"], q=s["q"], q_out=s["q_out"], rot_dim=c["rot"],
                                 interleaved=c["layout"] == "interleaved", rope_scale=s["factor"], norm=c["norm"],
                                 norm_eps=EPS, q_weight=s["wq"], k_weight=s["wk"])
        got = [s["k_pages"], s["v_pages"]] if s["q"] is None else [s["q_out"], s["k_pages"], s["v_pages"]]
        if op == "append":
            return got
    q = s["q"] if op == "attend" else s["q_out"]
    if s["workspace"] is None:
        size = da.diffattn_v2_paged_fwd_workspace_size(q.shape[0], c["B"], c["N"], c["h"], c["h_kv"], c["d"],
                                                       gate_given=s["gate"] is not None)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    out = da.diffattn_v2_paged_fwd(q, *where, max_new=c["N"], gate=s["gate"], x=s["x"], w_lambda=s["w_lambda"], out=s["out"],
                                   workspace=s["workspace"])
    return out if op == "attend" else (out, *got)


# ------------------------------------------------------------------- work ---
def work(case):
    c = case
    d, op = c["d"], c["op"]
    if op == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        rows = c["B"] * c["N"] * (c["h_q"] + c["h_k"])
        # forward: rows in and out; backward: rows and their outputs' gradients in, gradients out
        return {"bytes": rows * d * size * (5 if c["backward"] else 2) + c["B"] * c["N"] * 4, "flops": rows * d * (20 if c["backward"] else 8)}
    n = _counts(c)
    T, h_kv = sum(n), c["h_kv"]
    small = (c["B"] * -(-c["L_max"] // c["page"]) + 2 * c["B"]) * 4
    done = {"bytes": 0, "flops": 0}
    if op in ("append", "step"):
        h_q = c["h_q"] if op == "append" else 2 * c["h"]
        done = {"bytes": T * (h_q + 2 * h_kv) * d * 4 + small, "flops": T * (h_q + h_kv) * d * 8}
    if op == "append":
        return done
    h = c["h"]
    keys = pairs = 0.0
    for x in filter(None, n):
        L = c["L_max"] if c["full"] else (x + c["L_max"]) / 2
        keys += L
        pairs += x * (L - (x - 1) / 2)
    done["bytes"] += keys * h_kv * d * 4 + T * 3 * h * d * 2 + (T + h) * c["d_model"] * 2 + small
    done["flops"] += pairs * 2 * h * d * 4 + 2 * T * h * c["d_model"]
    return done


# ------------------------------------------------------------------ exact ---
def _rotated64(s, x, w, positions, transposed=False):
    """The definition on rows x [tokens, heads, d], feature pair by feature pair."""
    c = s["case"]
    x = x.double()
    if w is not None and not transposed:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS) * w.double()
    y = x.clone()
    for i in range(c["rot"] // 2):
        u, v = (i, i + c["rot"] // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        a = positions.double() * float(s["inv_freq"][i])
        co, si = torch.cos(a)[:, None] * s["factor"], torch.sin(a)[:, None] * s["factor"]
        if transposed:
            si = -si
        y[..., u] = x[..., u] * co - x[..., v] * si
        y[..., v] = x[..., v] * co + x[..., u] * si
    return y


def _exact_rope(s, c):
    pos = s["positions"].reshape(-1)
    flat = [s[x].reshape(-1, s[x].shape[2], c["d"]) for x in ("q", "k")]
    outs = [_rotated64(s, x, w, pos).reshape(s[n].shape) for x, w, n in zip(flat, (s["wq"], s["wk"]), ("q", "k"))]
    if not c["backward"]:
        return outs
    dw = []
    for x, w, n in zip(flat, (s["wq"], s["wk"]), ("dq", "dk")):
        dz = _rotated64(s, s[n].reshape(x.shape), None, pos, transposed=True)
        if w is not None:
            x = x.double()
            rms = torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS)
            dw.append((dz * x / rms).sum((0, 1)))
            gx = dz * w.double()
            dz = gx / rms - x * (gx * x).sum(-1, keepdim=True) / (c["d"] * rms ** 3)
        outs.append(dz.reshape(s[n].shape))
    return outs + dw


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        return _exact_rope(s, c)
    n = s["n"]
    if work(c)["flops"] > 1e13:
        return None
    lengths, outs = s["seqlens"].tolist(), []
    q, pages = s["q"], [s["k_pages"], s["v_pages"]]
    if c["op"] != "attend":
        b = [i for i, x in enumerate(n) for _ in range(x)]
        pos = [lengths[i] - x + j for i, x in enumerate(n) for j in range(x)]
        table, pos = s["table"].cpu(), torch.tensor(pos)
        page = table[torch.tensor(b), pos // c["page"]].long().to(DEV)
        slot, pos = (pos % c["page"]).to(DEV), pos.to(DEV)
        if q is not None:
            q = _rotated64(s, q, s["wq"], pos)
            outs.append(q)
        outs += [p.double() for p in pages]
        outs[-2][page, slot] = _rotated64(s, s["k"], s["wk"], pos)
        outs[-1][page, slot] = s["v"].double()
        if c["op"] == "append":
            return outs
        # the attention reads what the pages and the rotated queries hold: bf16 rows
        q, pages = q.to(BF16), [x.to(BF16) for x in outs[1:]]
    h, h_kv, d = c["h"], c["h_kv"], c["d"]
    G = 2 * h // h_kv
    out = torch.zeros((sum(n), h, d), dtype=torch.float64, device=DEV)
    t0 = 0
    for b, x in enumerate(n):
        L = lengths[b]
        used = s["table"][b, :-(-L // c["page"])].long()
        if s["gate"] is None:
            gate = torch.sigmoid(s["x"][t0:t0 + x].double() @ s["w_lambda"].double())
        else:
            gate = s["gate"][t0:t0 + x].double()
        last = torch.arange(L - x, L, device=DEV)
        for g in range(h_kv):
            k, v = (p[used, :, g].reshape(-1, d)[:L].double() for p in pages)
            for p in range(g * G // 2, (g + 1) * G // 2):
                o = []
                for j in (2 * p, 2 * p + 1):
                    t = q[t0:t0 + x, j].double() @ k.T * d ** -0.5
                    t[torch.arange(L, device=DEV) > last[:, None]] = -torch.inf
                    o.append(torch.softmax(t, -1) @ v)
                out[t0:t0 + x, p] = o[0] - gate[:, p:p + 1] * o[1]
        t0 += x
    return out if c["op"] == "attend" else (out, *outs)
