"""Measured cases of the serving-cache operators: a KV cache held in 4 bits
(append, read back, V2 decode over it), the differential attention weight
that each cached key gathers, and the eviction of the keys that gather least.

``run`` computes an operator either in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, with ``own`` true, by the
calls that a user's program makes.  ``exact`` restates the definitions in 64
bits.

A 4-bit record holds one key and one value row of one KV head, d + 16 bytes:
    [K codes, d/2][V codes, d/2][K s0 s1 m0 m1][V s0 s1 m0 m1]
Byte i of a code row holds feature 2i in its low and 2i + 1 in its high four
bits.  A row has two groups of d/2 features, each with a bf16 scale s and
minimum m: s = bf16((max - min) / 15), code = rint((x - m) / s) in 0..15,
value = s * code + m.  A group with s = 0 has codes 0; a group whose scale is
not finite (a NaN or an infinity in it) is stored as NaN.

The weight that key j gathers in one decode step, per KV head:
    w[j] = sum over the head's pairs p of |A_2p[j] - gate_p A_2p+1[j]|.
"""

import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # one new token per sequence of a serving batch (the library's decode batch): launch latency
        dict(name="append one token", op="append", B=64, N=1, h_kv=8, d=128, L_max=4096, ragged=False, layout="head",
             strided=False),
        # a padded batch of prompts goes into the cache straight out of a fused q/k/v projection
        dict(name="append prompts", op="append", B=4, N=4096, h_kv=8, d=128, L_max=4224, ragged=True, layout="head",
             strided=True),
        # a short cached prefix read back for the next chunk of a prefill; odd length, token-major cache
        dict(name="read short prefix", op="read", B=1, N=777, h_kv=4, d=64, L_max=1000, ragged=False, layout="token"),
        # the cached prefixes of a batch read back for an attention over bf16 rows
        dict(name="read prefixes", op="read", B=4, N=8192, h_kv=8, d=128, L_max=8192, ragged=True, layout="head"),
        # a single conversation of ordinary length: latency of one decode step
        dict(name="decode4 one sequence", op="decode4", B=1, h=32, h_kv=8, d=128, L_max=1000, ragged=False,
             layout="head", weights=False, d_model=0),
        # the library's decode workload (64 sequences of 32768, 64 query / 8 KV heads), gate from x
        dict(name="decode4 batch", op="decode4", B=64, h=32, h_kv=8, d=128, L_max=32768, ragged=False, layout="head",
             weights=False, d_model=4096),
        # a ragged batch at head dim 64 with 16 query heads per KV head, keys' weights gathered, token-major cache
        dict(name="decode4 ragged weights", op="decode4", B=16, h=16, h_kv=2, d=64, L_max=8192, ragged=True,
             layout="token", weights=True, d_model=0),
        # two very long contexts whose keys' weights are gathered for an eviction
        dict(name="decode4 long weights", op="decode4", B=2, h=32, h_kv=8, d=128, L_max=131072, ragged=False,
             layout="head", weights=True, d_model=0),
        # the same gathering over a bf16 cache: a small ragged batch, and a large one
        dict(name="weighted ragged", op="weighted", B=8, h=32, h_kv=8, d=128, L_max=4096, ragged=True, d_model=0),
        dict(name="weighted batch", op="weighted", B=32, h=32, h_kv=8, d=128, L_max=16384, ragged=False, d_model=4096),
        # prompts of a batch cut down to a budget after their prefill (bf16 K and V, first eviction)
        dict(name="evict prompts", op="evict", B=16, h_kv=8, d=128, L_max=8192, keep=2048, sinks=4, recent=256,
             ragged=True, kind="bf16", positions=False),
        # steady state of a long-running batch: 256 tokens over the budget, slots out of order by now (4-bit records)
        dict(name="evict steady state", op="evict", B=64, h_kv=8, d=128, L_max=4352, keep=4096, sinks=4, recent=512,
             ragged=False, kind="kv4", positions=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode4", "decode4", "weighted", "evict"])
    B, h_kv, d = _log(rng, 1, 64), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    ragged, layout = rng.random() < 0.5, rng.choice(["head", "token"])
    if op in ("append", "read"):
        N = max(1, min(_log(rng, 1, 16384), 65536 // B))
        c = dict(op=op, B=B, N=N, h_kv=h_kv, d=d, L_max=N + _log(rng, 1, 2000), ragged=ragged, layout=layout)
        if op == "append":
            c["strided"] = rng.random() < 0.5
        return c
    if op == "evict":
        L = max(2, min(_log(rng, 2, 131072), 262144 // B))
        keep = max(1, int(L * rng.uniform(0.05, 1.0)))
        sinks = min(keep, rng.choice([0, 1, 4]))
        return dict(op=op, B=B, h_kv=h_kv, d=d, L_max=L, keep=keep, sinks=sinks,
                    recent=int((keep - sinks) * rng.uniform(0.0, 0.5)), ragged=ragged, kind=rng.choice(["bf16", "kv4"]),
                    positions=rng.random() < 0.5)
    G = rng.choice([2, 4, 6, 8, 12, 16])
    L = max(1, min(_log(rng, 1, 131072), 524288 // B))
    c = dict(op=op, B=B, h=h_kv * G // 2, h_kv=h_kv, d=d, L_max=L, ragged=ragged,
             d_model=rng.choice([0, 0, 256, 4096]))
    if op == "decode4":
        c.update(layout=layout, weights=rng.random() < 0.5)
    return c


# ----------------------------------------------------------- the 4-bit form --
def _quantise(x):
    """codes [..., d] (uint8), scale and minimum [..., 2] (fp32, bf16 values) of rows x [..., d]."""
    g = x.float().unflatten(-1, (2, -1))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) / 15).to(BF16).float()
    n = torch.where((s > 0)[..., None], (g - lo[..., None]) / s[..., None], 0.0).round().clamp(0, 15)
    bad = ~torch.isfinite(s)
    s, lo = torch.where(bad, torch.nan, s), torch.where(bad, torch.nan, lo)
    n = torch.where(bad[..., None], 0.0, n)
    return n.flatten(-2).to(torch.uint8), s, lo


def _pack(k, v):
    """Records [..., d + 16] of key and value rows [..., d]."""
    parts, params = [], []
    for x in (k, v):
        n, s, m = _quantise(x)
        parts.append(n[..., 0::2] | (n[..., 1::2] << 4))
        params.append(torch.cat((s, m), -1).to(BF16).view(torch.uint8))
    return torch.cat(parts + params, -1)


def _unpack(rec, dtype=torch.float32):
    """The key and value rows [..., d] that records [..., d + 16] stand for."""
    d = rec.shape[-1] - 16
    out = []
    for i in (0, 1):
        c = rec[..., i * (d // 2):(i + 1) * (d // 2)]
        n = torch.stack((c & 15, c >> 4), -1).flatten(-2).to(dtype).unflatten(-1, (2, -1))
        p = rec[..., d + 8 * i:d + 8 * i + 8].contiguous().view(BF16).to(dtype)
        out.append((n * p[..., 0:2, None] + p[..., 2:4, None]).flatten(-2))
    return out


def _cache(B, L_max, h_kv, row, layout, dtype):
    """A zeroed cache [B, L_max, h_kv, row], laid out head by head or token by token."""
    if layout == "head":
        return torch.zeros((B, h_kv, L_max, row), dtype=dtype, device=DEV).transpose(1, 2)
    return torch.zeros((B, L_max, h_kv, row), dtype=dtype, device=DEV)


def _randn(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(BF16)


def _lengths(B, lo, hi, ragged, g):
    if not ragged:
        return torch.full((B,), hi, dtype=torch.int32, device=DEV)
    n = torch.randint(lo, hi + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    n[0] = hi
    return n


# ---------------------------------------------------------------- prepare ---
def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    B, h_kv, d, L_max, op = c["B"], c["h_kv"], c["d"], c["L_max"], c["op"]
    s = dict(op=op, case=c)
    if op == "append":
        N = c["N"]
        if c["strided"]:  # views into a fused projection, four query heads per KV head in front of them
            x = _randn((B, N, 6 * h_kv, d), g)
            s["k"], s["v"] = x[:, :, 4 * h_kv:5 * h_kv], x[:, :, 5 * h_kv:]
        else:
            s["k"], s["v"] = _randn((B, N, h_kv, d), g), _randn((B, N, h_kv, d), g)
        s["cache"] = _cache(B, L_max, h_kv, d + 16, c["layout"], torch.uint8)
        s["counts"] = _lengths(B, 0, N, c["ragged"], g)
        s["start"] = torch.randint(0, L_max - N + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["positions"] = torch.full((B, h_kv, L_max), -1, dtype=torch.int32, device=DEV)
        s["weights"] = torch.ones((B, h_kv, L_max), device=DEV)
        s["k_out"], s["v_out"] = (torch.zeros((B, N, h_kv, d), dtype=BF16, device=DEV) for _ in range(2))
        return s
    if op == "read":
        N = c["N"]
        s["cache"] = _cache(B, L_max, h_kv, d + 16, c["layout"], torch.uint8)
        for b in range(B):
            s["cache"][b] = _pack(_randn((L_max, h_kv, d), g), _randn((L_max, h_kv, d), g))
        s["counts"] = _lengths(B, 0, N, c["ragged"], g)
        s["start"] = torch.randint(0, L_max - N + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["k_out"], s["v_out"] = (torch.zeros((B, N, h_kv, d), dtype=BF16, device=DEV) for _ in range(2))
        return s
    if op == "evict":
        s["seqlens"] = _lengths(B, min(c["keep"] + 1, L_max), L_max, c["ragged"], g)
        # gathered weights spread over orders of magnitude; one slot in ten has gathered nothing, so ties occur
        w = torch.randn((B, h_kv, L_max), generator=g, device=DEV).mul_(2.0).exp_()
        s["weights"] = torch.where(torch.rand((B, h_kv, L_max), generator=g, device=DEV) < 0.1, 0.0, w)
        if c["kind"] == "bf16":
            s["rows"] = [_randn((B, L_max, h_kv, d), g) for _ in range(2)]
        else:
            s["rows"] = [torch.randint(0, 256, (B, h_kv, L_max, d + 16), generator=g, device=DEV,
                                       dtype=torch.uint8).transpose(1, 2)]
        s["positions"] = s["next"] = None
        if c["positions"]:  # half again as many tokens seen as slots filled; the slots in no order
            seen = L_max + L_max // 2 + 1
            s["positions"] = torch.rand((B, h_kv, seen), generator=g, device=DEV).argsort(-1)[..., :L_max].int()
            s["next"] = torch.full((B,), seen, dtype=torch.int32, device=DEV)
        s["weights_out"] = torch.zeros_like(s["weights"])
        s["positions_out"] = torch.full((B, h_kv, L_max), -1, dtype=torch.int32, device=DEV)
        s["seqlens_out"] = torch.zeros_like(s["seqlens"])
        s["workspace"] = None  # a serving loop keeps one: made by the first pass
        return s
    h = c["h"]
    s["q"] = _randn((B, 2 * h, d), g)
    s["seqlens"] = _lengths(B, 1, L_max, c["ragged"], g)
    if c["d_model"]:
        s["gate"], s["x"], s["w_lambda"] = None, _randn((B, c["d_model"]), g), _randn((c["d_model"], h), g, 0.02)
    else:
        s["gate"], s["x"], s["w_lambda"] = torch.rand((B, h), generator=g, device=DEV), None, None
    if op == "decode4":
        s["cache"] = _cache(B, L_max, h_kv, d + 16, c["layout"], torch.uint8)
        for b in range(B):
            s["cache"][b] = _pack(_randn((L_max, h_kv, d), g), _randn((L_max, h_kv, d), g))
    else:
        s["k"], s["v"] = _randn((B, L_max, h_kv, d), g), _randn((B, L_max, h_kv, d), g)
    s["weights"] = s["weights_out"] = None
    if op == "weighted" or c["weights"]:
        # what some sixteen steps before this one have gathered
        s["weights"] = torch.rand((B, h_kv, L_max), generator=g, device=DEV).mul_(16.0 * h / h_kv / L_max)
        s["weights_out"] = torch.zeros((B, h_kv, L_max), device=DEV)
    s["workspace"] = None  # a serving loop keeps one: made by the first pass
    return s


# ------------------------------------------------------------- plain forms --
def _slots(start, counts, N):
    """(b, i, slot) of every row that a call with these starts and counts touches."""
    b, i = torch.nonzero(torch.arange(N, device=DEV)[None, :] < counts[:, None], as_tuple=True)
    return b, i, i + start[b]


def _plain_append(s):
    N = s["case"]["N"]
    b, i, slot = _slots(s["start"], s["counts"], N)
    s["cache"][b, slot] = _pack(s["k"][b, i], s["v"][b, i])
    s["weights"][b, :, slot] = 0.0
    s["positions"][b, :, slot] = slot.int()[:, None]
    return (*_plain_read(s), s["weights"], s["positions"])


def _plain_read(s):
    N = s["case"]["N"]
    b, i, slot = _slots(s["start"], s["counts"], N)
    k, v = _unpack(s["cache"][b, slot])
    s["k_out"][b, i], s["v_out"][b, i] = k.to(BF16), v.to(BF16)
    return s["k_out"], s["v_out"]


def _plain_decode(s):
    c = s["case"]
    B, h, h_kv, d, L = c["B"], c["h"], c["h_kv"], c["d"], c["L_max"]
    G = 2 * h // h_kv
    if c["op"] == "decode4":
        k, v = _unpack(s["cache"].transpose(1, 2))
    else:
        k, v = s["k"].transpose(1, 2).float(), s["v"].transpose(1, 2).float()
    gate = s["gate"]
    if gate is None:
        gate = 1 / (1 + torch.exp(-(s["x"].float() @ s["w_lambda"].float())))
    t = torch.matmul(s["q"].float().reshape(B, h_kv, G, d) / math.sqrt(d), k.transpose(-1, -2))
    seen = torch.arange(L, device=DEV)[None, :] < s["seqlens"][:, None]
    t = torch.where(seen[:, None, None, :], t, -torch.inf)
    p = torch.exp(t - t.amax(-1, keepdim=True))
    a = (p / p.sum(-1, keepdim=True)).reshape(B, h_kv, G // 2, 2, L)
    del t, p
    a = a[:, :, :, 0] - gate.reshape(B, h_kv, G // 2, 1) * a[:, :, :, 1]
    out = torch.matmul(a, v).reshape(B, h, d).to(BF16)
    if s["weights_out"] is None:
        return out
    w = torch.where(seen[:, None, :], s["weights"] + a.abs().sum(2), s["weights_out"])
    s["weights_out"].copy_(w)
    return out, s["weights_out"]


def _plain_evict(s):
    c = s["case"]
    B, h_kv, L, keep = c["B"], c["h_kv"], c["L_max"], c["keep"]
    slot = torch.arange(L, device=DEV).expand(B, h_kv, L)
    n = s["seqlens"][:, None, None].long()
    pos = slot if s["positions"] is None else s["positions"].long()
    end = n if s["next"] is None else s["next"][:, None, None].long()
    safe = (pos < c["sinks"]) | (pos >= end - c["recent"])
    key = torch.where(safe, torch.inf, s["weights"])
    key = torch.where(slot < n, key, -torch.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices  # ties: the lowest slot first
    kept = torch.zeros((B, h_kv, L), dtype=torch.bool, device=DEV)
    kept.scatter_(-1, order[..., :keep], True)
    kept &= slot < n
    m = torch.minimum(n, torch.tensor(keep, device=DEV))
    hole, late = (slot < m) & ~kept, kept & (slot >= m)
    # the i-th hole below the new length takes the i-th kept slot above it
    dst, src = torch.nonzero(hole, as_tuple=True), torch.nonzero(late, as_tuple=True)[2]
    frm = slot.clone()
    frm[dst] = src
    live = slot < m
    s["weights_out"].copy_(torch.where(live, s["weights"].gather(-1, frm), s["weights_out"]))
    s["positions_out"].copy_(torch.where(live, pos.gather(-1, frm).int(), s["positions_out"]))
    s["seqlens_out"].copy_(m.reshape(B))
    for r in s["rows"]:
        r[dst[0], dst[2], dst[1]] = r[dst[0], src, dst[1]]
    return (*_rows_out(s), s["weights_out"], s["positions_out"], s["seqlens_out"])


def _rows_out(s):
    """The cache after an eviction: bf16 rows, or 4-bit records as the 32-bit words that were moved (none is recomputed)."""
    return [r if r.dtype == BF16 else r.transpose(1, 2).view(torch.int32) for r in s["rows"]]


# -------------------------------------------------------------------- run ---
def run(state):
    s = state
    op = s["op"]
    if own:
        import differential_attention_diff_gb300 as da
        if op == "append":
            da.diffattn_kv4_append(s["k"], s["v"], s["cache"], start=s["start"], counts=s["counts"],
                                   key_weights=s["weights"], positions=s["positions"])
            k, v = da.diffattn_kv4_read(s["cache"], s["case"]["N"], start=s["start"], counts=s["counts"],
                                        k_out=s["k_out"], v_out=s["v_out"])
            return k, v, s["weights"], s["positions"]
        if op == "read":
            return da.diffattn_kv4_read(s["cache"], s["case"]["N"], start=s["start"], counts=s["counts"],
                                        k_out=s["k_out"], v_out=s["v_out"])
        c = s["case"]
        if op == "evict":
            if s["workspace"] is None:
                n = da.diffattn_kv_evict_workspace_size(c["B"], c["h_kv"], c["L_max"], c["keep"])
                s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
            da.diffattn_kv_evict(s["rows"], s["weights"], c["keep"], sinks=c["sinks"], recent=c["recent"],
                                 seqlens=s["seqlens"], positions=s["positions"], next_position=s["next"],
                                 weights_out=s["weights_out"], positions_out=s["positions_out"],
                                 seqlens_out=s["seqlens_out"], workspace=s["workspace"])
            return (*_rows_out(s), s["weights_out"], s["positions_out"], s["seqlens_out"])
        kw = dict(seqlens=s["seqlens"], gate=s["gate"], x=s["x"], w_lambda=s["w_lambda"], weights_in=s["weights"],
                  weights_out=s["weights_out"])
        size = (c["B"], c["h"], c["h_kv"], c["d"], c["L_max"])
        if op == "decode4":
            if s["workspace"] is None:
                n = da.diffattn_v2_decode_kv4_workspace_size(*size, gate_given=s["gate"] is not None,
                                                             weights=s["weights_out"] is not None)
                s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
            out = da.diffattn_v2_decode_kv4(s["q"], s["cache"], workspace=s["workspace"], **kw)
        else:
            if s["workspace"] is None:
                n = da.diffattn_v2_decode_weighted_workspace_size(*size, gate_given=s["gate"] is not None)
                s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
            out = da.diffattn_v2_decode_weighted(s["q"], s["k"], s["v"], workspace=s["workspace"], **kw)
        return out if s["weights_out"] is None else (out, s["weights_out"])
    if op == "append":
        return _plain_append(s)
    if op == "read":
        return _plain_read(s)
    if op == "evict":
        return _plain_evict(s)
    return _plain_decode(s)


# ------------------------------------------------------------------- work ---
def _mean_length(c, lo, hi):
    return (lo + hi) / 2 if c["ragged"] else hi


def work(case):
    c = case
    B, h_kv, d, op = c["B"], c["h_kv"], c["d"], c["op"]
    if op in ("append", "read"):
        rows = B * h_kv * _mean_length(c, 0, c["N"])
        # append: 2 bf16 rows in, a record out, then that record in and 2 bf16 rows out; weight and position reset
        per = 2 * (4 * d + d + 16) + 8 if op == "append" else 4 * d + d + 16
        return {"bytes": rows * per, "flops": rows * 2 * d * (6 if op == "append" else 2)}
    if op == "evict":
        n = _mean_length(c, min(c["keep"] + 1, c["L_max"]), c["L_max"])
        row = 4 * d if c["kind"] == "bf16" else d + 16
        # the weights (and positions) of all slots in, of the kept ones out; every hole's row in and out
        moved = c["keep"] * max(0.0, n - c["keep"]) / n
        units = B * h_kv
        per_slot = 8 if c["positions"] else 4
        return {"bytes": units * (n * per_slot + min(n, c["keep"]) * 8 + 2 * moved * row), "flops": units * n}
    h = c["h"]
    keys = B * h_kv * _mean_length(c, 1, c["L_max"])
    row = d + 16 if op == "decode4" else 4 * d
    weights = 8 if op == "weighted" or c["weights"] else 0
    small = B * 2 * h * d * 2 + B * h * d * 2 + (B + h) * c["d_model"] * 2
    return {"bytes": keys * (row + weights) + small, "flops": keys * (2 * h / h_kv) * d * 4}


# ------------------------------------------------------------------ exact ---
def _values64(x):
    """What the 4-bit form of rows x [n, d] stands for, from its definition in 64 bits."""
    n, d = x.shape
    g = x.double().reshape(n * 2, d // 2)
    lo, hi = torch.aminmax(g, dim=1)
    s = ((hi - lo) / 15).float().to(BF16).double()
    code = torch.round((g - lo[:, None]) / s[:, None]).clamp(max=15)
    code[s == 0] = 0
    v = s[:, None] * code + lo[:, None]
    v[~torch.isfinite(s)] = torch.nan
    return v.reshape(n, d)


def _record64(rec):
    """The key and value rows of records [n, d + 16], in 64 bits."""
    rec = rec.contiguous()
    n, d = rec.shape[0], rec.shape[1] - 16
    rows = []
    for i in (0, 1):
        byte = rec[:, i * d // 2:(i + 1) * d // 2].to(torch.int16)
        v = torch.empty((n, d), dtype=torch.float64, device=rec.device)
        v[:, 0::2], v[:, 1::2] = (byte % 16).double(), (byte // 16).double()
        p = rec[:, d + 8 * i:d + 8 * i + 8].contiguous().view(BF16).double()
        for half in (0, 1):
            v[:, half * d // 2:(half + 1) * d // 2] *= p[:, half:half + 1]
            v[:, half * d // 2:(half + 1) * d // 2] += p[:, 2 + half:3 + half]
        rows.append(v)
    return rows


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    B, h_kv, d, L_max, op = c["B"], c["h_kv"], c["d"], c["L_max"], c["op"]
    if op in ("append", "read"):
        outs = [s["k_out"].double(), s["v_out"].double()]
        for b in range(B):
            n, first = int(s["counts"][b]), int(s["start"][b])
            if n == 0:
                continue
            if op == "append":
                rows = [_values64(s[x][b, :n].reshape(n * h_kv, d)) for x in ("k", "v")]
                s["weights"][b, :, first:first + n] = 0
                s["positions"][b, :, first:first + n] = torch.arange(first, first + n, device=DEV).int()
            else:
                rows = _record64(s["cache"][b, first:first + n].reshape(n * h_kv, d + 16))
            for o, r in zip(outs, rows):
                o[b, :n] = r.reshape(n, h_kv, d)
        return (*outs, s["weights"].double(), s["positions"]) if op == "append" else tuple(outs)
    if op == "evict":
        return _exact_evict(s, c)
    h = c["h"]
    G = 2 * h // h_kv
    out = torch.zeros((B, h, d), dtype=torch.float64, device=DEV)
    gathered = None if s["weights_out"] is None else s["weights_out"].double()
    for b in range(B):
        n = int(s["seqlens"][b])
        if s["gate"] is None:
            gate = torch.sigmoid((s["x"][b].double()[:, None] * s["w_lambda"].double()).sum(0))
        else:
            gate = s["gate"][b].double()
        for g in range(h_kv):
            if op == "decode4":
                k, v = _record64(s["cache"][b, :n, g])
            else:
                k, v = s["k"][b, :n, g].double(), s["v"][b, :n, g].double()
            a = torch.softmax(s["q"][b, g * G:(g + 1) * G].double() @ k.T * d ** -0.5, dim=-1)
            diff = a[0::2] - gate[g * G // 2:(g + 1) * G // 2, None] * a[1::2]
            out[b, g * G // 2:(g + 1) * G // 2] = diff @ v
            if gathered is not None:
                gathered[b, g, :n] = s["weights"][b, g, :n].double() + diff.abs().sum(0)
    return out if gathered is None else (out, gathered)


def _exact_evict(s, c):
    lengths = s["seqlens"].tolist()
    w_out, p_out, n_out = s["weights_out"].double(), s["positions_out"].clone(), s["seqlens_out"].clone()
    rows = _rows_out(s)
    moved = [r.clone() for r in rows]
    for b, n in enumerate(lengths):
        m = min(n, c["keep"])
        n_out[b] = m
        end = n if s["next"] is None else int(s["next"][b])
        for g in range(c["h_kv"]):
            w = s["weights"][b, g, :n].double()
            at = torch.arange(n, device=DEV)
            p = at if s["positions"] is None else s["positions"][b, g, :n].long()
            rank = w.clone()
            rank[(p < c["sinks"]) | (p >= end - c["recent"])] = torch.inf
            # the (n - m) least, of equal ones the highest slots
            gone = torch.argsort(rank.flip(0), stable=True)[:n - m]
            stays = torch.ones(n, dtype=torch.bool, device=DEV)
            stays[n - 1 - gone] = False
            frm = at[:m].clone()
            frm[~stays[:m]] = at[m:][stays[m:]]
            w_out[b, g, :m], p_out[b, g, :m] = w[frm], p[frm].int()
            for r, o in zip(rows, moved):
                if r.dtype == BF16:
                    o[b, :m, g] = r[b, frm, g]
                else:
                    o[b, g, :m] = r[b, g, frm]
    return (*[o.double() if o.dtype == BF16 else o for o in moved], w_out, p_out, n_out)
