"""Plain fp64 definitions of the serving-cache operators: the 4-bit record form
of a key/value row, the weight that cached keys gather in a V2 decode step,
and eviction by gathered weight.  Nothing is shared with the GPU path.

A row of d features has two groups of d/2; a group stores its minimum m, its
scale s = bf16((max - min) / 15) and codes n = rint((x - m) / s) in 0..15; it
stands for s n + m.  s = 0: codes 0.  s not finite: s = m = NaN, codes 0.
max - min and x - m are rounded to fp32, as the definition has it.
"""

from __future__ import annotations

import numpy as np

from .diffattn_oracle import attention_maps


def round_bf16(x):
    """fp64 -> the nearest bf16 value (ties to even), as fp64."""
    with np.errstate(over="ignore"):
        f = np.asarray(x, np.float64).astype(np.float32)
    u = f.view(np.uint32)
    r = ((u >> 16) & 1) + np.uint32(0x7FFF)
    with np.errstate(over="ignore"):
        v = ((u + r) & np.uint32(0xFFFF0000)).view(np.float32)
    return np.where(np.isfinite(f), v, f).astype(np.float64)


def bf16_bits(x):
    """The bits of values that bf16 holds exactly (NaN: 0x7fff)."""
    f = np.asarray(x, np.float64).astype(np.float32)
    return np.where(np.isnan(f), np.uint16(0x7FFF), (f.view(np.uint32) >> 16).astype(np.uint16))


def kv4_quantise(x):
    """x [..., d] -> codes [..., d] (uint8), s, m [..., 2]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], 2, x.shape[-1] // 2)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        m = g.min(-1)
        s = round_bf16((g.max(-1) - m).astype(np.float32).astype(np.float64) / 15)
        bad = ~np.isfinite(s)
        above = (g - m[..., None]).astype(np.float32).astype(np.float64)
        n = np.minimum(np.rint(above / s[..., None]), 15)
        n = np.where((s == 0)[..., None] | bad[..., None], 0, n)
    s, m = np.where(bad, np.nan, s), np.where(bad, np.nan, m)
    return n.reshape(x.shape).astype(np.uint8), s, m


def kv4_pack(k, v):
    """Records [..., d + 16] (uint8) of key and value rows [..., d]."""
    codes, params = [], []
    for x in (k, v):
        n, s, m = kv4_quantise(x)
        codes.append(n[..., 0::2] | (n[..., 1::2] << 4))
        bits = np.ascontiguousarray(bf16_bits(np.concatenate([s, m], -1)).astype("<u2"))
        params.append(bits.view(np.uint8))
    return np.concatenate(codes + params, -1)


def kv4_values(rec):
    """The key and value rows [..., d] (fp64) that records [..., d + 16] stand for."""
    rec = np.asarray(rec, np.uint8)
    d = rec.shape[-1] - 16
    rows = []
    for i in (0, 1):
        c = rec[..., i * (d // 2):(i + 1) * (d // 2)]
        n = np.stack([c & 15, c >> 4], -1).reshape(*rec.shape[:-1], 2, d // 2).astype(np.float64)
        bits = np.ascontiguousarray(rec[..., d + 8 * i:d + 8 * i + 8]).view("<u2").astype(np.uint32) << 16
        p = bits.view(np.float32).astype(np.float64)
        rows.append((n * p[..., 0:2, None] + p[..., 2:4, None]).reshape(*rec.shape[:-1], d))
    return rows


def key_weights(q, k, gate, scale=None):
    """What each of the keys gathers in one decode step of one sequence.
    q [2h, d]; k [L, h_kv, d]; gate [h].  Returns (w [h_kv, L], both maps'
    total [h_kv, L]): sum over pairs of |A_2p - g A_2p+1| and of A_2p + |g| A_2p+1."""
    q, k, gate = (np.asarray(t, np.float64) for t in (q, k, gate))
    H2, d = q.shape
    L, hkv = k.shape[:2]
    G = H2 // hkv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    w, total = np.zeros((hkv, L)), np.zeros((hkv, L))
    for p in range(H2 // 2):
        g = 2 * p // G
        a, _ = attention_maps(q[2 * p:2 * p + 2], k[:, g], scale, causal=False)
        w[g] += np.abs(a[0] - gate[p] * a[1])
        total[g] += a[0] + np.abs(gate[p]) * a[1]
    return w, total


def evict(weights, keep, *, sinks=0, recent=0, positions=None, next_position=None):
    """Eviction of one head's L slots.  Returns (m, source): after it, slot i <
    m holds what slot source[i] held."""
    w = [float(x) for x in weights]
    L = len(w)
    pos = list(range(L)) if positions is None else [int(x) for x in positions]
    end = L if next_position is None else int(next_position)
    m = min(L, keep)

    def rank(j):
        if pos[j] < sinks or pos[j] >= end - recent:
            return (2, 0.0)
        return (1, 0.0) if w[j] != w[j] else (0, w[j])

    order = sorted(range(L), key=lambda j: (-rank(j)[0], -rank(j)[1], j))
    stays = set(order[:m])
    late = iter(sorted(j for j in stays if j >= m))
    return m, [j if j in stays else next(late) for j in range(m)]
