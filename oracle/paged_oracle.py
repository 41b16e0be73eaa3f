"""64-bit definitions of the norm and rotation of queries and keys, the paged
cache and the V2 attention over it (numpy; see include/diffattn.h)."""

import numpy as np


def angles(positions, inv_freq):
    """position * frequency, [..., rot / 2]: frequencies as the fp32 numbers that they are.  Exact to 2^-52 of a
    turn of the product, which is why far positions are not a problem here."""
    return np.asarray(positions, np.float64)[..., None] * np.asarray(inv_freq, np.float32).astype(np.float64)


def rotate(z, ang, rot, interleaved, scale=1.0):
    """Rows z [..., heads, d] turned by angles [..., rot / 2]."""
    y = np.array(z, np.float64)
    c, s = np.cos(ang)[..., None, :] * scale, np.sin(ang)[..., None, :] * scale
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    zu, zv = np.array(y[..., u]), np.array(y[..., v])
    y[..., u], y[..., v] = zu * c - zv * s, zv * c + zu * s
    return y


def norm(x, w, eps):
    z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return z if w is None else z * w


def qk_rope(x, inv_freq, positions, rot, interleaved=False, scale=1.0, do_norm=False, eps=1e-5, w=None):
    z = norm(x, w, eps) if do_norm else x
    return rotate(z, angles(positions, inv_freq), rot, interleaved, scale) if rot else np.array(z)


def qk_rope_bwd(x, dy, inv_freq, positions, rot, interleaved=False, scale=1.0, do_norm=False, eps=1e-5, w=None):
    """(dx, dw): the chain rule, dw summed over every row (None without norm)."""
    dz = rotate(dy, -angles(positions, inv_freq), rot, interleaved, scale) if rot else np.array(dy)
    if not do_norm:
        return dz, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dw = (dz * xh).reshape(-1, x.shape[-1]).sum(0)
    g = dz if w is None else dz * w
    return r * (g - xh * (g * xh).mean(-1, keepdims=True)), dw


def gather(pages, table, L):
    """The first L rows [L, h_kv, d] of the sequence whose pages `table` names (pages [n, size, h_kv, d]); pages that
    there are not are zeros."""
    n, size = pages.shape[:2]
    out = np.zeros((L, *pages.shape[2:]))
    for j in range(L):
        p = table[j // size]
        if 0 <= p < n:
            out[j] = pages[p, j % size]
    return out


def attend(q, k, v, gate, n_keys, scale=None, sizes=False):
    """V2 attention of tokens q [n, 2h, d] over keys k, v [L, h_kv, d]; token i sees the first n_keys[i].  With
    `sizes` also what errors of the weights are relative to: sum A_2p |v| + |gate| sum A_2p+1 |v|."""
    n, h2, d = q.shape
    G = h2 // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, size = np.zeros((n, h2, v.shape[-1])), np.zeros((n, h2, v.shape[-1]))
    hidden = np.arange(k.shape[0])[None, :] >= np.asarray(n_keys)[:, None]
    for j in range(h2):
        t = q[:, j] @ k[:, j // G].T * scale
        t[hidden] = -np.inf
        e = np.exp(t - t.max(-1, keepdims=True))
        a = e / e.sum(-1, keepdims=True)
        o[:, j], size[:, j] = a @ v[:, j // G], a @ np.abs(v[:, j // G])
    out = o[:, 0::2] - gate[..., None] * o[:, 1::2]
    return (out, size[:, 0::2] + np.abs(gate)[..., None] * size[:, 1::2]) if sizes else out
