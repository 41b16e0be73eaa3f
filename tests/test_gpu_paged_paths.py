"""V2 attention over a paged cache, where its paths part: several turns of the
CTAs over a long prompt's shares, and a running maximum that is raised in each
of the kernels for few tokens.  Bars as in test_gpu_paged.py."""

import numpy as np
import pytest
import torch

from differential_attention_diff_gb300 import binding as bd
from test_gpu_paged import BF16, U, call, check, gen, i32, make, randn

pytestmark = pytest.mark.gpu
TILE, ITEM = 128, 3  # keys of a tile; what an item costs beside its tiles, in tiles


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert bd.diffattn_get_device_status() == bd.DA_OK


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def long_batch(n, L, page, h, hkv, d, max_pages, seed):
    """As `make`, by whole pages: long caches are filled on the device at once."""
    g = gen(seed)
    count = sum(-(-x // page) for x in L) + 2
    order = torch.randperm(count, generator=g, device="cuda").int()
    table = torch.full((len(n), max_pages), -1, dtype=torch.int32, device="cuda")
    pages, at = [randn((count, page, hkv, d), g) for _ in range(2)], 0
    for b, x in enumerate(L):
        used = -(-x // page)
        table[b, :used] = order[at:at + used]
        at += used
        if x % page:
            for t in pages:
                t[table[b, used - 1].long(), x % page:] = float("nan")
    T = sum(n)
    return dict(q=randn((T, 2 * h, d), g), k=pages[0], v=pages[1], table=table, cu=i32(np.cumsum([0] + n)), sl=i32(L),
                gate=torch.rand((T, h), generator=g, device="cuda"), n=n, L=L)


def check_on_device(t, out):
    """`check` with the 64-bit definition computed on the device, every token of every head."""
    d, hkv = t["q"].shape[-1], t["k"].shape[2]
    G, t0 = t["q"].shape[1] // hkv, 0
    for b, (n, L) in enumerate(zip(t["n"], t["L"])):
        used = t["table"][b, :-(-L // t["k"].shape[1])].long()
        k, v = (t[x][used].flatten(0, 1)[:L].double() for x in ("k", "v"))
        q, gate, got = (x[t0:t0 + n].double() for x in (t["q"], t["gate"], out))
        hidden = torch.arange(L, device="cuda") > torch.arange(L - n, L, device="cuda")[:, None]
        for p in range(G * hkv // 2):
            j = 2 * p // G
            o = []
            for x in (2 * p, 2 * p + 1):
                e = 64 * U * (1 + d ** -0.5 * (q[:, x].abs() * k[:, j].abs().amax(0)).sum(-1, keepdim=True))
                a = torch.softmax((q[:, x] @ k[:, j].T * d ** -0.5).masked_fill(hidden, -torch.inf), -1)
                o.append((a @ v[:, j], a @ v[:, j].abs(), e))
            g = gate[:, p:p + 1]
            ref, size, e = o[0][0] - g * o[1][0], o[0][1] + g * o[1][1], torch.maximum(o[0][2], o[1][2])
            err = (got[:, p] - ref).abs()
            bar = (2.0 ** -8 + 2.0 ** -16 + 2 * e) * size + 2.0 ** -8 * ref.abs()
            assert bool((err <= bar).all()), (b, p, float((err / bar).max()))
        t0 += n


@pytest.mark.parametrize("d,n,L,turns", [
    (128, [260, 5, 150, 300], [9000, 300, 12000, 10000], 2),
    (128, [260, 150, 3, 300], [17000, 16300, 200, 18000], 4),
    (64, [300, 150, 4, 260], [18000, 24000, 500, 20000], 2),
    (64, [260, 2, 150, 300], [34000, 130, 32600, 36000], 4),
])
def test_turns_of_the_ctas(d, n, L, turns):
    """Long prompts whose keys do not fit L2, read for many items: the CTAs take several shares each.  That the sizes
    get there is computed as the launch and the kernel do: the host allows several turns, the lengths ask for `turns`,
    a sequence is shorter than a share, and some item is cut between two turns."""
    h, hkv, page = 128, 8, 128
    tq, C, max_pages = 2 * (128 // (2 * h // hkv)), sms(), max(L) // page + 1
    t = long_batch(n, L, page, h, hkv, d, max_pages, seed=d + turns)
    assert sum(n) // tq * hkv >= 4 * C and len(n) * max_pages * page * hkv * d * 4 >= 96 << 20
    units = [[-(-min(x - m + (i + 1) * tq, x) // TILE) + ITEM for i in range(-(-m // tq))] for m, x in zip(n, L)]
    line = [u for s in units for _ in range(hkv) for u in s]
    total = sum(line)
    assert min(sum(L) * hkv * d * 4 // (48 << 20), total // (C * 128), 4) == turns
    share, more = divmod(total, turns * C)
    assert min(sum(s) * hkv for s in units) < share
    starts = np.cumsum([0] + line)
    cuts = [c * share + min(c, more) for c in range(C, turns * C, C)]
    assert any(x - starts[np.searchsorted(starts, x, "right") - 1] > ITEM for x in cuts)
    out = torch.full((sum(n), h, d), 7.0, dtype=BF16, device="cuda")
    call(t, out=out)
    check_on_device(t, out)
    again = call(t)
    assert torch.equal(again, out)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 8), (2, 8), (4, 8), (1, 32), (3, 10), (16, 2)])  # 8, 16 and 32 columns
@pytest.mark.parametrize("where", ["cut", "whole"])
def test_scores_that_grow_for_few_tokens(n, G, d, page, where):
    """Scores far above the first tile's, in the instance for each number of columns: for all of them, and for the
    tokens (or heads) of either half only, so that one warpgroup of two raises its maxima and the other does not."""
    if where == "cut":  # few sequences: every item is cut
        L = [1500, 1333]
    else:  # as many units to each CTA as two items have: none is cut
        L = [600] * (2 * sms())
    t = make([n] * len(L), L, page, G // 2, 1, d, seed=d + n)
    if where == "whole":
        assert G * n <= 32 and (5 + ITEM) * len(L) % sms() == 0 and (5 + ITEM) * len(L) // sms() == 2 * (5 + ITEM)
    for b, x in enumerate(L):
        j = torch.arange(x, device="cuda")
        at = (t["table"][b].long()[j // page], j % page)
        t["k"][at] = t["k"][at] * torch.linspace(0.0, 40.0, x, device="cuda").to(BF16)[:, None, None]
    q = t["q"]
    columns = torch.arange(n * G, device="cuda").reshape(n, G).repeat(len(L), 1)[..., None]
    for which in ("all", "first", "last"):
        quiet = dict(all=columns < 0, first=columns >= n * G // 2, last=columns < n * G // 2)[which]
        t["q"] = torch.where(quiet, q * 2.0 ** -6, q)
        check(t, call(t, max_new=n), only=(0, 1, len(L) // 2, len(L) - 1), tag=which)
