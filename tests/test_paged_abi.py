"""Refusals of the rotation, paged append and paged attention, before anything
is launched (no GPU: pointers are never dereferenced)."""

import ctypes as C

import pytest

from differential_attention_diff_gb300 import binding as bd

FAKE = 1 << 20
INV, UNS, WS, CU, OK = bd.DA_ERR_INVALID_ARG, bd.DA_ERR_UNSUPPORTED, bd.DA_ERR_WORKSPACE, bd.DA_ERR_CUDA, bd.DA_OK


def with_(p, kw):
    q = type(p).from_buffer_copy(p)
    for name, v in kw.items():
        o = q
        *path, last = name.split(".")
        for n in path:
            o = getattr(o, n)
        setattr(o, last, v)
    return C.byref(q)


def t4(off=0, sb=1 << 16, sn=1 << 10, sh=128):
    return bd.da_t4(FAKE + off, sb, sn, sh)


def t3(off=0, st=1 << 10, sh=128):
    return bd.da_t3(FAKE + off, st, sh)


def rope():
    return bd.da_qk_rope_fwd_params(2, 5, 8, 2, 128, bd.DA_BF16, 128, 0, FAKE, 1.0, 1, 1e-5, FAKE, FAKE, FAKE, t4(), t4(),
                                    t4(), t4())


def cache():
    return bd.da_paged_cache(2, 5, 2, 128, 16, 10, 4, t4(), t4(), FAKE, FAKE, FAKE)


ROPE = [(dict(B=-1), INV), (dict(h_q=-1), INV), (dict(dtype=5), INV), (dict(d=96), UNS), (dict(rot_dim=136), INV),
        (dict(rot_dim=-8), INV), (dict(rot_dim=12), UNS), (dict(inv_freq=None), INV), (dict(inv_freq=FAKE + 2), INV),
        (dict(rope_scale=float("inf")), INV), (dict(norm_eps=-1.0), INV), (dict(norm_eps=float("nan")), INV),
        (dict(q_weight=FAKE + 2), INV), (dict(positions=FAKE + 1), INV), (dict(B=1 << 16, N=1 << 16), UNS),
        (dict(B=1 << 15, N=(1 << 14) + 1), UNS),
        (dict(B=0), OK), (dict(N=0), OK), (dict(h_q=0, h_k=0), OK)]


@pytest.mark.parametrize("kw,want", ROPE + [
    (dict(q=bd.da_t4(None, 0, 0, 0)), INV), (dict(q=t4(8)), INV), (dict(k_out=t4(sn=100)), INV), (dict(k=t4(sb=-8)), INV)])
def test_rope_fwd(lib, kw, want):
    assert lib.diffattn_qk_rope_fwd(with_(rope(), kw), None) == want


def test_rope_not_looked_at(lib):
    """Without heads, norm or rotation their arguments are not checked: what is left is refused for the lack of a
    device here, or runs; nothing is launched for empty calls."""
    for kw in (dict(h_q=0, q=bd.da_t4(None, 0, 0, 0), N=0), dict(norm=0, q_weight=FAKE + 2, norm_eps=-1.0, N=0),
               dict(rot_dim=0, inv_freq=None, N=0)):
        assert lib.diffattn_qk_rope_fwd(with_(rope(), kw), None) == OK


@pytest.mark.parametrize("kw,want", [({"fwd." + k: v for k, v in kw.items()}, want) for kw, want in ROPE if want != OK] + [
    (dict(dq_out=t4(8)), INV), (dict(dk=bd.da_t4(None, 0, 0, 0)), INV), ({"fwd.q": bd.da_t4(None, 0, 0, 0)}, INV),
    (dict(dq_weight=FAKE + 2), INV), ({"fwd.norm": 0}, INV), (dict(), WS), (dict(workspace=FAKE, workspace_bytes=64), WS),
    (dict(workspace=FAKE + 64, workspace_bytes=1 << 30), WS)])
def test_rope_bwd(lib, kw, want):
    p = bd.da_qk_rope_bwd_params(rope(), t4(), t4(), t4(), t4(), FAKE, FAKE, None, 0)
    assert lib.diffattn_qk_rope_bwd(with_(p, kw), None) == want
    assert lib.diffattn_qk_rope_bwd(None, None) == INV and lib.diffattn_qk_rope_fwd(None, None) == INV


CACHE = [({"cache.B": -1}, INV), ({"cache.T": -1}, INV), ({"cache.h_kv": 0}, INV), ({"cache.d": 96}, UNS),
         ({"cache.page_size": 0}, INV), ({"cache.n_pages": -1}, INV), ({"cache.page_size": 1 << 20, "cache.max_pages": 1 << 20}, UNS),
         ({"cache.B": 1 << 16, "cache.max_pages": 1 << 20, "cache.page_size": 16}, UNS),
         ({"cache.cu_seqlens": None}, INV), ({"cache.seqlens": FAKE + 2}, INV), ({"cache.block_table": None}, INV),
         ({"cache.k_pages": bd.da_t4(None, 0, 0, 0)}, INV), ({"cache.v_pages": t4(8)}, INV), ({"cache.k_pages": t4(sh=100)}, INV),
         ({"cache.T": 0}, OK), ({"cache.B": 0}, OK)]


@pytest.mark.parametrize("kw,want", CACHE + [
    (dict(h_q=-1), INV), (dict(h_q=1 << 25), UNS), ({"cache.T": (1 << 29) + 1}, UNS), (dict(rot_dim=12), UNS),
    (dict(inv_freq=None), INV), (dict(norm_eps=-1.0), INV), (dict(positions=FAKE + 2), INV),
    (dict(k=t3(8)), INV), (dict(v=bd.da_t3(None, 0, 0)), INV), (dict(q=t3(8)), INV), (dict(q_out=bd.da_t3(None, 0, 0)), INV),
    (dict(v=t3(sh=4)), INV)])
def test_paged_append(lib, kw, want):
    p = bd.da_paged_append_params(cache(), 8, 128, 0, FAKE, 1.0, 1, 1e-5, FAKE, FAKE, None, t3(), t3(), t3(), t3())
    assert lib.diffattn_paged_append(with_(p, kw), None) == want
    assert lib.diffattn_paged_append(None, None) == INV


@pytest.mark.parametrize("kw,want", CACHE + [
    (dict(h=0), INV), ({"h": 7, "cache.h_kv": 3}, INV), ({"h": 3, "cache.h_kv": 2}, INV), (dict(h=192), UNS), (dict(max_new=-1), INV),
    ({"cache.page_size": 8}, UNS), ({"cache.page_size": 24}, UNS), ({"cache.T": 1 << 30}, UNS),
    ({"cache.max_pages": 0}, INV), ({"cache.n_pages": 0}, INV), ({"cache.k_pages": t4(sh=0)}, INV), ({"cache.v_pages": t4(sh=136)}, UNS),
    (dict(q=t3(8)), INV), (dict(q=t3(sh=0)), INV), (dict(out=bd.da_t3(None, 0, 0)), INV), (dict(out=t3(st=4)), INV),
    (dict(gate=FAKE + 2), INV), (dict(gate=None), INV), (dict(gate=None, x=FAKE, w_lambda=FAKE, d_model=100), UNS),
    (dict(gate=None, x=FAKE + 8, w_lambda=FAKE, d_model=128), INV), (dict(), WS),
    (dict(workspace=FAKE, workspace_bytes=4096), WS), (dict(workspace=FAKE + 8, workspace_bytes=1 << 40), WS)])
def test_paged_fwd(lib, kw, want):
    p = bd.da_v2_paged_fwd_params(cache(), 4, 0, 0, 0.0, t3(), FAKE, None, None, t3(), None, 0)
    assert lib.diffattn_v2_paged_fwd(with_(p, kw), None) == want
    assert lib.diffattn_v2_paged_fwd(None, None) == INV


def test_workspace_sizes(lib):
    size = lib.diffattn_v2_paged_fwd_workspace_size
    a = size(64, 64, 1, 32, 8, 128, 1)
    assert a > 0 and size(64, 64, 1, 32, 8, 128, 0) >= a + 64 * 32 * 4
    assert size(0, 64, 1, 32, 8, 128, 1) == 0 and size(64, 64, 1, 7, 3, 128, 1) == 0 and size(4, 2, 0, 256, 2, 64, 1) == 0
    assert lib.diffattn_qk_rope_bwd_workspace_size(1, 1, 1, 1, 64) > 0
    assert lib.diffattn_qk_rope_bwd_workspace_size(0, 1, 1, 1, 64) == 0
