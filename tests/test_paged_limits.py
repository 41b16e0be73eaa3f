"""Sizes at which counts in 32 bits would end, refused before anything is launched
(no GPU: pointers are never dereferenced)."""

import pytest

from differential_attention_diff_gb300 import binding as bd
from test_paged_abi import FAKE, OK, UNS, WS, cache, t3, with_


@pytest.mark.parametrize("B,attend,append", [(2 ** 20, WS, OK), (2 ** 20 + 1, UNS, OK), (2 ** 30, UNS, OK),
                                             (2 ** 30 + 1, UNS, UNS), (2 ** 31 - 1, UNS, UNS)])
def test_sequences(lib, B, attend, append):
    """2^20 sequences may attend (what is left is refused for the lack of a workspace), 2^30 be appended to (nothing, here)."""
    kw = {"cache.B": B, "cache.max_pages": 1}
    p = bd.da_v2_paged_fwd_params(cache(), 4, 0, 0, 0.0, t3(), FAKE, None, None, t3(), None, 0)
    assert lib.diffattn_v2_paged_fwd(with_(p, kw), None) == attend
    p = bd.da_paged_append_params(cache(), 8, 128, 0, FAKE, 1.0, 1, 1e-5, FAKE, FAKE, None, t3(), t3(), t3(), t3())
    assert lib.diffattn_paged_append(with_(p, dict(kw, **{"cache.T": 0})), None) == append
