"""Refusals of the exact token cache's calls that need no GPU."""
import ctypes

import pytest

PTR = 1 << 20  # an aligned address that no refused call may touch
INVALID, WORKSPACE = 1, 3


@pytest.fixture(scope="module")
def R():
    import kv_cache_vector_segmented_b200 as R
    return R


@pytest.fixture(scope="module")
def C():
    from kv_cache_vector_segmented_b200 import _tokens
    return _tokens


def test_wait_selftest_refusals(R, C):
    lib, b = R.lib, ctypes.byref
    c = C.CTokenCache(2, 2, 4, 128, 64, PTR, 2 * PTR, 3 * PTR, 4 * PTR, 5 * PTR)
    good = C.CTokenPrefix(PTR, PTR, 10, 0, 128, 1280)
    need = lib.ri_token_attend_workspace(b(c), 10)

    def call(p=good, hand_off=1, limit=1000, q=PTR, n=need):
        return lib.ri_selftest_token_attend_timeout(b(c), q, None if p is None else b(p), PTR,
                                                    None, 1, PTR, n, hand_off, limit, None)
    for kw in (dict(p=None), dict(p=C.CTokenPrefix(PTR, PTR, 0, 0, 128, 1280)),
               dict(hand_off=0), dict(hand_off=3), dict(limit=0), dict(limit=10 ** 10 + 1),
               dict(q=None)):
        assert call(**kw) == INVALID, kw
    assert call(n=need - 1) == WORKSPACE
