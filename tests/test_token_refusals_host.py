"""Refusals of the exact token cache's calls that need no GPU."""
import ctypes

import pytest
import torch

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


def test_rotary_out_records_no_gradient(R):
    """With `out` no gradient could be recorded: refused rather than lost."""
    x = torch.zeros(1, 2, 3, 128)
    pos = torch.zeros(1, 2, dtype=torch.int32)
    t = R.RotaryTable.make(128, device="cpu")
    leaf = x.clone().requires_grad_()
    for a, out in ((leaf, torch.zeros_like(x)), (x, leaf), (leaf, leaf), (leaf * 1, x)):
        with pytest.raises(ValueError, match="gradient"):
            R.rotary(a, pos, t, out=out)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # past the check
            R.rotary(a, pos, t, out=out)
