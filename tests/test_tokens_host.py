"""Rotary tables and the exact token cache without a GPU: tables against the
formulas, the oracle against a library or by hand, argument refusals of the C
ABI and of the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import token_cache as T


@pytest.fixture(scope="module")
def R():
    import kv_cache_vector_segmented_b200 as R
    return R


@pytest.fixture(scope="module")
def C():
    from kv_cache_vector_segmented_b200 import _tokens
    return _tokens


INVALID, UNSUPPORTED, WORKSPACE, CAPACITY = 1, 2, 3, 4
PTR = 1 << 20  # an aligned address that no refused call may touch


# ------------------------------------------------------------------- tables
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "bands", "yarn"])
@pytest.mark.parametrize("n", [2, 20, 64, 128, 256])
def test_table_matches_formula(R, scaling, n):
    t = R.RotaryTable.make(n, base=500000.0, scaling=scaling, factor=8.0, original_len=8192,
                           device="cpu")
    f, mag = T.frequencies(n, 500000.0, scaling, 8.0, 8192)
    got = t.frequencies.numpy()
    # both are a handful of fp64 operations on the same formula
    assert np.allclose(got, f, rtol=1e-13, atol=0)
    assert t.magnitude == pytest.approx(mag, rel=1e-6)
    turns = t.turns.numpy().astype(np.uint64).astype(np.float64) / 2.0 ** 64
    assert np.allclose(turns * 2 * math.pi, f, rtol=1e-12, atol=1e-18)


def test_fixed_point_turns_are_exact_far_out(R):
    """position * turns mod 2^64 against exact rational arithmetic."""
    from fractions import Fraction
    t = R.RotaryTable.make(128, base=500000.0, device="cpu")
    two_pi = Fraction("6.28318530717958647692528676655900576839")
    for i in (0, 1, 31, 63):
        turn = Fraction(float(t.frequencies[i])) / two_pi
        for pos in (1, 131071, 2 ** 31 - 1, -7, -2 ** 31):
            want = (turn * pos) % 1
            got = Fraction((int(t.turns.numpy().astype(np.uint64)[i]) * pos) % 2 ** 64, 2 ** 64)
            err = abs(want - got)
            # half a unit of 2^-64 per step; long double's pi adds 2^-63 relative
            assert min(err, 1 - err) <= Fraction(abs(pos) * 2, 2 ** 64) + abs(turn * pos) / 2 ** 60


def test_rotary_layouts_agree_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    f = np.array([math.pi / 2, math.pi])
    assert np.allclose(T.rotary(x, np.array([1]), f), [[[-3, -2, 1, -4, 9]]])
    assert np.allclose(T.rotary(x, np.array([1]), f, interleaved=True), [[[-2, 1, -3, -4, 9]]])
    back = T.rotary(T.rotary(x, np.array([5]), f, 2.0), np.array([5]), f, 2.0, inverse=True)
    assert np.allclose(back[..., :4], 4 * x[..., :4])


def test_oracle_attend_matches_library():
    g = torch.Generator().manual_seed(3)
    q, K, V = (torch.randn(n, 128, generator=g, dtype=torch.float64) for n in (4, 50, 50))
    out, lse, w, a = T.attend(q.numpy(), K.numpy()[20:], V.numpy()[20:], K.numpy()[:20],
                              V.numpy()[:20])
    want = torch.nn.functional.scaled_dot_product_attention(q[None], K[None], V[None])[0]
    s = (q @ K.T / math.sqrt(128))
    assert np.allclose(out, want.numpy(), atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(s, 1).numpy(), atol=1e-12)
    assert np.allclose(w, torch.softmax(s, 1)[:, 20:].sum(0).numpy(), atol=1e-12)
    assert (a >= np.abs(out) - 1e-12).all()


def test_oracle_evict_by_hand():
    pos = np.array([10, 0, 11, 3, 12, 5, 7])
    w = np.array([0.1, 0.0, 0.0, 0.9, 0.0, 0.5, 0.9])
    # held: position 0 (first) and 12 (newest); then rows 3 and 6 (0.9)
    assert T.evict(pos, w, 4, 1, 1).tolist() == [4, 1, 6, 3]
    # ties go to the lower row; NaN is last
    assert T.evict(pos, np.array([1, 1, 1, 1, 1, np.nan, 1.0]), 3, 0, 0).tolist() == [0, 1, 2]
    assert T.evict(pos, np.array([np.nan] * 6 + [0.0]), 1, 0, 0).tolist() == [6]
    assert T.evict(pos, w, 9, 0, 0).tolist() == list(range(7))


# ----------------------------------------------------------------- refusals
@pytest.mark.parametrize("field,value", [
    ("rotary_dim", 0), ("rotary_dim", 3), ("rotary_dim", 258), ("scaling", 5), ("scaling", -1),
    ("base", 1.0), ("base", math.nan), ("base", math.inf), ("factor", 0.0), ("factor", math.nan),
    ("factor", 1e-9), ("original_len", 0), ("low", 0.0), ("low", 5.0), ("high", math.inf),
    ("reserved", 1)])
def test_table_refusals(R, field, value):
    cfg = R.RotaryConfig(128, 3, 8192, 0, 500000.0, 8.0, 1.0, 4.0)
    setattr(cfg, field, value)
    turns = (ctypes.c_uint64 * 128)()
    mag = ctypes.c_double(7.0)
    assert R.lib.ri_rotary_table(ctypes.byref(cfg), turns, None, ctypes.byref(mag)) == INVALID
    assert mag.value == 7.0 and not any(turns)


def _cache(C, **over):
    v = dict(batch=2, num_kv_heads=2, group_size=4, head_dim=128, capacity=64, K=PTR,
             V=2 * PTR, pos=3 * PTR, weight=4 * PTR, lens=5 * PTR)
    v.update(over)
    return C.CTokenCache(*[v[f] for f, _ in C.CTokenCache._fields_])


BAD_CACHES = [dict(batch=0), dict(num_kv_heads=0), dict(capacity=0), dict(group_size=0),
              dict(group_size=9), dict(head_dim=64), dict(K=None), dict(V=None), dict(pos=None),
              dict(weight=None), dict(lens=None), dict(K=PTR + 8), dict(weight=PTR + 4)]


@pytest.mark.parametrize("over", BAD_CACHES)
def test_cache_refusals(R, C, over):
    lib, c = R.lib, _cache(C, **over)
    h = C.CHeads(PTR, 512, 256, 128)
    b = ctypes.byref
    assert lib.ri_token_append(b(c), 1, b(h), b(h), PTR, 1, None, None, None, PTR, PTR,
                               None) == INVALID
    assert lib.ri_token_attend(b(c), PTR, None, PTR, None, 1, PTR, 1 << 30, None) == INVALID
    assert lib.ri_token_evict(b(c), 8, 0, 0, b(c), PTR, 1 << 30, None) == INVALID
    assert lib.ri_last_error()


def test_size_limits(R, C):
    lib, b = R.lib, ctypes.byref
    assert lib.ri_token_attend_workspace(b(_cache(C, batch=65537, num_kv_heads=1)), 0) == 0
    assert lib.ri_token_attend_workspace(b(_cache(C, capacity=(1 << 28) + 1)), 0) == 0
    assert lib.ri_token_attend_workspace(b(_cache(C)), -1) == 0
    many = _cache(C, batch=8192, num_kv_heads=8, group_size=8)  # over 2^31 tiles of work
    assert lib.ri_token_attend_workspace(b(many), 1 << 28) == 0
    p = C.CTokenPrefix(PTR, PTR, 1 << 28, 0, 128, 1 << 35)
    assert lib.ri_token_attend(b(many), PTR, b(p), PTR, None, 1, PTR, 1 << 40, None) == UNSUPPORTED
    x, rope = C.CHeads(PTR, 512, 256, 128), C.CRope(PTR, 128, 0, 1.0)
    assert lib.ri_rotary(1 << 16, 1 << 15, 1, 128, 0, b(x), PTR, 0, b(rope), b(x), 0,
                         None) == UNSUPPORTED
    assert lib.ri_token_append(b(_cache(C, batch=32768)), 1 << 16, b(x), b(x), PTR, 0, None, None,
                               None, 5 * PTR, PTR, None) == UNSUPPORTED
    assert lib.ri_token_evict_workspace(b(_cache(C)), 0) == 0
    big = _cache(C, capacity=(1 << 24) + 1)
    assert lib.ri_token_evict_workspace(b(big), 8) == 0
    assert lib.ri_token_evict(b(big), 8, 0, 0, b(big), PTR, 1 << 30, None) == UNSUPPORTED
    assert lib.ri_token_attend(b(_cache(C, batch=65537, num_kv_heads=1)), PTR, None, PTR, None, 1,
                               PTR, 1 << 30, None) == UNSUPPORTED


def test_rotary_refusals(R, C):
    lib, b = R.lib, ctypes.byref
    x, rope = C.CHeads(PTR, 512, 256, 128), C.CRope(PTR, 128, 0, 1.0)

    def call(B=1, T=1, H=1, d=128, dtype=0, x=x, pos=PTR, rope=rope, out=x):
        return lib.ri_rotary(B, T, H, d, dtype, None if x is None else b(x), pos, 0,
                             None if rope is None else b(rope), None if out is None else b(out),
                             0, None)
    for kw in (dict(B=0), dict(T=0), dict(H=0), dict(d=1), dict(d=257), dict(dtype=3),
               dict(x=None), dict(out=None), dict(pos=None), dict(pos=PTR + 2), dict(rope=None),
               dict(x=C.CHeads(None, 1, 1, 1)), dict(x=C.CHeads(PTR + 1, 512, 256, 128)),
               dict(rope=C.CRope(None, 128, 0, 1.0)), dict(rope=C.CRope(PTR + 4, 128, 0, 1.0)),
               dict(rope=C.CRope(PTR, 127, 0, 1.0)), dict(rope=C.CRope(PTR, 130, 0, 1.0)),
               dict(rope=C.CRope(PTR, 0, 0, 1.0)), dict(rope=C.CRope(PTR, 128, 0, math.nan)),
               dict(out=C.CHeads(PTR, 512, 128, 256))):
        assert call(**kw) == INVALID, kw


def test_append_refusals(R, C):
    lib, b, c = R.lib, ctypes.byref, _cache(C)
    h = C.CHeads(PTR, 512, 256, 128)
    rope = C.CRope(PTR, 128, 0, 1.0)

    def call(T=1, k=h, v=h, pos=PTR, rope=rope, q=None, q_out=None, lens=5 * PTR, ws=PTR):
        ref = lambda s: None if s is None else b(s)  # noqa: E731
        return lib.ri_token_append(b(c), T, ref(k), ref(v), pos, 1, ref(rope), ref(q), q_out,
                                   lens, ws, None)
    for kw in (dict(T=0), dict(k=None), dict(v=None), dict(k=C.CHeads(PTR + 8, 512, 256, 128)),
               dict(k=C.CHeads(PTR, 512, 256, 132)), dict(v=C.CHeads(PTR, 4, 256, 128)),
               dict(pos=None), dict(rope=C.CRope(PTR, 130, 0, 1.0)), dict(q=h),
               dict(q_out=PTR), dict(q=h, q_out=PTR + 8), dict(lens=None), dict(lens=PTR + 2),
               dict(lens=5 * PTR + 4), dict(ws=None), dict(ws=PTR + 4)):
        assert call(**kw) == INVALID, kw


def test_attend_refusals(R, C):
    lib, b, c = R.lib, ctypes.byref, _cache(C)
    good = C.CTokenPrefix(PTR, PTR, 10, 0, 128, 1280)
    need = lib.ri_token_attend_workspace(b(c), 10)
    assert need > 256

    def call(q=PTR, p=good, out=PTR, lse=None, ws=PTR, n=need):
        return lib.ri_token_attend(b(c), q, b(p), out, lse, 1, ws, n, None)
    for kw in (dict(q=None), dict(q=PTR + 8), dict(out=None), dict(lse=PTR + 2), dict(ws=None),
               dict(p=C.CTokenPrefix(None, PTR, 10, 0, 128, 1280)),
               dict(p=C.CTokenPrefix(PTR, PTR + 8, 10, 0, 128, 1280)),
               dict(p=C.CTokenPrefix(PTR, PTR, -1, 0, 128, 1280)),
               dict(p=C.CTokenPrefix(PTR, PTR, 10, 1, 128, 1280)),
               dict(p=C.CTokenPrefix(PTR, PTR, 10, 0, 64, 1280)),
               dict(p=C.CTokenPrefix(PTR, PTR, 10, 0, 132, 1280)),
               dict(p=C.CTokenPrefix(PTR, PTR, 10, 0, 128, 0))):
        assert call(**kw) == INVALID, kw
    assert call(n=need - 1) == WORKSPACE


def test_evict_refusals(R, C):
    lib, b, c = R.lib, ctypes.byref, _cache(C)
    need = lib.ri_token_evict_workspace(b(c), 8)

    def call(budget=8, first=0, recent=0, out=c, ws=PTR, n=need):
        return lib.ri_token_evict(b(c), budget, first, recent, None if out is None else b(out),
                                  ws, n, None)
    for kw in (dict(budget=0), dict(first=-1), dict(recent=-1), dict(first=4, recent=5),
               dict(out=None), dict(ws=None), dict(out=_cache(C, batch=1)),
               dict(out=_cache(C, num_kv_heads=1)),
               dict(out=_cache(C, capacity=60)),       # the same arrays, another capacity
               dict(out=_cache(C, K=PTR + 256)),       # overlapping, not the same
               dict(out=_cache(C, K=2 * PTR, V=PTR))):  # each other's arrays
        assert call(**kw) == INVALID, kw
    c6 = _cache(C, batch=3)  # 24 bytes of lengths
    assert lib.ri_token_evict(b(c6), 8, 0, 0, b(_cache(C, batch=3, lens=5 * PTR + 16)), PTR,
                              1 << 20, None) == INVALID
    apart = dict(K=11 * PTR, V=12 * PTR, pos=13 * PTR, weight=14 * PTR, lens=15 * PTR)
    assert call(out=_cache(C, capacity=7, **apart)) == CAPACITY
    assert call(n=need - 1) == WORKSPACE


def test_binding_refusals(R, C):
    """The binding's own checks run before any CUDA call."""
    x = torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16)
    pos = torch.zeros(1, 2, dtype=torch.int32)
    t = R.RotaryTable.make(128, device="cpu")
    with pytest.raises(ValueError):
        R.rotary(x[0], pos, t)
    with pytest.raises(TypeError):
        R.rotary(x.double(), pos, t)
    with pytest.raises(TypeError):
        R.rotary(x, pos.long(), t)
    with pytest.raises(ValueError):
        R.rotary(x, pos[:, :1], t)
    with pytest.raises(ValueError):
        R.rotary(x.transpose(2, 3), pos, t)
    with pytest.raises(ValueError):
        R.rotary(x, pos, t, out=torch.zeros(1, 1, 3, 128, dtype=x.dtype).expand(1, 2, 3, 128))
    with pytest.raises(ValueError):
        R.rotary(x, pos, t)  # not on a GPU
    with pytest.raises(ValueError):
        R.RotaryTable.make(128, scaling="other", device="cpu")
    with pytest.raises(R.RIError):
        R.RotaryTable.make(7, device="cpu")
    z = torch.zeros(1, 2, 8, 128, dtype=torch.bfloat16)
    meta = (torch.zeros(1, 2, 8, dtype=torch.int32), torch.zeros(1, 2, 8),
            torch.zeros(1, 2, dtype=torch.int32))
    cache = R.TokenCache(z, z.clone(), *meta, group_size=2)
    with pytest.raises(R.RIError):
        R.TokenCache(z, z.clone(), *meta, group_size=9)
    with pytest.raises(R.RIError):
        R.TokenCache(z[..., :64].contiguous(), z[..., :64].contiguous(), *meta)
    with pytest.raises(TypeError):
        R.TokenCache(z.float(), z, *meta)
    with pytest.raises(ValueError):
        R.TokenCache(z, z.clone(), meta[0][:, :, :4], *meta[1:])
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        R.token_attend(q[:, :3], cache)
    with pytest.raises(ValueError):
        R.token_attend(q, cache, prefix=(z[0], z[0, :, :4]))
    with pytest.raises(ValueError):
        R.token_attend(q, cache, prefix=(z[0, :1], z[0, :1]))
    k = torch.zeros(1, 2, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        R.token_append(cache, k, k[:, :1], pos)
    with pytest.raises(ValueError):
        R.token_append(cache, k, k, pos, q_out=q)
    with pytest.raises(ValueError):
        R.token_append(cache, k, k, pos, t, q=q)
    with pytest.raises(R.RIError):
        R.token_evict_workspace_bytes(cache, 0)
