"""Rotary positions and the exact token cache on the GPU against the fp64
oracle.

Tolerances, per element, from the arithmetic:
 * a rounding to the stored type is off by at most half a step, eps / 2 of the
   value (fp16: at least half of 2^-24, its subnormal step);
 * rotary: the angle in half turns is rounded to 24 bits (2^-25 absolute, pi *
   2^-25 radians), cos and sin to 2 units of 2^-24 each, the magnitude, the two
   products and the sum to half a unit each: (|a| + |b|) * mag * (pi 2^-25 +
   (2 + 1 + 2) 2^-24) < (|a| + |b|) * mag * 4.1e-7;
 * attention: a score is a sum of 128 products of bf16 values in fp32, off by
   at most 128 * 2^-23 * |q| |k| / sqrt(128) =: e (a truncating accumulator
   counted), so a probability is off by a factor within exp(2 e) and 2^-18 for
   the exponentials, sums and merges in fp32; rounded to bf16 it is p (1 + d),
   |d| <= 2^-8, in the value product and in the sum that divides it, so a weight
   is p (1 + d) / (1 + mean of d), within 2 * 2^-8 / (1 - 2^-8) of p; the
   output's own rounding adds 2^-8 of the value.
"""
import math

import numpy as np
import pytest
import torch

from oracle import token_cache as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROTARY = 4.1e-7


@pytest.fixture(scope="module")
def R():
    import kv_cache_vector_segmented_b200 as R
    return R


def _np(t):
    return t.detach().double().cpu().numpy()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------- rotary
def _rotary_tol(x, y, n, mag, interleaved, dtype):
    """Per element bound of |device - y| for inputs x [..., d]."""
    ax = np.abs(x)
    pair = np.zeros_like(ax)
    if interleaved:
        s = ax[..., 0:2 * n:2] + ax[..., 1:2 * n:2]
        pair[..., 0:2 * n:2] = pair[..., 1:2 * n:2] = s
    else:
        s = ax[..., :n] + ax[..., n:2 * n]
        pair[..., :n] = pair[..., n:2 * n] = s
    inner = ROTARY * mag * pair
    half = torch.finfo(dtype).eps / 2
    return inner + half * (np.abs(y) + inner) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,n", [(128, 128), (128, 64), (128, 20), (128, 2), (96, 96), (256, 128),
                                 (6, 4)])
def test_rotary(R, dtype, interleaved, d, n):
    for B, Tn, H in ((1, 1, 1), (2, 5, 7), (3, 33, 9)):
        g = _gen(B * 100 + Tn)
        x = torch.randn(B, Tn, H, d, generator=g).to(dtype)
        pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, Tn), generator=g).to(torch.int32)
        pos[0, 0] = 2 ** 31 - 1
        pos[-1, -1] = -2 ** 31
        t = R.RotaryTable.make(n, base=500000.0, scaling="yarn", factor=4.0,
                               interleaved=interleaved, device=DEV)
        f, mag = T.frequencies(n, 500000.0, "yarn", 4.0)
        for inverse in (False, True):
            y = _np(R.rotary(x.to(DEV), pos.to(DEV), t, inverse=inverse))
            want = T.rotary(_np(x), pos.numpy(), f, mag, interleaved, inverse)
            # fp64 angles of the oracle at 2^31 positions: 2^31 * 2^-53 * |f| relative, radians
            slack = 2.0 ** 31 * 2.0 ** -52 * mag * np.abs(_np(x)).max() * 2
            assert (np.abs(y - want) <= _rotary_tol(_np(x), want, n // 2, mag, interleaved, dtype)
                    + slack).all()
            assert (y[..., n:] == _np(x)[..., n:]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_strides(R, interleaved):
    """Slices of a projection in, the index build's layout out, in place, and
    rows that are not 16-byte aligned."""
    B, Tn, H, d = 2, 37, 5, 128
    t = R.RotaryTable.make(64, interleaved=interleaved, device=DEV)
    f, mag = T.frequencies(64, 10000.0)
    pos = torch.arange(Tn, dtype=torch.int32).expand(B, Tn)
    for pad in (0, 8, 2, 3):
        big = torch.randn(B, Tn, 3 * H, d + pad, generator=_gen(pad)).bfloat16().to(DEV)
        x = big[:, :, H:2 * H, :d]
        before = big.clone()
        want = T.rotary(_np(x), pos.numpy(), f, mag, interleaved)
        tol = _rotary_tol(_np(x), want, 32, mag, interleaved, torch.bfloat16)
        out = torch.full((B, H, Tn, d), 7.0, dtype=torch.bfloat16, device=DEV)
        got = R.rotary(x, pos.to(DEV), t, out=out.transpose(1, 2))
        assert got.data_ptr() == out.data_ptr()
        assert (np.abs(_np(out).transpose(0, 2, 1, 3) - want) <= tol).all()
        assert torch.equal(big, before)
        R.rotary(x, pos.to(DEV)[:1].expand(B, Tn), t, out=x)
        assert (np.abs(_np(x) - want) <= tol).all()
        big[:, :, H:2 * H, :d] = before[:, :, H:2 * H, :d]
        assert torch.equal(big, before)  # nothing beside the heads was written


def test_rotary_backward_is_inverse(R):
    """<R(x), w> differentiated: against the formula (R^T w) and differences."""
    B, Tn, H, d, n = 2, 3, 2, 128, 64
    for interleaved in (False, True):
        t = R.RotaryTable.make(n, interleaved=interleaved, scaling="yarn", factor=4.0, device=DEV)
        f, mag = T.frequencies(n, 10000.0, "yarn", 4.0)
        g = _gen(5)
        x, w = (torch.randn(B, Tn, H, d, generator=g) for _ in range(2))
        pos = torch.randint(0, 100000, (B, Tn), generator=g).to(torch.int32).to(DEV)
        grad = R.rotary(w.to(DEV), pos, t, inverse=True)
        want = T.rotary(_np(w), pos.cpu().numpy(), f, mag, interleaved, inverse=True)
        tol = _rotary_tol(_np(w), want, n // 2, mag, interleaved, torch.float32)
        assert (np.abs(_np(grad) - want) <= tol).all()
        # the map is linear: its difference quotient over a unit step is exact
        # but for the roundings, at most mag * 2 * 4.1e-7 * (|x| + 1) each
        base = _np(R.rotary(x.to(DEV), pos, t))
        for at in ((0, 0, 0, 0), (1, 2, 1, 33), (1, 1, 0, 40), (0, 2, 1, 100)):
            xe = x.clone()
            xe[at] += 1.0
            diff = ((_np(R.rotary(xe.to(DEV), pos, t)) - base) * _np(w)).sum()
            bound = 8 * ROTARY * mag * (np.abs(_np(x)).max() + 1) * np.abs(_np(w)).max() * 2
            assert abs(diff - _np(grad)[at]) <= bound


# ------------------------------------------------------------------- append
def _random_cache(R, B, H, G, cap, lens, seed, poison=True):
    g = _gen(seed)
    c = R.TokenCache.empty(B, H, G, cap, DEV)
    K, V = (torch.randn(B, H, cap, 128, generator=g).bfloat16() for _ in range(2))
    lens = torch.tensor(lens, dtype=torch.int32).reshape(B, H)
    if poison:  # rows behind the last token hold what no result may see
        dead = torch.arange(cap) >= lens[..., None]
        K[dead] = float("nan")
        V[dead] = float("inf")
    c.K.copy_(K)
    c.V.copy_(V)
    c.lens.copy_(lens)
    c.weight.copy_(torch.rand(B, H, cap, generator=g))
    c.pos.copy_(torch.rand(B, H, cap, generator=g).argsort(-1).int())
    return c


def _state(c):
    return {k: getattr(c, k).clone() for k in ("K", "V", "pos", "weight", "lens")}


def _same(a, b):
    """Equal bits (NaN included)."""
    bits = {torch.bfloat16: torch.int16, torch.float32: torch.int32}.get(a.dtype, a.dtype)
    return torch.equal(a.view(bits), b.view(bits))


@pytest.mark.parametrize("Tn", [1, 3, 70])
@pytest.mark.parametrize("G", [1, 4, 7])
@pytest.mark.parametrize("rope", ["half", "inter", "odd", None])
def test_append(R, Tn, G, rope):
    B, H, cap = 3, 2, 100
    lens = [0, 5, 30, 29, 11, 30]
    for apart in (False, True):
        c = _random_cache(R, B, H, G, cap, lens, 1)
        before = _state(c)
        g = _gen(Tn)
        qkv = torch.randn(B, Tn, H * (G + 2), 128, generator=g).bfloat16()
        pos = torch.randint(0, 10 ** 6, (B, Tn), generator=g).to(torch.int32)
        n = {"half": 128, "inter": 96, "odd": 20}.get(rope, 0)
        t = R.RotaryTable.make(n, interleaved=rope == "inter", device=DEV) if rope else None
        dev = qkv.to(DEV)
        q, k, v = dev[:, :, :H * G], dev[:, :, H * G:H * G + H], dev[:, :, H * G + H:]
        lens_out = torch.zeros(B, H, dtype=torch.int32, device=DEV) if apart else None
        q_out = R.token_append(c, k, v, pos.to(DEV), t, q=q, lens_out=lens_out)
        assert R.read_device_status(c.status) == 0
        x = _np(qkv)
        f, mag = T.frequencies(n, 10000.0) if n else (np.zeros(0), 1.0)
        want = T.rotary(x, pos.numpy(), f, mag, rope == "inter")
        tol = _rotary_tol(x, want, n // 2, mag, rope == "inter", torch.bfloat16)
        assert (np.abs(_np(q_out) - want[:, :, :H * G]) <= tol[:, :, :H * G]).all()
        new = (before["lens"].cpu() + Tn)
        assert torch.equal((lens_out if apart else c.lens).cpu(), new)
        assert torch.equal(c.lens.cpu(), before["lens"].cpu() if apart else new)
        after = _state(c)
        for b in range(B):
            for h in range(H):
                a = lens[b * H + h]
                rows = slice(a, a + Tn)
                kk = H * G + h
                assert (np.abs(_np(after["K"][b, h, rows]) - want[b, :, kk])
                        <= tol[b, :, kk]).all()
                assert torch.equal(after["V"][b, h, rows], v[b, :, h])
                assert torch.equal(after["pos"][b, h, rows].cpu(), pos[b])
                assert (after["weight"][b, h, rows] == 0).all()
                for name in ("K", "V", "pos", "weight"):  # all other rows as they were
                    for part in (slice(0, a), slice(a + Tn, cap)):
                        assert _same(after[name][b, h, part], before[name][b, h, part])


def test_append_without_room_or_length(R):
    """A full head stores nothing; lengths out of range are reported; the
    other heads go on."""
    B, H, cap = 2, 2, 40
    k = torch.randn(B, 3, H, 128, device=DEV).bfloat16()
    pos = torch.arange(3, dtype=torch.int32, device=DEV).expand(B, 3)
    for lens, status, want in (([38, 0, 37, 40], 4, [38, 3, 40, 40]),
                               ([1, -5, 2, 3], 1, [4, 3, 5, 6]),
                               ([1, 2, 41, 3], 1, [4, 5, 40, 6])):
        c = _random_cache(R, B, H, 1, cap, [0] * 4, 3, poison=False)
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32).view(B, H))
        before = _state(c)
        R.token_append(c, k, k, pos)
        assert R.read_device_status(c.status) == status
        assert R.read_device_status(c.status) == 0
        assert c.lens.view(-1).tolist() == want
        full = lens.index(38) if 38 in lens else lens.index(41) if 41 in lens else None
        if full is not None:
            assert _same(c.K.view(4, cap, 128)[full], before["K"].view(4, cap, 128)[full])


# ------------------------------------------------------------------- attend
def _prefix(H, P, seed, form):
    g = _gen(seed + 17)
    pk, pv = (torch.randn(H, P, 128, generator=g).bfloat16() for _ in range(2))
    if form == "dense":
        return pk.to(DEV), pv.to(DEV)
    if form == "padded":  # a slice of a longer buffer: the rest must not be seen
        out = []
        for x in (pk, pv):
            big = torch.full((H, P + 9, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
            big[:, :P] = x.to(DEV)
            out.append(big[:, :P])
        return tuple(out)
    return tuple(x.to(DEV).transpose(0, 1).contiguous().transpose(0, 1) for x in (pk, pv))


def _check_attend(R, c, before, q, prefix, out, lse, add=True, scale=1.0):
    B, H, G = c.batch, c.num_kv_heads, c.group_size
    K, V, lens = _np(before["K"]), _np(before["V"]), before["lens"].cpu().numpy()
    qn, o, l, w = _np(q).reshape(B, H, G, 128), _np(out), _np(lse), _np(c.weight)
    w0 = _np(before["weight"])
    for h in range(H):
        pk, pv = (None, None) if prefix is None else (_np(prefix[0][h]), _np(prefix[1][h]))
        for b in range(B):
            n = int(min(max(lens[b, h], 0), c.capacity))
            want, want_l, want_w, mean = T.attend(qn[b, h], K[b, h, :n], V[b, h, :n], pk, pv)
            norms = [np.linalg.norm(x, axis=1).max() for x in (K[b, h, :n], pk)
                     if x is not None and len(x)]
            e = 128 * 2.0 ** -23 * (max(norms) if norms else 0.0) * np.linalg.norm(
                qn[b, h], axis=1).max() / math.sqrt(128)
            off = math.expm1(2 * e) + 2.0 ** -18
            rows = slice(h * G, (h + 1) * G)
            tol = (off + 2 * 2.0 ** -8 / (1 - 2.0 ** -8)) * mean + 2.0 ** -8 * np.abs(want)
            assert (np.abs(o[b, rows] - want) <= tol * (1 + 2.0 ** -8)).all(), (b, h)
            if n + (0 if pk is None else len(pk)) == 0:
                assert (l[b, rows] == -np.inf).all() and (o[b, rows] == 0).all()
            else:
                assert (np.abs(l[b, rows] - want_l) <= e + 2.0 ** -18
                        + 2.0 ** -22 * np.abs(want_l)).all()
            if add:
                # fp32: 8 probabilities summed, then added to the weight; one of
                # them below 2^-126 may be flushed
                tol_w = want_w * (off + 2.0 ** -20) + (w0[b, h, :n] + want_w) * 2.0 ** -23 + 2e-37
                assert (np.abs(w[b, h, :n] - w0[b, h, :n] - want_w) <= tol_w).all()
                assert (w[b, h, n:] == w0[b, h, n:]).all()
    if not add:
        assert (w == w0).all()
    for name in ("K", "V", "pos", "lens"):
        assert _same(getattr(c, name), before[name])


def _attend_case(R, B, H, G, P, cap, lens, form="dense", add=True, seed=0, gain=1.0):
    c = _random_cache(R, B, H, G, cap, lens, seed)
    prefix = _prefix(H, P, seed, form) if P else None
    q = (gain * torch.randn(B, H * G, 128, generator=_gen(seed + 5))).bfloat16().to(DEV)
    before = _state(c)
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)
    out, lse = R.token_attend(q, c, prefix, add_weight=add, workspace=ws)
    assert R.read_device_status(ws) == 0
    _check_attend(R, c, before, q, prefix, out, lse, add)
    return c, q, prefix, out, lse, ws


def _ragged(B, H, top, seed=0):
    g = np.random.default_rng(seed)
    lens = g.integers(0, top + 1, B * H)
    lens[0] = top
    if B * H > 1:
        lens[-1] = 0
    return lens.tolist()


@pytest.mark.parametrize("P", [0, 1, 2, 63, 64, 127, 128, 129, 255, 257, 1000])
def test_attend_prefix_lengths(R, P):
    _attend_case(R, 3, 2, 4, P, 70, _ragged(3, 2, 66, P))


@pytest.mark.parametrize("cap", [1, 2, 15, 16, 17, 63, 65, 127, 300, 1111])
def test_attend_own_lengths(R, cap):
    for P in (0, 130):
        _attend_case(R, 2, 3, 4, P, cap, _ragged(2, 3, cap, cap))


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_attend_groups(R, G):
    _attend_case(R, 5, 2, G, 200, 50, _ragged(5, 2, 50, G))


@pytest.mark.parametrize("B,G", [(16, 8), (17, 8), (19, 7), (33, 4), (65, 4), (130, 2), (300, 1)])
def test_attend_many_rows(R, B, G):
    """Query rows below, at and past one and two 128-row tiles, ragged ones."""
    _attend_case(R, B, 2, G, 391, 20, _ragged(B, 2, 20, B))


@pytest.mark.parametrize("form", ["padded", "token_major"])
def test_attend_prefix_strides(R, form):
    for H, P in ((1, 77), (3, 140), (2, 1)):
        _attend_case(R, 2, H, 4, P, 24, _ragged(2, H, 24), form)


def test_attend_nothing(R):
    _attend_case(R, 2, 2, 4, 0, 8, [0] * 4)
    _attend_case(R, 1, 1, 1, 0, 8, [0])
    _attend_case(R, 2, 2, 4, 300, 8, [0] * 4)
    _attend_case(R, 1, 1, 1, 0, 8, [1])


def test_attend_without_weights(R):
    _attend_case(R, 3, 2, 4, 150, 70, _ragged(3, 2, 66), add=False)


@pytest.mark.parametrize("gain", [0.0, 30.0, 400.0])
def test_attend_sharp_and_flat(R, gain):
    """Equal scores, and scores of thousands: one token takes all."""
    _attend_case(R, 3, 2, 4, 500, 300, _ragged(3, 2, 300), gain=gain)


def test_attend_rising_scores(R):
    """Every later token outscores all before it: the running maximum moves at
    every tile."""
    B, H, G, P, cap = 2, 1, 4, 2000, 600
    c = _random_cache(R, B, H, G, cap, [600, 500], 2)
    pk, pv = (x.clone() for x in _prefix(H, P, 2, "dense"))
    q = torch.zeros(B, H * G, 128)
    q[..., 0] = 8.0
    pk[..., 0] = torch.linspace(-60, 60, P).bfloat16().to(DEV)
    c.K[..., 0] = torch.linspace(61, 200, cap).bfloat16().to(DEV)
    q = q.bfloat16().to(DEV)
    before = _state(c)
    before["K"][1, 0, 500:] = float("nan")
    c.K[1, 0, 500:] = float("nan")
    out, lse = R.token_attend(q, c, (pk, pv))
    _check_attend(R, c, before, q, (pk, pv), out, lse)
    out, lse = R.token_attend(q, _no_tokens(R, c), (pk, pv), add_weight=False)
    e = _no_tokens(R, c)
    _check_attend(R, e, _state(e), q, (pk, pv), out, lse, add=False)


def _no_tokens(R, c):
    return R.TokenCache(c.K, c.V, c.pos, c.weight, torch.zeros_like(c.lens), c.group_size)


def test_attend_long(R):
    _attend_case(R, 1, 1, 4, 70001, 33000, [32900])
    _attend_case(R, 2, 2, 7, 40000, 100, _ragged(2, 2, 100))


def test_attend_long_and_mixed_tiles(R):
    """Three row tiles (a pair and a single one) over many key tiles, the blocks'
    shares cut at odd places."""
    _attend_case(R, 65, 1, 4, 20011, 40, _ragged(65, 1, 40))
    _attend_case(R, 37, 3, 8, 9001, 40, _ragged(37, 3, 40))


def test_attend_bad_lengths_reported(R):
    c = _random_cache(R, 2, 2, 4, 30, [0] * 4, 1, poison=False)
    c.lens.copy_(torch.tensor([[-3, 31], [2 ** 31 - 1, 4]], dtype=torch.int32))
    before = _state(c)
    q = torch.randn(2, 8, 128, device=DEV).bfloat16()
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, 0), DEV)
    out, lse = R.token_attend(q, c, workspace=ws)
    assert R.read_device_status(ws) == 1
    _check_attend(R, c, before, q, None, out, lse)


def test_attend_same_result_each_time(R):
    """No atomics whose order could change a result."""
    c, q, prefix, out, lse, ws = _attend_case(R, 9, 2, 5, 3000, 700, _ragged(9, 2, 700))
    w0 = c.weight.clone()
    ref = None
    for _ in range(5):
        c.weight.copy_(w0)
        o, l = R.token_attend(q, c, prefix, workspace=ws)
        got = (o.clone(), l.clone(), c.weight.clone())
        assert ref is None or all(torch.equal(a, b) for a, b in zip(ref, got))
        ref = got
    assert torch.equal(ref[0], out) and torch.equal(ref[1], lse)


# -------------------------------------------------------------------- evict
def _check_evict(c_before, out_before, out, budget, first, recent):
    B, H = c_before["lens"].shape
    cap = c_before["pos"].shape[2]
    for b in range(B):
        for h in range(H):
            n = int(min(max(int(c_before["lens"][b, h]), 0), cap))
            src = T.evict(c_before["pos"][b, h, :n].cpu().numpy(),
                          c_before["weight"][b, h, :n].cpu().numpy(), budget, first, recent)
            m = len(src)
            assert int(out.lens[b, h]) == m
            at = torch.from_numpy(src).to(DEV)
            for name in ("K", "V", "pos", "weight"):
                x = getattr(out, name)[b, h]
                assert _same(x[:m], c_before[name][b, h][at]), (b, h, name)
                assert _same(x[m:], out_before[name][b, h][m:]), (b, h, name)


def _evict_case(R, B, H, cap, lens, budget, first, recent, into="self", seed=0, edit=None):
    c = _random_cache(R, B, H, 2, cap, lens, seed)
    if edit:
        edit(c)
    before = _state(c)
    if into == "self":
        out = c
    elif into == "shared":  # K and V in place, the rest elsewhere
        out = R.TokenCache(c.K, c.V, torch.full_like(c.pos, -9), torch.full_like(c.weight, -9.0),
                           torch.full_like(c.lens, -9), 2)
    else:
        out = _random_cache(R, B, H, 1, min(budget, cap) + 3, [0] * (B * H), seed + 1)
    out_before = _state(out)
    ws = R.alloc_workspace(R.token_evict_workspace_bytes(c, budget), DEV)
    assert R.token_evict(c, budget, first, recent, out=None if into == "self" else out,
                         workspace=ws) is out
    assert R.read_device_status(ws) == 0
    _check_evict(before, out_before, out, budget, first, recent)
    if into == "other":
        assert all(_same(getattr(c, k), before[k]) for k in before)
    return c, out, ws


@pytest.mark.parametrize("into", ["self", "shared", "other"])
@pytest.mark.parametrize("cap,budget,first,recent", [
    (1, 1, 0, 0), (2, 1, 0, 1), (33, 32, 4, 8), (100, 10, 2, 3), (100, 99, 0, 99),
    (700, 1, 1, 0), (1025, 1024, 4, 64), (3000, 1500, 0, 0), (5000, 130, 100, 30)])
def test_evict(R, into, cap, budget, first, recent):
    _evict_case(R, 2, 3, cap, _ragged(2, 3, cap, cap), budget, first, recent, into)


@pytest.mark.parametrize("budget", [64, 65, 1000])
def test_evict_nothing_to_do(R, budget):
    for into in ("self", "shared", "other"):
        _evict_case(R, 2, 2, 64, [64, 10, 1, 0], budget, 4, 8, into)


def _ties(c):
    c.weight.copy_((c.weight * 4).floor())


def _all_equal(c):
    c.weight.zero_()


def _odd_values(c):
    w = c.weight
    w[..., ::7] = float("nan")
    w[..., 1::7] = float("inf")
    w[..., 2::7] = -float("inf")
    w[..., 3::7] = -0.0
    w[..., 4::7] = 0.0
    w[..., 5::7] = -w[..., 5::7]


def _same_positions(c):
    c.pos.fill_(5)


@pytest.mark.parametrize("edit", [_ties, _all_equal, _odd_values, _same_positions])
@pytest.mark.parametrize("into", ["self", "other"])
def test_evict_ties_and_odd_values(R, edit, into):
    for cap, budget, first, recent in ((257, 100, 3, 5), (2100, 2000, 0, 1), (2100, 7, 0, 0)):
        _evict_case(R, 2, 2, cap, _ragged(2, 2, cap, 3), budget, first, recent, into, edit=edit)


def test_evict_long(R):
    _evict_case(R, 1, 2, 70000, [70000, 65000], 5000, 4, 64, "other")
    _evict_case(R, 1, 1, 40000, [40000], 39000, 4, 64, "self")


@pytest.mark.parametrize("into", ["self", "shared", "other"])
def test_evict_few_heads(R, into):
    """Few heads with many rows: the rows move in a launch of their own."""
    _evict_case(R, 1, 2, 9000, [9000, 4000], 4500, 4, 64, into)
    _evict_case(R, 1, 1, 9000, [4100], 4500, 4, 64, into)


@pytest.mark.parametrize("into", ["self", "shared", "other"])
def test_evict_longer_than_shared_memory(R, into):
    """A slice too long to be held: its keys are read from memory each time."""
    _evict_case(R, 1, 1, 400000, [399000], 30000, 4, 64, into, edit=_ties)


def test_evict_bad_lengths_reported(R):
    c = _random_cache(R, 1, 4, 1, 30, [0] * 4, 1, poison=False)
    c.lens.copy_(torch.tensor([[-3, 31, 2 ** 31 - 1, 4]], dtype=torch.int32))
    before = _state(c)
    ws = R.alloc_workspace(R.token_evict_workspace_bytes(c, 10), DEV)
    R.token_evict(c, 10, 0, 0, workspace=ws)
    assert R.read_device_status(ws) == 1
    _check_evict(before, before, c, 10, 0, 0)


# ----------------------------------------------------------- as they are used
def _steps(R, c, t, prefix, P, steps, budget, seed=9):
    """Decode steps: append, attend, evict; yields each step's inputs and outputs."""
    B, H, G = c.batch, c.num_kv_heads, c.group_size
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)
    es = R.alloc_workspace(R.token_evict_workspace_bytes(c, budget), DEV)
    for i in range(steps):
        qkv = torch.randn(B, 1, H * (G + 2), 128, generator=_gen(seed + i)).bfloat16().to(DEV)
        pos = torch.full((B, 1), P + i, dtype=torch.int32, device=DEV)
        q, k, v = qkv[:, :, :H * G], qkv[:, :, H * G:H * G + H], qkv[:, :, H * G + H:]
        qr = R.token_append(c, k, v, pos, t, q=q).view(B, H * G, 128)
        before = _state(c)
        out, lse = R.token_attend(qr, c, prefix, workspace=ws)
        mid = _state(c)
        R.token_evict(c, budget, keep_first=0, keep_recent=4, workspace=es)
        yield qr, before, out, lse, mid
    for w in (ws, es, c.status):
        assert R.read_device_status(w) == 0


def test_decode_loop(R):
    """append, attend and evict in turn, each step checked from the state it met."""
    B, H, G, P = 3, 2, 4, 140
    c = R.TokenCache.empty(B, H, G, 16, DEV)
    t = R.RotaryTable.make(128, device=DEV)
    prefix = _prefix(H, P, 1, "dense")
    for i, (q, before, out, lse, mid) in enumerate(_steps(R, c, t, prefix, P, 30, 12)):
        assert (before["lens"] == min(i + 1, 13)).all()
        held = R.TokenCache(before["K"], before["V"], before["pos"], mid["weight"],
                            before["lens"], G)
        _check_attend(R, held, before, q, prefix, out, lse)
        _check_evict(mid, mid, c, 12, 0, 4)
    assert (c.lens == 12).all()
    # the newest four positions are held in every head
    for u in range(B * H):
        assert set(range(P + 26, P + 30)) <= set(c.pos.view(B * H, -1)[u, :12].tolist())


def test_index_beside_cache(R):
    """Rotated keys in the index build's layout, the new token's in index_append:
    the wave index reads what rotary writes."""
    B, H, G, N = 1, 2, 4, 700
    g = _gen(4)
    k, v = (torch.randn(B, N, H, 128, generator=g).bfloat16().to(DEV) for _ in range(2))
    q = torch.randn(B, 1, H * G, 128, generator=g).bfloat16().to(DEV)
    t = R.RotaryTable.make(128, device=DEV)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)[None]
    K = torch.empty(B, H, N, 128, dtype=torch.bfloat16, device=DEV)
    R.rotary(k, pos, t, out=K.transpose(1, 2))
    V = v.transpose(1, 2).contiguous()
    cfg = R.IndexConfig.make(B, H, G, N, clusters_per_seg=64, iters=3)
    idx = R.build_index(K, V, cfg)
    qr = R.rotary(q, pos[:, -1:], t).view(B, H * G, 128)
    # every cluster retrieved: the index's attention is the exact one
    C = idx.geom.clusters
    out, lse, _ = R.decode(qr, idx, R.DecodeConfig(C, 0))
    empty = R.TokenCache.empty(B, H, G, 1, DEV)
    out2, lse2 = R.token_attend(qr, empty, (K[0], V[0]))
    assert torch.allclose(lse, lse2, rtol=1e-5, atol=1e-4)
    assert (out.float() - out2.float()).abs().max() <= 2e-2 * out2.float().norm(dim=-1).max()


def test_other_stream_and_two_at_once(R):
    """Two caches on two streams at once, each with its workspace."""
    want, got, keep = [], [], []
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for i in range(2):
        c, q, prefix, out, lse, ws = _attend_case(R, 4, 2, 4, 5000, 900, _ragged(4, 2, 900, i),
                                                  seed=i)
        w = torch.zeros_like(c.weight)
        keep.append((R.TokenCache(c.K, c.V, c.pos, w, c.lens, 4), q, prefix, ws))
        want.append((out, lse))
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (c, q, prefix, ws) in zip(streams, keep):
            with torch.cuda.stream(s):
                got.append(R.token_attend(q, c, prefix, workspace=ws))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_captured_steps_share_a_workspace(R):
    """Two graphs of a decode step (two caches) over one workspace, replayed in
    turn: the same results as the calls one by one."""
    B, H, G, P, cap, budget = 2, 2, 4, 300, 40, 24
    t = R.RotaryTable.make(128, device=DEV)
    prefix = _prefix(H, P, 3, "dense")

    def make(seed):
        c = _random_cache(R, B, H, G, cap, [20] * 4, seed)
        qkv = torch.randn(B, 1, H * (G + 2), 128, generator=_gen(seed)).bfloat16().to(DEV)
        pos = torch.full((B, 1), P + 100, dtype=torch.int32, device=DEV)
        bufs = (torch.empty(B, 1, H * G, 128, dtype=torch.bfloat16, device=DEV),
                torch.empty(B, H * G, 128, dtype=torch.bfloat16, device=DEV),
                torch.empty(B, H * G, dtype=torch.float32, device=DEV))
        return c, qkv, pos, bufs

    probe = make(0)[0]
    n = max(R.token_attend_workspace_bytes(probe, P), R.token_evict_workspace_bytes(probe, budget))
    ws = R.alloc_workspace(n, DEV)

    def step(c, qkv, pos, bufs):
        R.token_append(c, qkv[:, :, H * G:H * G + H], qkv[:, :, H * G + H:], pos, t,
                       q=qkv[:, :, :H * G], q_out=bufs[0])
        R.token_attend(bufs[0].view(B, H * G, 128), c, prefix, out=bufs[1], lse=bufs[2],
                       workspace=ws)
        R.token_evict(c, budget, 0, 4, workspace=ws)

    plain, graphed = [make(s) for s in (1, 2)], [make(s) for s in (1, 2)]
    step(*make(7))  # kernels loaded before the capture
    torch.cuda.synchronize()
    graphs = []
    for x in graphed:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(*x)
        graphs.append(g)
    for _ in range(7):
        for x, y, g in zip(plain, graphed, graphs):
            step(*x)
            g.replay()
    torch.cuda.synchronize()
    assert R.read_device_status(ws) == 0
    for x, y in zip(plain, graphed):
        assert (x[0].lens == budget).all()
        for a, b in zip(_state(x[0]).values(), _state(y[0]).values()):
            assert _same(a, b)
        for a, b in zip(x[3], y[3]):
            assert torch.equal(a, b)


def test_side_stream_equals_default(R):
    """The decode loop on a stream of its own: the same results, bit for bit."""
    B, H, G, P = 2, 2, 4, 200
    t = R.RotaryTable.make(128, device=DEV)
    prefix = _prefix(H, P, 6, "dense")

    def loop():
        c = R.TokenCache.empty(B, H, G, 24, DEV)
        c.K.zero_()
        c.V.zero_()
        got = [(out.clone(), lse.clone()) for _, _, out, lse, _ in
               _steps(R, c, t, prefix, P, 20, 10)]
        return got, _state(c)

    want, state = loop()
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    with torch.cuda.stream(s):
        got, state2 = loop()
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(_same(state[k], state2[k]) for k in state)


def test_captured_long_calls(R):
    """A graph of the calls at sizes that take all their launches (prefix, own
    tokens, merge; selection and moves): replays repeat the eager results."""
    B, H, G, P, cap, budget = 1, 2, 4, 5000, 9000, 4200
    c = _random_cache(R, B, H, G, cap, [8800, 9000], 3)
    prefix = _prefix(H, P, 3, "dense")
    q = torch.randn(B, H * G, 128, generator=_gen(8)).bfloat16().to(DEV)
    out = R.TokenCache(c.K, c.V, *(torch.zeros_like(x) for x in (c.pos, c.weight, c.lens)), G)
    ws = R.alloc_workspace(max(R.token_attend_workspace_bytes(c, P),
                               R.token_evict_workspace_bytes(c, budget)), DEV)
    o, l = torch.empty_like(q), torch.empty(B, H * G, device=DEV)
    before = _state(c)

    def calls():
        R.token_attend(q, c, prefix, out=o, lse=l, workspace=ws)
        R.token_evict(c, budget, 0, 64, out=out, workspace=ws)

    def restore():
        c.K.copy_(before["K"])
        c.V.copy_(before["V"])
        c.weight.copy_(before["weight"])

    calls()
    want = (o.clone(), l.clone(), _state(out))
    restore()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(3):
        restore()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
        assert all(_same(getattr(out, k), v) for k, v in want[2].items())
    assert R.read_device_status(ws) == 0
