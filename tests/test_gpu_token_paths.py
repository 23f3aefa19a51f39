"""The exact token cache and rotary positions where the work is split most: long
prefixes, many heads, the row kernels' walk over many tokens, with inputs in
which a lost or exchanged piece of the work shows.

Three kinds of input for the attention:
 * flat: q = 0, so that every probability is 1 exactly, and values that mark
   their tile of 128 tokens: column j holds 1024 in the tiles t = j mod 128 and
   0 in all others.  Sums of these are exact in fp32, so the output is off by the
   roundings of 1 / r, the product and the store: 2^-23 and half a bf16 step.  A
   tile left out, or taken twice, moves its column by one part in the column's
   tiles.
 * picked: every query row has one key of its own, 2.5 times the query, which
   holds nearly all of its weight: the output is that key's value.  The keys
   picked are the first, a middle and the last one of every tile in turn.
 * gentle: queries of a tenth, whose scores are close and whose probabilities
   are no bf16 numbers.

Tolerances: a score is a sum of 128 products in fp32, off by at most e = 128 *
2^-23 * |q| |k| / sqrt(128) (a truncating accumulator counted), a probability so
by a factor within exp(2 e) and 2^-18 for exponentials, sums and merges =: off.
Own tokens' probabilities enter the value product to 2^-15.  The prefix's are
rounded to bf16, p (1 + d) with |d| <= 2^-8, in the value product and, or not, in
the sum that divides it: 2^-8 / (1 - 2^-8) of the prefix's part of sum_i p_i
|v_i| and of its part of the weight times |out|.  The output's own rounding is
half a bf16 step, 2^-8.
"""
import math

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
DEV = "cuda:0"
D = 128
TILE = 128


@pytest.fixture(scope="module")
def R():
    import kv_cache_vector_segmented_b200 as R
    return R


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ reference
def _formula(q, K, V, lens, PK, PV):
    """In 64 bits, q [B][H][G][d]: out, lse, weight [B][H][cap], sum_i p_i |v_i|
    of the prefix and of all, the prefix's part of the weight."""
    B, H, G, _ = q.shape
    cap, P = K.shape[2], PK.shape[1]
    res = [[] for _ in range(6)]
    for h in range(H):
        qh = q[:, h].double() / math.sqrt(D)
        x = torch.cat(((qh.reshape(B * G, D) @ PK[h].double().T).view(B, G, P),
                       qh @ K[:, h].double().transpose(1, 2)), 2)
        dead = torch.arange(cap, device=q.device) >= lens[:, h, None]
        x[:, :, P:].masked_fill_(dead[:, None], -math.inf)
        lse = torch.logsumexp(x, 2)
        p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        pre = p[..., :P].reshape(B * G, P)
        v = V[:, h].double().masked_fill(dead[..., None], 0.0)
        parts = [((pre @ f(PV[h].double())).view(B, G, D), p[..., P:] @ f(v))
                 for f in (lambda t: t, torch.abs)]
        for r, t in zip(res, (parts[0][0] + parts[0][1], lse, p[..., P:].sum(1), parts[1][0],
                              parts[1][0] + parts[1][1], p[..., :P].sum(2))):
            r.append(t)
    return [torch.stack(r, 1) for r in res]


def _check(R, q, c, prefix, out, lse, w0, exact_sums=False):
    """Compares a call's results with the formula's; returns its output."""
    B, H, G = c.batch, c.num_kv_heads, c.group_size
    none = torch.zeros(H, 0, D, dtype=torch.bfloat16, device=DEV)
    PK, PV = prefix if prefix is not None else (none, none)
    q = q.view(B, H, G, D)
    want, want_l, add, pre, mean, part = _formula(q, c.K, c.V, c.lens, PK, PV)
    norm = max([float(t.double().norm(dim=-1).max()) for t in (c.K, PK) if t.numel()])
    e = 128 * 2.0 ** -23 * norm * float(q.double().norm(dim=-1).max()) / math.sqrt(D)
    off = math.expm1(2 * e) + 2.0 ** -18
    if exact_sums:
        tol = want.abs() * 2.0 ** -8 * (1 + 2.0 ** -14)
    else:
        tol = (off + 2.0 ** -14) * mean + 2.0 ** -8 / (1 - 2.0 ** -8) * (
            pre + part[..., None] * mean)
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    over = ((out.view(B, H, G, D).double() - want).abs() - tol)
    worst = float(over.max())
    assert worst <= 0, (worst, tuple(int(i) for i in (over == over.max()).nonzero()[0]))
    fine = want_l > -math.inf
    off_l = (lse.view(B, H, G).double() - want_l)[fine].abs()
    assert (off_l <= (e + 2.0 ** -18 + 2.0 ** -22 * want_l.abs())[fine]).all()
    assert (lse.view(B, H, G)[~fine] == -math.inf).all()
    tol_w = add * (off + 2.0 ** -20) + (w0.double() + add) * 2.0 ** -23 + 2e-37
    assert ((c.weight.double() - w0.double() - add).abs() <= tol_w).all()
    return want


def _random(R, B, H, G, P, cap, lens, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = R.TokenCache.empty(B, H, G, cap, DEV)
    for t in (c.K, c.V):
        t.copy_(torch.randn(t.shape, generator=g, device=DEV))
    c.weight.copy_(torch.rand(c.weight.shape, generator=g, device=DEV))
    c.lens.copy_(torch.as_tensor(lens, dtype=torch.int32).view(B, H) if lens is not None else
                 torch.randint(0, cap + 1, (B, H), generator=_gen(seed)))
    prefix = tuple(torch.randn(H, P, D, generator=g, device=DEV).bfloat16() for _ in range(2)) \
        if P else None
    q = torch.randn(B, H * G, D, generator=g, device=DEV)
    return c, prefix, q, g


def _call(R, q, c, prefix, ws):
    w0 = c.weight.clone()
    out, lse = R.token_attend(q, c, prefix, workspace=ws)
    assert R.read_device_status(ws) == 0
    return out, lse, w0


# ------------------------------------------------- long and mixed-tile prefixes
# B, H, G, P, capacity, lengths (None: random): one row tile, two, three (a pair
# and a single one), five; own tokens alone, and long
SPLIT = [(1, 1, 4, 70001, 33000, [32900]), (2, 2, 7, 40000, 100, None),
         (65, 1, 4, 20011, 40, None), (37, 3, 8, 9001, 40, None), (80, 1, 8, 30000, 70, None),
         (64, 2, 4, 16500, 300, None), (1, 2, 8, 0, 50000, [50000, 41111])]


def _marks(n):
    """Values that mark their tile: 1024 in column t mod 128 of tile t."""
    v = torch.zeros(n, D)
    i = torch.arange(n)
    v[i, (i // TILE) % D] = 1024.0
    return v


def _marked(P, cap):
    """Marks of a prefix, and of own tokens counted on from a tile behind it."""
    pv = _marks(P)
    start = (P // TILE + 1) * TILE
    return pv, _marks(start + cap)[start:]


@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_marks_show_a_lost_tile(case):
    """Without a GPU: leaving out any tile of the prefix, or any 16 own tokens,
    moves the flat output by more than the tolerance."""
    B, H, G, P, cap, lens = SPLIT[case]
    own = cap if lens is None else max(lens)
    pv, v = _marked(P, cap)
    vals = torch.cat((pv, v[:own])).double()
    want = vals.sum(0) / len(vals)
    tol = want.abs() * 2.0 ** -8 * (1 + 2.0 ** -14)
    pieces = [(a, min(a + TILE, P)) for a in range(0, P, TILE)]
    pieces += [(P + a, P + min(a + 16, own)) for a in range(0, own, 16)]
    for a, b in pieces:
        for factor in (0, 2):  # left out, taken twice
            got = want + (factor - 1) * vals[a:b].sum(0) / len(vals)
            # (the last tile of the prefix, a token or two, may not show)
            assert ((got - want).abs() > tol).any() or b - a < 16, (a, b)


@gpu
@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_attend_flat(R, case):
    B, H, G, P, cap, lens = SPLIT[case]
    c, prefix, q, _ = _random(R, B, H, G, P, cap, lens, case)
    pv, v = _marked(P, cap)
    c.V.copy_(v.to(DEV).expand_as(c.V))
    if P:
        prefix[1].copy_(pv.to(DEV).expand_as(prefix[1]))
    q = torch.zeros_like(q).bfloat16()
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)
    out, lse, w0 = _call(R, q, c, prefix, ws)
    _check(R, q, c, prefix, out, lse, w0, exact_sums=True)


@gpu
@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_attend_picked(R, case):
    """Every tile's first, middle and last key is the one that some row picks,
    each by rows of all row tiles."""
    B, H, G, P, cap, lens = SPLIT[case]
    c, prefix, q, g = _random(R, B, H, G, P, cap, lens, case)
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)
    rows = B * G
    n_tiles = (P + TILE - 1) // TILE
    at = torch.cat([torch.tensor([t * TILE, min(t * TILE + 17 + t % 90, P - 1),
                                  min((t + 1) * TILE, P) - 1]) for t in range(n_tiles)]) \
        if P else torch.zeros(0, dtype=torch.long)
    per_turn = max(1, -(-len(at) // rows))
    for call in range(per_turn * ((rows + TILE - 1) // TILE) if P else 1):
        q = torch.randn(q.shape, generator=g, device=DEV).bfloat16()
        heads = q.view(B, H, G, D)
        for h in range(H):
            qh = (2.5 * heads[:, h].float()).bfloat16()
            if P:
                i = torch.arange(min(rows, len(at)))
                take = at[(call % per_turn * rows + i) % len(at)].to(DEV)
                prefix[0][h, take] = qh.reshape(rows, D)[
                    ((i + call // per_turn * TILE) % rows).to(DEV)]
            if not P or call % 2:
                for b in range(B):  # the first row's pick among its own tokens
                    n = int(c.lens[b, h])
                    if n:
                        c.K[b, h, (call * 977 + 15 * b) % n] = qh[b, 0]
        out, lse, w0 = _call(R, q, c, prefix, ws)
        want = _check(R, q, c, prefix, out, lse, w0)
        if P:
            assert float(want.abs().amax(-1).median()) > 1.5  # a picked value, not an average


@gpu
@pytest.mark.parametrize("case", range(len(SPLIT)))
def test_attend_gentle(R, case):
    B, H, G, P, cap, lens = SPLIT[case]
    c, prefix, q, _ = _random(R, B, H, G, P, cap, lens, case + 50)
    q = (0.1 * q).bfloat16()
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)
    out, lse, w0 = _call(R, q, c, prefix, ws)
    _check(R, q, c, prefix, out, lse, w0)


# --------------------------------------------------------- own tokens by themselves
@pytest.mark.parametrize("n", [17, 127, 300])
def test_own_tolerance_shows_one_part(n):
    """Without a GPU: probabilities of one bf16 part in the value product are
    off by more than the bound of own tokens."""
    g = _gen(n)
    q = (0.1 * torch.randn(64, D, generator=g)).bfloat16().double()
    K, V = (torch.randn(n, D, generator=g).bfloat16().double() for _ in range(2))
    x = q @ K.T / math.sqrt(D)
    e = torch.exp(x - x.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    got = (e.bfloat16().double() @ V / e.sum(1, keepdim=True)).bfloat16().double()
    slack = 128 * 2.0 ** -23 * float(K.norm(dim=1).max() * q.norm(dim=1).max()) / math.sqrt(D)
    off = math.expm1(2 * slack) + 2.0 ** -18 + 2.0 ** -14
    want, mean = p @ V, p @ V.abs()
    tol = off * mean
    tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert ((got - want).abs() > tol).any()


@gpu
@pytest.mark.parametrize("gain", [0.1, 1.0, 4.0])
@pytest.mark.parametrize("cap", [1, 16, 17, 127, 300, 1111])
def test_attend_own_tokens(R, cap, gain):
    c, _, q, _ = _random(R, 9, 3, 7, 0, cap, None, cap)
    q = (gain * q).bfloat16()
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, 0), DEV)
    out, lse, w0 = _call(R, q, c, None, ws)
    _check(R, q, c, None, out, lse, w0)


@gpu
@pytest.mark.parametrize("B,H,cap", [(64, 8, 300), (300, 4, 130), (128, 8, 1100)])
def test_attend_many_own_tasks(R, B, H, cap):
    """More tasks than warps without a prefix: the later ones are taken from the
    counter, which the next calls on the workspace find at 0, one with a prefix
    and one without."""
    c, prefix, q, g = _random(R, B, H, 4, 200, cap, None, cap)
    ws = R.alloc_workspace(max(R.token_attend_workspace_bytes(c, n) for n in (0, 200)), DEV)
    first = None
    for pre in (None, prefix, None):
        w = torch.zeros_like(c.weight)
        one = R.TokenCache(c.K, c.V, c.pos, w, c.lens, 4)
        qh = q.bfloat16()
        out, lse, w0 = _call(R, qh, one, pre, ws)
        _check(R, qh, one, pre, out, lse, w0)
        if pre is None:
            got = (out, lse, w.clone())
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
            first = got


@gpu
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("P", [0, 391])
def test_attend_many_heads(R, G, P):
    """More (sequence, KV head)s than the merge has blocks at a time: a block
    joins all rows of its group."""
    c, prefix, q, _ = _random(R, 155, 4, G, P, 90, None, G)
    q = q.bfloat16()
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)
    out, lse, w0 = _call(R, q, c, prefix, ws)
    _check(R, q, c, prefix, out, lse, w0)


# ------------------------------------------------------------- rotary and append
def _turned(x, pos, f, mag, interleaved, inverse=False):
    """In 64 bits, x [B][T][heads][d] and sum of |a|, |b| of each pair."""
    ang = pos.double()[..., None, None] * torch.as_tensor(f, device=x.device)
    c, s = mag * ang.cos(), mag * ang.sin() * (-1 if inverse else 1)
    n = len(f)
    y, pair = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else \
        (slice(0, n), slice(n, 2 * n))
    a, b = x[..., ia].double(), x[..., ib].double()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    pair[..., ia] = pair[..., ib] = a.abs() + b.abs()
    return y, pair


def _rotary_tol(y, pair, mag, dtype):
    """The angle's fraction cut to 32 bits, its scaling, the polynomials, the
    magnitude, the products and the sum: less than 10 * 2^-24 = 6e-7 of mag (|a| +
    |b|); and half a step of the type."""
    inner = 6e-7 * mag * pair
    return inner + torch.finfo(dtype).eps / 2 * (y.abs() + inner) + \
        (2.0 ** -25 if dtype == torch.float16 else 0.0)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("form", ["wide", "words", "elements"])
def test_rotary_many_tokens(R, form, interleaved, dtype):
    """Several tokens to a thread, over sequences: accesses of 16 bytes, of words
    and of elements, into the index build's layout and in place."""
    from oracle import token_cache as T
    B, Tn, H = 3, 14001, 3
    n = 64 if form == "wide" else 20
    # rows that do not start on 16 bytes, or (16 bit) on a word
    pad = {"wide": 8, "words": 2, "elements": 1}[form]
    g = torch.Generator(device=DEV).manual_seed(n)
    big = torch.randn(B, Tn, H, D + pad, generator=g, device=DEV).to(dtype)
    x = big[..., :D]
    pos = torch.randint(0, 10 ** 6, (B, Tn), generator=g, device=DEV).int()
    t = R.RotaryTable.make(n, scaling="yarn", factor=4.0, interleaved=interleaved, device=DEV)
    f, mag = T.frequencies(n, 10000.0, "yarn", 4.0)
    want, pair = _turned(x, pos, f, mag, interleaved)
    tol = _rotary_tol(want, pair, mag, dtype)
    tol[..., n:] = 0.0
    out = torch.full((B, H, Tn, D), 7.0, dtype=dtype, device=DEV)
    R.rotary(x, pos, t, out=out.transpose(1, 2))
    assert ((out.transpose(1, 2).double() - want).abs() <= tol).all()
    rest = big[..., D:].clone()
    R.rotary(x, pos, t, out=x)
    assert ((x.double() - want).abs() <= tol).all() and torch.equal(big[..., D:], rest)


@gpu
@pytest.mark.parametrize("n", [128, 20, 6, 0])
@pytest.mark.parametrize("Tn", [1, 2])
def test_append_many_sequences(R, n, Tn):
    """Several sequences to a block, lengths in place, accesses of 16 bytes (128
    and nothing rotated), of words (20) and of elements (6); full heads and
    lengths of 0 among them."""
    from oracle import token_cache as T
    B, H, G, cap = 5003, 2, 2, 5
    c, _, _, g = _random(R, B, H, G, 0, cap, None, n)
    before = {k: getattr(c, k).clone() for k in ("K", "V", "pos", "weight", "lens")}
    qkv = torch.randn(B, Tn, H * (G + 2), D, generator=g, device=DEV).bfloat16()
    pos = torch.randint(0, 10 ** 6, (B, Tn), generator=g, device=DEV).int()
    q, k, v = qkv[:, :, :H * G], qkv[:, :, H * G:H * G + H], qkv[:, :, H * G + H:]
    t = R.RotaryTable.make(n, device=DEV) if n else None
    f, mag = T.frequencies(n, 10000.0) if n else (np.zeros(0), 1.0)
    got = R.token_append(c, k, v, pos, t, q=q)
    want, pair = _turned(qkv, pos, f, mag, False)
    tol = _rotary_tol(want, pair, mag, torch.bfloat16)
    tol[..., n:] = 0.0
    assert ((got.double() - want[:, :, :H * G]).abs() <= tol[:, :, :H * G]).all()
    lens = before["lens"].long()
    room = lens + Tn <= cap
    assert room.any() and not room.all()
    assert R.read_device_status(c.status) == R.STATUS_CODES["RI_ERR_CAPACITY"]
    assert torch.equal(c.lens.long(), torch.where(room, lens + Tn, lens))
    i = torch.arange(cap, device=DEV)
    new = room[..., None] & (i >= lens[..., None]) & (i < (lens + Tn)[..., None])
    src = (i - lens[..., None]).clamp(0, Tn - 1)  # token of the step that lies in row i
    rows = src[..., None].expand(B, H, cap, D)
    for name, x, y in (("K", want, tol), ("V", qkv.double(), torch.zeros_like(tol))):
        first = H * G + (H if name == "V" else 0)
        x, y = (a[:, :, first:first + H].transpose(1, 2).gather(2, rows) for a in (x, y))
        z = getattr(c, name).double()
        assert ((z - x).abs() <= y)[new].all()
        assert torch.equal(getattr(c, name)[~new], before[name][~new])
    at = pos[:, None].expand(B, H, Tn).gather(2, src)
    assert torch.equal(c.pos, torch.where(new, at, before["pos"]))
    assert torch.equal(c.weight, torch.where(new, 0.0, before["weight"]))


@gpu
@pytest.mark.parametrize("P", [1, 50, 300, 1000])
@pytest.mark.parametrize("B,H,G", [(520, 32, 4), (4, 400, 4), (37, 160, 7)])
def test_attend_many_units(R, B, H, G, P):
    """More (KV head, pair of row tiles) units than SMs: a block takes several in a
    row, whole ones and parts, pairs and single ones among them."""
    c, prefix, q, _ = _random(R, B, H, G, P, 20, None, P)
    q = q.bfloat16()
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)
    out, lse, w0 = _call(R, q, c, prefix, ws)
    _check(R, q, c, prefix, out, lse, w0)
