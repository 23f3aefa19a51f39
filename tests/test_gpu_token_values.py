"""Live NaN and infinities in the exact token cache's attention, against the
formula in 64 bits: what a query, key or value holds reaches the output, lse and
weights as the formula has it, and no share of the work loses it.

A score of -inf has weight 0 (a mask's row, say); a row without any other score
is one with nothing to attend to: out = 0, lse = -inf.  A score of +inf or NaN
makes its row NaN.

Tolerances of the finite results, from the arithmetic: a score is a sum of 128
products in fp32, off by at most e = 128 * 2^-23 * |q| |k| / sqrt(128) (a
truncating accumulator counted), a probability so by a factor within exp(2 e)
and 2^-18 for the exponentials, sums and merges; rounded to bf16 in the value
product and in the sum that divides it, 2 * 2^-8 / (1 - 2^-8); half a step of
bf16, 2^-8, for the output.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def R():
    import kv_cache_vector_segmented_b200 as R
    return R


def _formula(q, keys, vals):
    """One head group in 64 bits, products and sums written out so that 0 * inf
    and inf - inf are what they are: out, lse, p and sum_i p_i |v_i| of the
    finite values."""
    x = torch.stack([(q[g] * keys).sum(-1) for g in range(q.shape[0])]) / math.sqrt(D)
    if x.shape[1] == 0:
        z = q.new_zeros(q.shape)
        return z, q.new_full(q.shape[:1], -INF), x, z
    top = x.amax(-1, keepdim=True)
    base = top.masked_fill(top == -INF, 0.0)
    e = torch.exp(x - base)
    den = e.sum(-1, keepdim=True)
    p = e / den.masked_fill(den == 0, 1.0)
    out = torch.stack([(p[g][:, None] * vals).sum(0) for g in range(q.shape[0])])
    flat = vals.nan_to_num(0.0, 0.0, 0.0).abs()
    return out, (base + torch.log(den))[:, 0], p, p.nan_to_num(0.0) @ flat


def _near(got, want, tol, what):
    """NaN and infinities alike, finite values within tol."""
    got, inf, fine = got.double(), want.isinf(), want.isfinite()
    nan_alike = torch.equal(got.isnan(), want.isnan())
    inf_alike = torch.equal(got[inf], want[inf])
    assert nan_alike and inf_alike, what
    off = (got - want).abs()[fine]
    within = bool((off <= torch.broadcast_to(tol, want.shape)[fine]).all())
    assert within, (what, float(off.max()))


def _case(R, B, H, G, P, cap, seed, edit):
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, cap + 1, (B, H), generator=g, dtype=torch.int32)
    lens[0, 0] = cap
    c = R.TokenCache.empty(B, H, G, cap, DEV)
    s = {"lens": lens,
         "q": torch.randn(B, H * G, D, generator=g).bfloat16(),
         "K": torch.randn(B, H, cap, D, generator=g).bfloat16(),
         "V": torch.randn(B, H, cap, D, generator=g).bfloat16(),
         "PK": torch.randn(H, P, D, generator=g).bfloat16(),
         "PV": torch.randn(H, P, D, generator=g).bfloat16()}
    s["q"][..., 3] = s["q"][..., 3].abs() + 0.5  # one sign: keys of -inf there score -inf
    edit(s)
    s = {k: t.to(DEV) for k, t in s.items()}
    c.K.copy_(s["K"])
    c.V.copy_(s["V"])
    c.lens.copy_(s["lens"])
    w0 = torch.rand(B, H, cap, generator=g).to(DEV)
    c.weight.copy_(w0)
    ws = R.alloc_workspace(R.token_attend_workspace_bytes(c, P), DEV)
    prefix = (s["PK"], s["PV"]) if P else None
    out, lse = R.token_attend(s["q"], c, prefix, workspace=ws)
    assert R.read_device_status(ws) == 0
    for b in range(B):
        for h in range(H):
            n = int(lens[b, h])
            rows = slice(h * G, (h + 1) * G)
            q = s["q"][b, rows].double()
            keys = torch.cat((s["PK"][h], s["K"][b, h, :n])).double()
            vals = torch.cat((s["PV"][h], s["V"][b, h, :n])).double()
            want, want_l, p, mean = _formula(q, keys, vals)
            norm = keys[keys.isfinite().all(-1)].norm(dim=-1)
            e = 128 * 2.0 ** -23 * float(norm.max() if len(norm) else 0.0) * float(
                q.nan_to_num(0.0, 0.0, 0.0).norm(dim=-1).max()) / math.sqrt(D)
            off = math.expm1(2 * e) + 2.0 ** -18
            at = (b, h)
            _near(out[b, rows], want, ((off + 2 * 2.0 ** -8 / (1 - 2.0 ** -8)) * mean
                                       + 2.0 ** -8 * want.abs()) * (1 + 2.0 ** -8), ("out", at))
            _near(lse[b, rows], want_l, e + 2.0 ** -18 + 2.0 ** -22 * want_l.abs(), ("lse", at))
            add = p[:, P:].sum(0)
            tol = add * (off + 2.0 ** -20) + (w0[b, h, :n].double() + add) * 2.0 ** -23 + 2e-37
            _near(c.weight[b, h, :n], w0[b, h, :n].double() + add, tol, ("weight", at))
            behind = torch.equal(c.weight[b, h, n:], w0[b, h, n:])
            assert behind, at


# own tokens alone; a prefix of one tile; a pair of row tiles and a single one,
# several key tiles to a share; one row tile with several key tiles to a share
SHAPES = [(3, 2, 4, 0, 40), (2, 1, 7, 1, 3), (2, 2, 4, 700, 300), (65, 1, 4, 20011, 40),
          (2, 1, 8, 80000, 600)]


def _set(name, *index):
    def edit(s, value):
        if s[name].numel():
            s[name][index] = value
    return edit


def _every_key(s, value):
    s["K"][..., 3] = value
    s["PK"][..., 3] = value


WHERE = {
    "query": _set("q", slice(None), 1, 5),
    "own_key": _set("K", slice(None), slice(None), 0, 3),
    "own_tile": _set("K", slice(None), slice(None), slice(0, 16), 3),
    "own_keys": _set("K", Ellipsis, 3),
    "prefix_key": _set("PK", slice(None), -1, 3),
    "prefix_first": _set("PK", slice(None), 0, 3),
    "prefix_tiles": _set("PK", slice(None), slice(0, 640), 3),
    "prefix_half": _set("PK", slice(None), slice(0, None, 2), 3),
    "prefix_keys": _set("PK", Ellipsis, 3),
    "every_key": _every_key,
    "own_value": _set("V", slice(None), slice(None), 0, 7),
    "prefix_value": _set("PV", slice(None), -1, 7),
}


@pytest.mark.parametrize("where", ["query", "own_key", "own_keys", "prefix_key", "prefix_tiles",
                                   "prefix_keys", "every_key"])
def test_attend_nan(R, where):
    """A NaN in a query or a key makes its rows NaN: out, lse and weights."""
    for i, shape in enumerate(SHAPES):
        _case(R, *shape, i, lambda s: WHERE[where](s, NAN))


@pytest.mark.parametrize("where", ["query", "own_key", "own_keys", "prefix_key", "prefix_tiles",
                                   "prefix_keys", "every_key"])
def test_attend_infinite_score(R, where):
    """A score of +inf has no finite probability: its row is NaN."""
    for i, shape in enumerate(SHAPES):
        _case(R, *shape, i, lambda s: WHERE[where](s, INF))


@pytest.mark.parametrize("where", ["own_key", "own_tile", "own_keys", "prefix_first",
                                   "prefix_tiles", "prefix_half", "prefix_keys", "every_key"])
def test_attend_minus_infinite_score(R, where):
    """A score of -inf has weight 0, in a first tile, a whole share or everywhere."""
    for i, shape in enumerate(SHAPES):
        _case(R, *shape, i, lambda s: WHERE[where](s, -INF))


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["own_value", "prefix_value"])
def test_attend_values(R, where, value):
    """A value's NaN or infinity reaches its column of the output and no other."""
    for i, shape in enumerate(SHAPES):
        _case(R, *shape, i, lambda s: WHERE[where](s, value))


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["own_value", "prefix_value"])
def test_attend_values_of_equal_scores(R, where, value):
    """The same with probabilities that a bf16 holds exactly."""
    def edit(s):
        WHERE[where](s, value)
        s["q"].zero_()
    for i, shape in enumerate(SHAPES):
        _case(R, *shape, i, edit)


@pytest.mark.parametrize("where", ["own_value", "prefix_value"])
def test_attend_nan_value_of_no_weight(R, where):
    """A NaN value counts however small its probability is (0 * NaN is NaN)."""
    def edit(s):
        WHERE[where](s, NAN)
        # far below every other score: the probability is 0 in fp32, in a tile or
        # a share of its own
        name = "K" if where == "own_value" else "PK"
        WHERE["own_tile" if name == "K" else "prefix_tiles"](s, -2000.0)
        if name == "PK" and s["PV"].shape[1]:
            s["PV"][:, 0, 7] = NAN
    for i, shape in enumerate(SHAPES):
        _case(R, *shape, i, edit)
