"""Layouts that the documentation allows: strides of extents of one (torch leaves
them at any value), and an eviction's result in every mix of own and other arrays."""
import itertools

import numpy as np
import pytest
import torch

from oracle import token_cache as T

gpu = pytest.mark.gpu
DEV = "cuda:0"
D = 128


@pytest.fixture(scope="module")
def R():
    import kv_cache_vector_segmented_b200 as R
    return R


def _odd(t, *dims):
    """The same elements, the extents of one among `dims` with an odd stride."""
    strides = list(t.stride())
    for d in dims:
        assert t.shape[d] == 1
        strides[d] = 12345 + d
    return t.as_strided(t.shape, strides)


def test_strides_of_one_do_not_matter(R):
    """Without a GPU: the structs of two such views are the same."""
    from kv_cache_vector_segmented_b200 import _tokens as C
    x = torch.zeros(1, 1, 1, D, dtype=torch.bfloat16)
    a, b = (C._heads(t, "x", x.dtype, x.shape, x.device) for t in (x, _odd(x, 0, 1, 2)))
    assert [getattr(a, f) for f, _ in a._fields_] == [getattr(b, f) for f, _ in b._fields_]
    y = torch.zeros(2, 3, 4, D, dtype=torch.bfloat16)
    c = C._heads(y, "y", y.dtype, y.shape, y.device)
    assert (c.stride_b, c.stride_t, c.stride_h) == y.stride()[:3]


@gpu
def test_rotary_and_append_with_strides_of_one(R):
    t = R.RotaryTable.make(D, device=DEV)
    for B, Tn, H, dims in ((1, 1, 1, (0, 1, 2)), (1, 5, 3, (0,)), (4, 1, 2, (1,)),
                           (3, 2, 1, (2,))):
        g = torch.Generator().manual_seed(B)
        x = torch.randn(B, Tn, H, D, generator=g).bfloat16().to(DEV)
        pos = torch.randint(0, 1000, (B, Tn), generator=g).int().to(DEV)
        want = R.rotary(x, pos, t)
        assert torch.equal(R.rotary(_odd(x, *dims), pos, t), want)
        y = x.clone()  # in place, under another view of the same elements
        R.rotary(y, pos, t, out=_odd(y, *dims))
        assert torch.equal(y, want)
        got = []
        for view in (x, _odd(x, *dims)):
            c = R.TokenCache.empty(B, H, 1, 8, DEV)
            c.K.zero_()
            c.V.zero_()
            q = R.token_append(c, view, view, pos, t, q=view)
            assert R.read_device_status(c.status) == 0
            got.append((q, c.K, c.V, c.pos, c.lens))
        assert all(torch.equal(a, b) for a, b in zip(*got))


@gpu
def test_prefix_with_strides_of_one(R):
    """Prefix K and V of one head, or of one token, from buffers of their own."""
    for H, P, dims in ((1, 77, (0,)), (3, 1, (1,)), (1, 1, (0, 1))):
        g = torch.Generator().manual_seed(P)
        c = R.TokenCache.empty(2, H, 4, 16, DEV)
        c.K.copy_(torch.randn(c.K.shape, generator=g))
        c.V.copy_(torch.randn(c.V.shape, generator=g))
        c.lens.fill_(9)
        q = torch.randn(2, 4 * H, D, generator=g).bfloat16().to(DEV)
        K, V = (torch.randn(H, P, D, generator=g).bfloat16().to(DEV) for _ in range(2))
        want = R.token_attend(q, c, (K, V), add_weight=False)
        for k, v in ((_odd(K, *dims), V), (K, _odd(V, *dims)), (_odd(K, *dims), _odd(V, *dims))):
            got = R.token_attend(q, c, (k, v), add_weight=False)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


NAMES = ("K", "V", "pos", "weight", "lens")


@gpu
@pytest.mark.parametrize("heads,cap,budget", [(4, 300, 90), (4, 300, 400), (2, 9000, 4500)])
def test_evict_into_any_mix_of_arrays(R, heads, cap, budget):
    """Every array of the result the cache's own or another: in one launch, with
    nothing to drop, and with a launch of its own for the moves."""
    first, recent = 3, 20
    for apart in itertools.product((False, True), repeat=5):
        g = torch.Generator().manual_seed(budget)
        c = R.TokenCache.empty(1, heads, 1, cap, DEV)
        for t in (c.K, c.V, c.weight):
            t.copy_(torch.randn(t.shape, generator=g))
        c.pos.copy_(torch.rand(c.pos.shape, generator=g).argsort(-1))
        c.lens.copy_(torch.randint(0, cap + 1, (1, heads), generator=g))
        c.lens[0, 0] = cap
        before = {n: getattr(c, n).clone() for n in NAMES}
        other = {n: torch.full_like(before[n], -9) for n in NAMES}
        out = R.TokenCache(*(other[n] if a else getattr(c, n) for n, a in zip(NAMES, apart)))
        ws = R.alloc_workspace(R.token_evict_workspace_bytes(c, budget), DEV)
        R.token_evict(c, budget, first, recent, out=out, workspace=ws)
        assert R.read_device_status(ws) == 0
        for h in range(heads):
            n = int(before["lens"][0, h])
            src = torch.from_numpy(T.evict(before["pos"][0, h, :n].cpu().numpy(),
                                           before["weight"][0, h, :n].cpu().numpy(), budget,
                                           first, recent)).to(DEV)
            m = len(src)
            assert int(out.lens[0, h]) == m
            for name, a in zip(NAMES[:4], apart):
                got, old = getattr(out, name)[0, h], before[name][0, h]
                assert torch.equal(got[:m], old[src]), (apart, h, name)
                assert torch.equal(got[m:], torch.full_like(old[m:], -9) if a else old[m:])
        for name, a in zip(NAMES, apart):
            assert not a or torch.equal(getattr(c, name), before[name]), (apart, name)


@pytest.mark.parametrize("weights", [[.5, .1, .9, .7, .3], [float("nan")] * 5])
def test_held_beyond_the_budget_stay_by_row(weights):
    """Without a GPU, by hand: where more tokens are held than the budget (equal
    positions, say), the lowest rows of them stay, whatever their weights."""
    w = np.array(weights)
    assert T.evict(np.array([7, 7, 7, 7, 7]), w, 2, 0, 1).tolist() == [0, 1]
    assert T.evict(np.array([9, 0, 9, 1, 9]), w, 2, 2, 0).tolist() == [3, 1]
    assert T.evict(np.array([9, 0, 9, 1, 9]), w, 3, 2, 1).tolist() == [0, 1, 2]
