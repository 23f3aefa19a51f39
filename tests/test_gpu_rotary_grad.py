"""Gradients through rotary positions, against the formula (the transposed
rotation of the output's gradient) in 64 bits and against differences.

Tolerance of a rotated element, from the kernel's arithmetic: the angle's
fraction of a turn is cut to 32 bits (2 pi 2^-32 radians), taken to fp32 (2^-24
of at most pi / 4) and scaled by a rounded constant and a rounded product (2 *
2^-24 of pi / 4); the polynomials are off by 8.1e-9 and 5.9e-10, and their
roundings by less than 3 * 2^-24 together; the magnitude's product, the
rotation's two products and the sum are rounded, 4 * 2^-24: in all less than
10 * 2^-24 = 6e-7 of mag (|a| + |b|); and half a step of the stored type.
"""
import numpy as np
import pytest
import torch

from oracle import token_cache as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ANGLE = 6e-7


@pytest.fixture(scope="module")
def R():
    import kv_cache_vector_segmented_b200 as R
    return R


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(got, x, pos, n, f, mag, interleaved, inverse):
    want = T.rotary(x, pos, f, mag, interleaved, inverse)
    tol = np.abs(want) * torch.finfo(got.dtype).eps / 2 + (2.0 ** -25 if got.dtype ==
                                                            torch.float16 else 0)
    # |a| + |b| of a pair is at most twice the head's largest element
    tol = tol + 2 * np.abs(x).max(-1, keepdims=True) * ANGLE * mag * (1 + torch.finfo(
        got.dtype).eps)
    off = np.abs(_np(got) - want)
    assert (off <= tol).all(), float((off - tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [128, 20])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_gradient(R, dtype, interleaved, n, inverse):
    """Dense, sliced and transposed inputs; gradients of any layout."""
    B, Tn, H = 2, 5, 3
    g = torch.Generator().manual_seed(n)
    t = R.RotaryTable.make(n, scaling="yarn", factor=4.0, interleaved=interleaved, device=DEV)
    f, mag = T.frequencies(n, 10000.0, "yarn", 4.0)
    pos = torch.randint(0, 100000, (B, Tn), generator=g).to(torch.int32)
    for layout in ("dense", "slice", "heads_first"):
        base = torch.randn(B, Tn, H + 2, 128, generator=g).to(dtype).to(DEV).requires_grad_()
        x = {"dense": base, "slice": base[:, :, 1:-1],
             "heads_first": base.transpose(1, 2).contiguous().transpose(1, 2)}[layout]
        y = R.rotary(x, pos.to(DEV), t, inverse=inverse)
        assert y.requires_grad
        _near(y, _np(x), pos.numpy(), n, f, mag, interleaved, inverse)
        with torch.no_grad():
            z = R.rotary(x, pos.to(DEV), t, inverse=inverse)
        assert not z.requires_grad and torch.equal(y, z)
        w = torch.randn(y.shape, generator=g).to(dtype).to(DEV)
        if layout == "heads_first":
            w = w.transpose(1, 2).contiguous().transpose(1, 2)
        (grad,) = torch.autograd.grad(y, base, w)
        got = grad[:, :, 1:-1] if layout == "slice" else grad
        _near(got, _np(w), pos.numpy(), n, f, mag, interleaved, not inverse)
        if layout == "slice":
            assert (grad[:, :, 0] == 0).all() and (grad[:, :, -1] == 0).all()


def test_rotary_gradient_of_a_sum_and_of_a_broadcast(R):
    """A gradient that repeats one element; an input that all sequences share."""
    B, Tn, H, n = 3, 4, 2, 128
    t = R.RotaryTable.make(n, device=DEV)
    f, mag = T.frequencies(n, 10000.0)
    pos = torch.arange(B * Tn, dtype=torch.int32).view(B, Tn)
    x = torch.randn(1, Tn, H, 128, device=DEV, requires_grad=True)
    R.rotary(x.expand(B, Tn, H, 128), pos.to(DEV), t).sum().backward()
    one = np.ones((B, Tn, H, 128))
    want = T.rotary(one, pos.numpy(), f, mag, inverse=True).sum(0, keepdims=True)
    # B elements of at most 2 + 2 * ANGLE each, summed with B roundings
    assert (np.abs(_np(x.grad) - want) <= B * 2 * ANGLE + B * B * 2.0 ** -23).all()


def test_rotary_gradient_against_differences(R):
    """The map is linear: a unit step's difference is the derivative, but for
    the roundings of both sides."""
    B, Tn, H, n = 1, 3, 2, 64
    g = torch.Generator().manual_seed(1)
    t = R.RotaryTable.make(n, interleaved=True, device=DEV)
    pos = torch.randint(0, 1000, (B, Tn), generator=g).to(torch.int32).to(DEV)
    x = torch.randn(B, Tn, H, 128, generator=g).to(DEV).requires_grad_()
    w = torch.randn(B, Tn, H, 128, generator=g).to(DEV)
    (R.rotary(x, pos, t) * w).sum().backward()
    base = _np(R.rotary(x.detach(), pos, t))
    for at in ((0, 0, 0, 0), (0, 2, 1, 33), (0, 1, 0, 100)):
        step = x.detach().clone()
        step[at] += 1.0
        diff = ((_np(R.rotary(step, pos, t)) - base) * _np(w)).sum()
        # two elements change (or one); each side is off by ANGLE (|a| + |b|)
        # and the step by 2^-24 of the element
        top, scale = np.abs(_np(x)).max() + 1, np.abs(_np(w)).max()
        assert abs(diff - float(x.grad[at])) <= (2 * 2 * 2 * top + 2) * ANGLE * scale + \
            top * 2.0 ** -24 * 2 * scale


def test_rotary_second_gradient(R):
    """The gradient is itself a rotation of the output's gradient."""
    t = R.RotaryTable.make(128, device=DEV)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    x = torch.randn(1, 4, 2, 128, device=DEV, requires_grad=True)
    w = torch.randn(1, 4, 2, 128, device=DEV, requires_grad=True)
    (grad,) = torch.autograd.grad(R.rotary(x, pos, t), x, w, create_graph=True)
    v = torch.randn_like(x)
    (again,) = torch.autograd.grad(grad, w, v)
    assert torch.equal(again, R.rotary(v, pos, t))
