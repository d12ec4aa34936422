"""Pins of the fp64 oracle of the q/k norm with rotation: identities of rotations, torch autograd in
fp64 and central differences."""
import numpy as np
import pytest
import torch

from oracle import qk


def freq(R):
    return 10000.0 ** (-np.arange(0, R, 2) / max(R, 1))


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(inter):
    r = np.random.default_rng(1)
    x, y = r.normal(0, 1, (1, 4, 2, 12)), r.normal(0, 1, (1, 4, 2, 12))
    p = np.array([[0, 5, 100, 31]])
    a, b = (qk.turn(z, p, freq(8), inter) for z in (x, y))
    np.testing.assert_allclose((a * a).sum(-1), (x * x).sum(-1), rtol=1e-12)
    np.testing.assert_array_equal(a[..., 8:], x[..., 8:])
    np.testing.assert_array_equal(a[:, 0], x[:, 0])
    # the product of two turned heads depends on the difference of their positions only
    c, d = (qk.turn(z, p + 77, freq(8), inter) for z in (x, y))
    np.testing.assert_allclose(a[0, 1] @ b[0, 3].T, c[0, 1] @ d[0, 3].T, rtol=1e-10)
    np.testing.assert_allclose(qk.turn(a, p, freq(8), inter, -1.0), x, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("inter,R", [(False, 8), (True, 8), (False, 16), (True, 0)])
def test_backward_matches_autograd_and_differences(inter, R):
    r = np.random.default_rng(2)
    x, gamma, do = r.normal(0, 1, (2, 3, 2, 16)), r.normal(1, 0.3, 16), r.normal(0, 1, (2, 3, 2, 16))
    pos = r.integers(-5, 1000, (2, 3))
    f = freq(R)
    dx, dg = qk.norm_rope_bwd(x, gamma, pos, f, 1e-3, inter, do)
    tx, tg = (torch.tensor(z, requires_grad=True) for z in (x, gamma))
    xn = tg * tx * torch.rsqrt((tx * tx).mean(-1, keepdim=True) + 1e-3)
    a, b = qk.pairs(16, R, inter)
    t = torch.tensor(pos[:, :, None, None] * f)
    loss = 0.0
    d = torch.tensor(do)
    turned = {int(i): xn[..., i] * t[..., p].cos() - xn[..., j] * t[..., p].sin() for p, (i, j) in enumerate(zip(a, b))}
    turned.update({int(j): xn[..., j] * t[..., p].cos() + xn[..., i] * t[..., p].sin() for p, (i, j) in enumerate(zip(a, b))})
    for i in range(16):
        loss = loss + (turned.get(i, xn[..., i]) * d[..., i]).sum()
    loss.backward()
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dg, tg.grad.numpy(), rtol=1e-10, atol=1e-12)
    value = lambda z, g: float((qk.norm_rope_fwd(z, g, pos, f, 1e-3, inter) * do).sum())  # noqa: E731
    np.testing.assert_allclose(value(x, gamma), float(loss.detach()), rtol=1e-12)
    for z, grad, first in ((x, dx, True), (gamma, dg, False)):
        for i in r.integers(0, z.size, 5):
            lo, hi = z.copy(), z.copy()
            lo.flat[i] -= 1e-6
            hi.flat[i] += 1e-6
            num = (value(hi, gamma) - value(lo, gamma) if first else value(x, hi) - value(x, lo)) / 2e-6
            np.testing.assert_allclose(grad.flat[i], num, rtol=1e-6, atol=1e-8)
