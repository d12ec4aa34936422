"""Pins of the fp64 oracle of the layer's entry, the gated recurrence of channels and the orthogonalised update: closed
forms, torch autograd in fp64, central differences and singular values."""
import numpy as np
import pytest
import torch

from oracle import layer


def test_norm_rows_have_unit_mean_square_and_forget_their_scale():
    r = np.random.default_rng(1)
    h = r.normal(0, 3, (5, 24))
    out = layer.norm_fwd(h, np.ones(24), 0.0)
    np.testing.assert_allclose((out * out).mean(-1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(layer.norm_fwd(h * 1e6, np.ones(24), 0.0), out, rtol=1e-12)


@pytest.mark.parametrize("stream", [False, True])
def test_norm_backward_matches_autograd_and_differences(stream):
    r = np.random.default_rng(2)
    h, g, do, dh = r.normal(0, 1, (4, 12)), r.normal(1, 0.3, 12), r.normal(0, 1, (4, 12)), r.normal(0, 1, (4, 12))
    dx, dg = layer.norm_bwd(h, g, 1e-3, do, dh if stream else None)
    th, tg = (torch.tensor(z, requires_grad=True) for z in (h, g))
    loss = (tg * th * torch.rsqrt((th * th).mean(-1, keepdim=True) + 1e-3) * torch.tensor(do)).sum()
    if stream:
        loss = loss + (th * torch.tensor(dh)).sum()
    loss.backward()
    np.testing.assert_allclose(dx, th.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dg, tg.grad.numpy(), rtol=1e-10, atol=1e-12)
    f = lambda z: float((layer.norm_fwd(z, g, 1e-3) * do).sum() + (z * dh).sum() * stream)  # noqa: E731
    for i in (0, 17, 47):
        e = np.zeros(h.size)
        e[i] = 1e-6
        e = e.reshape(h.shape)
        np.testing.assert_allclose(dx.flat[i], (f(h + e) - f(h - e)) / 2e-6, rtol=1e-6, atol=1e-8)


def gated_inputs(B, T, D, seed):
    r = np.random.default_rng(seed)
    return r.normal(0, 1, (B, T, D)), r.normal(0, 2, (B, T, D)), r.uniform(0.2, 3, D), r.normal(0, 1, D), r.normal(0, 1, (B, D))


def test_gated_recurrence_closed_forms():
    v, a, alpha, beta, h0 = gated_inputs(2, 7, 3, 3)
    # alpha = 1: f is the logistic function of -(a + beta)
    f = layer.gate(a, np.ones(3), beta)[2]
    np.testing.assert_allclose(f, 1.0 / (1.0 + np.exp(a + beta)), rtol=1e-12)
    # the sum over steps, without a loop over states
    _, _, f, i = layer.gate(a, alpha, beta)
    y, h, _ = layer.gated_fwd(v, a, alpha, beta, h0)
    ref = np.prod(f, 1) * h0
    for t in range(7):
        ref = ref + np.prod(f[:, t + 1:], 1) * i[:, t] * v[:, t]
    np.testing.assert_allclose(h, ref, rtol=1e-12)
    np.testing.assert_array_equal(y[:, -1], h)
    # a constant input is a fixed point, and the state stays within the inputs' range
    c = np.broadcast_to(h0[:, None], v.shape)
    np.testing.assert_allclose(layer.gated_fwd(c, a, alpha, beta, h0)[0], c, rtol=1e-12)
    assert np.abs(y).max() <= max(np.abs(v).max(), np.abs(h0).max())
    # masked steps and steps past the end hold the state, whatever v is
    am, vm = a.copy(), v.copy()
    am[:, 3] = -np.inf
    vm[:, 3] = np.nan
    ym, hm, _ = layer.gated_fwd(vm, am, alpha, beta, h0)
    np.testing.assert_array_equal(ym[:, 3], ym[:, 2])
    cut = np.delete(np.arange(7), 3)
    np.testing.assert_allclose(hm, layer.gated_fwd(v[:, cut], a[:, cut], alpha, beta, h0)[1], rtol=1e-12)
    yl, hl, _ = layer.gated_fwd(v, a, alpha, beta, h0, [4, 0])
    np.testing.assert_array_equal(hl[0], y[0, 3])
    np.testing.assert_array_equal(hl[1], h0[1])
    assert not yl[0, 4:].any() and not yl[1].any()


@pytest.mark.parametrize("lens", [None, [5, 2]])
def test_gated_backward_matches_autograd_and_differences(lens):
    v, a, alpha, beta, h0 = gated_inputs(2, 6, 3, 4)
    r = np.random.default_rng(5)
    dy, dh = r.normal(0, 1, v.shape), r.normal(0, 1, h0.shape)
    got, _, _ = layer.gated_bwd(v, a, alpha, beta, dy, dh, h0, lens)
    t = {n: torch.tensor(x, requires_grad=True) for n, x in dict(v=v, a=a, alpha=alpha, beta=beta, h0=h0).items()}
    h, loss = t["h0"], 0.0
    n = torch.tensor([6, 6] if lens is None else lens)[:, None]
    for i in range(6):
        f = torch.exp(-t["alpha"] * torch.nn.functional.softplus(t["a"][:, i] + t["beta"], threshold=1e9))
        h = torch.where(i < n, f * h + (1 - f) * t["v"][:, i], h)
        loss = loss + (torch.where(i < n, h, 0.0 * h) * torch.tensor(dy[:, i])).sum()
    (loss + (h * torch.tensor(dh)).sum()).backward()
    for name, x in (("dv", "v"), ("da", "a"), ("dalpha", "alpha"), ("dbeta", "beta"), ("dh0", "h0")):
        np.testing.assert_allclose(got[name], t[x].grad.numpy(), rtol=1e-9, atol=1e-11)

    def value(**kw):
        p = dict(v=v, a=a, alpha=alpha, beta=beta, h0=h0)
        p.update(kw)
        y, hT, _ = layer.gated_fwd(p["v"], p["a"], p["alpha"], p["beta"], p["h0"], lens)
        return float((y * dy).sum() + (hT * dh).sum())
    for name, x, grad in (("a", a, "da"), ("alpha", alpha, "dalpha"), ("h0", h0, "dh0")):
        e = np.zeros(x.size)
        e[1] = 1e-6
        e = e.reshape(x.shape)
        num = (value(**{name: x + e}) - value(**{name: x - e})) / 2e-6
        np.testing.assert_allclose(got[grad].flat[1], num, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("m,n", [(5, 9), (9, 5), (6, 6), (1, 4)])
@pytest.mark.parametrize("coefs", [(3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0)])
def test_orthogonalized_singular_values(m, n, coefs):
    g = np.random.default_rng(6).normal(0, 2, (m, n))
    out = layer.orthogonalize(g, 5, coefs, 1e-7)
    U, s, Vt = np.linalg.svd(g, full_matrices=False)
    s = s / (np.sqrt((s * s).sum()) + 1e-7)
    for _ in range(5):
        s = coefs[0] * s + coefs[1] * s ** 3 + coefs[2] * s ** 5
    np.testing.assert_allclose(out, (U * s) @ Vt, rtol=1e-10, atol=1e-12)


def test_cubic_steps_converge_to_the_orthogonal_factor():
    g = np.random.default_rng(7).normal(0, 1, (4, 4)) + 3 * np.eye(4)
    U, _, Vt = np.linalg.svd(g)
    np.testing.assert_allclose(layer.orthogonalize(g, 40, (1.5, -0.5, 0.0), 0.0), U @ Vt, atol=1e-10)
