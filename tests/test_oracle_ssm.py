"""Pins of the fp64 oracle of the selective state space scan and the convolution with a window: the
closed form without a loop, torch autograd in fp64, central differences, and the block oracle."""
import numpy as np
import pytest
import torch

from oracle import block, ssm


def case(B, T, N, G, K, V, seed):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(0, 1, (B, T, G, K)), k=r.normal(0, 1, (B, T, G, K)), v=r.normal(0, 1, (B, T, N, V)),
                a=r.normal(0, 1, (B, T, N)), alpha=r.uniform(0.1, 2.0, N), beta=r.normal(0, 1, N),
                w_r=r.normal(0, 1, (N, V)), H0=r.normal(0, 1, (B, N, K, V)))


def test_forward_is_its_sum_over_earlier_steps():
    d = case(2, 7, 4, 2, 3, 5, 1)
    y, HT = ssm.fwd(**d)
    D = np.logaddexp(0, d["a"] + d["beta"])
    lf = -d["alpha"] * D
    q, k = (np.repeat(d[x], 2, axis=2) for x in "qk")
    for b in range(2):
        for n in range(4):
            for t in range(7):
                H = np.exp(lf[b, :t + 1, n].sum()) * d["H0"][b, n]
                for j in range(t + 1):
                    H = H + np.exp(lf[b, j + 1:t + 1, n].sum()) * D[b, j, n] * np.outer(k[b, j, n], d["v"][b, j, n])
                np.testing.assert_allclose(y[b, t, n], H.T @ q[b, t, n] + d["w_r"][n] * d["v"][b, t, n], rtol=1e-12)
            np.testing.assert_allclose(HT[b, n], H, rtol=1e-12)


@pytest.mark.parametrize("lens", [None, [5, 0], [6, 2]])
def test_backward_matches_autograd_and_differences(lens):
    d = case(2, 6, 4, 2, 3, 2, 2)
    r = np.random.default_rng(3)
    dy, dHT = r.normal(0, 1, (2, 6, 4, 2)), r.normal(0, 1, d["H0"].shape)
    lens_a = None if lens is None else np.array(lens)
    g = ssm.bwd(dy=dy, dH_T=dHT, lens=lens_a, **d)
    t = {n: torch.tensor(x, dtype=torch.float64, requires_grad=True) for n, x in d.items()}
    H, loss = t["H0"], 0.0
    D = torch.nn.functional.softplus(t["a"] + t["beta"])
    for s in range(6):
        on = torch.tensor([1.0 if lens is None or s < n else 0.0 for n in (lens or [0, 0])], dtype=torch.float64)
        Ds = D[:, s] * on[:, None]
        q, k = (t[x][:, s].repeat_interleave(2, 1) for x in "qk")
        H = torch.exp(-t["alpha"] * Ds)[..., None, None] * H + (Ds[..., None] * k)[..., None] * t["v"][:, s, :, None]
        y = ((H * q[..., None]).sum(2) + t["w_r"] * t["v"][:, s]) * on[:, None, None]
        loss = loss + (y * torch.tensor(dy[:, s])).sum()
    (loss + (H * torch.tensor(dHT)).sum()).backward()
    for n, x in t.items():
        np.testing.assert_allclose(g["d" + n], x.grad.numpy(), rtol=1e-11, atol=1e-12, err_msg=n)

    def value(**e):
        y, HT = ssm.fwd(lens=lens_a, **e)
        return float((y * dy).sum() + (HT * dHT).sum())
    for n in d:
        for i in r.integers(0, d[n].size, 4):
            lo, hi = dict(d), dict(d)
            lo[n], hi[n] = d[n].copy(), d[n].copy()
            lo[n].flat[i] -= 1e-5
            hi[n].flat[i] += 1e-5
            np.testing.assert_allclose(g["d" + n].flat[i], (value(**hi) - value(**lo)) / 2e-5, rtol=1e-6, atol=1e-7)


def test_window_convolution_continues_the_block_oracle():
    r = np.random.default_rng(4)
    x, w, b = r.normal(0, 1, (2, 9, 8)), r.normal(0, 1, (8, 4)), r.normal(0, 1, 8)
    whole = block.conv4_silu_fwd(x, w, b)
    for cut in (0, 1, 2, 5, 9):
        u0, win = ssm.conv4_silu_window(x[:, :cut], w, b, None)
        u1, last = ssm.conv4_silu_window(x[:, cut:], w, b, win)
        np.testing.assert_allclose(np.concatenate([u0, u1], 1), whole, rtol=1e-13)
        np.testing.assert_array_equal(last, x[:, 6:])
    u, win = ssm.conv4_silu_window(x, w, b, None, lens=np.array([4, 0]))
    np.testing.assert_allclose(u[0, :4], whole[0, :4], rtol=1e-13)
    assert not u[0, 4:].any() and not u[1].any() and not win[1].any()
    np.testing.assert_array_equal(win[0], x[0, 1:4])
