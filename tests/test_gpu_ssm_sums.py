"""The selective scan's sums over batch and time (dbeta, dw_r) where they cancel: half the sequences have the other
half's gradients with the other sign, so a sum in fp32 would keep the rounding of partial sums much larger than the result.

Tolerances are six standard deviations of the roundings that are left, each at most 2^-24 of its value and taken as
evenly distributed (2^-24 / sqrt 3).  dw_r: every product, the four levels of sums of 16 steps, a chunk's sum.
dbeta against the sum of the returned da: the rounding of every da; and the result's own rounding.
"""
import numpy as np
import pytest

from _gpu import say, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("V", [16, 64])
@pytest.mark.parametrize("B", [64, 66])  # 2048 chunks are one launch of the sums, more are two
def test_sums_that_cancel(B, V):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("ssm sums", B, V)
    T, N, K, L = 1024, 1, 16, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    x = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)  # noqa: E731
    q, k = x(B, T, 1, K).abs() * K ** -0.5, x(B, T, 1, K).abs() * K ** -0.5
    v, a = x(B, T, N, V).abs() + 1.0, x(B, T, N)
    alpha, beta, w_r = torch.full((N,), 0.5, device="cuda"), torch.full((N,), -2.0, device="cuda"), x(N, V)
    dy = torch.ones(B, T, N, V, device="cuda")
    dy[B // 2:] = -1.0
    args = (q, k, v, a, alpha, beta, w_r)
    ckpt = m2.m2rnn_ssm_fwd_ckpt(*args)[2]
    d = m2.m2rnn_ssm_bwd(*args, ckpt, dy)

    terms = (v.double() * dy.double())[:, :, 0].cpu().numpy()      # [B, T, V]
    level, var = terms, 0.0
    for _ in range(5):                                             # products, then sums of 2, 4, 8 and 16 of them
        var = var + np.sum(level ** 2, axis=(0, 1))
        level = level[:, 0::2] + level[:, 1::2]
    var = var + np.sum(terms.reshape(B, T // L, L, V).sum(2) ** 2, axis=(0, 1))
    ref = terms.sum((0, 1))
    tol = 6 * U * np.sqrt(var / 3) + U * np.abs(ref)
    err = np.abs(d["dw_r"][0].double().cpu().numpy() - ref)
    say("dw_r worst error over its bound: %.3g" % float(np.max(err / tol)))
    assert np.all(err <= tol)

    da = d["da"].double().cpu().numpy()
    assert abs(da[:B // 2].sum()) > 10 * abs(da.sum())             # (the case is what it is meant to be)
    ref = da.sum()
    tol = 6 * U * np.sqrt(np.sum(da ** 2) / 3) + U * abs(ref)
    err = abs(float(d["dbeta"][0]) - ref)
    say("dbeta error over its bound: %.3g" % (err / tol))
    assert err <= tol
