"""The gated recurrence where its chunks' maps are joined over more than one look (over 128 chunks: above 8192 steps forward, 4096 backward),
with memories that reach across all of them; its backward where gates are 0, 1 or above; single steps with masked gates.

Tolerances are those of test_gpu_gated.py; the backward's are summed in `backward_bounds` as they are there, with |1 - f| for gates
above 1.
"""
import numpy as np
import pytest

from _gpu import say, torch_cuda
from oracle import layer
from test_gpu_gated import U, f64, made, near, terms, test_forward_and_backward as check_both

pytestmark = pytest.mark.gpu

# chunks of the forward in groups of 16: the last chunk is the 5th, the 12th, the 1st and the 9th of its group
LONG = [(1, 8500, 8, "fp32", None, True), (1, 8900, 8, "bf16", None, False), (2, 16421, 4, "fp32", [16421, 9001], True),
        (3, 17921, 4, "bf16", [8193, 0, 17921], True), (5, 4200, 12, "fp32", [4200, 4097, 64, 4160, 1], True)]


@pytest.mark.parametrize("B,T,D,dtype,lens,h0", LONG)
def test_more_than_128_chunks(B, T, D, dtype, lens, h0):
    check_both(B, T, D, dtype, lens, h0, True)


def test_the_state_crosses_all_groups():
    """Gates that hold nearly everything: the first and the last state depend on each other through every join."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    B, T, D = 1, 12000, 4
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    alpha, beta = torch.full((D,), 1.0, device="cuda"), torch.full((D,), -12.0, device="cuda")
    h0, dh = torch.randn(B, D, device="cuda"), torch.randn(B, D, device="cuda")
    v, a = z(B, T, D), z(B, T, D)
    y, hT = m2.m2rnn_gated_scan_fwd(v, a, alpha, beta, h0)
    f = np.exp(-T * np.log1p(np.exp(-12.0)))  # 0.929
    for got, ref in ((hT, h0), (m2.m2rnn_gated_scan_bwd(v, a, alpha, beta, y, z(B, T, D), h0, dh)["dh0"], dh)):
        # each step's 1 - f is off by at most 36 u of itself (24 + |z|), so the product by that share of its logarithm, and each of the
        # steps' and joins' products is rounded
        tol = (36 * U * -np.log(f) + 8 * U * T) * np.abs(f64(ref)) * f
        near(got, f * f64(ref), tol)


def backward_bounds(args, y_error, before, gates, dy, dh, ends):
    """The bounds of dv, da, dh0 and of the terms of dalpha's sum."""
    V, A, AL, BE = args
    s, sg, f, i, z = gates
    i = np.abs(i)
    B, T, D = V.shape
    eC, mC = np.zeros((B, D)), np.abs(dh)
    eV, eA, eL = np.zeros_like(V), np.zeros_like(V), np.zeros_like(V)
    for t in range(T - 1, -1, -1):
        live = (t < ends)[:, None]
        r = mC + np.where(live, np.abs(dy[:, t]), 0.0)
        eR = eC + 2 * U * r
        eV[:, t] = i[:, t] * eR + U * (26 + z[:, t]) * i[:, t] * r
        C = f[:, t] * r
        eC = np.where(live, f[:, t] * eR + U * ((24 + z[:, t]) * i[:, t] * r + 8 * C), eC)
        mC = np.where(live, C, mC)
        span = np.abs(before[:, t] - V[:, t])
        eG = eC * span + C * (y_error[:, t] + 3 * U * (np.abs(before[:, t]) + np.abs(V[:, t])))
        eA[:, t] = live * np.abs(AL) * sg[:, t] * (eG + U * (20 + z[:, t]) * C * span)
        eL[:, t] = live * s[:, t] * (eG + U * (24 + z[:, t]) * C * span)
    return eV, eA, eL, eC


def test_far_gates_backward():
    """alpha = 0, gates that are 0 or 1, a constant gate next to 1, growing states (alpha < 0): the inputs of test_far_gates."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    v, a, alpha, beta, h0 = made(2, 700, 64, "fp32", 11)
    alpha[:8] = 0.0
    a[..., 8:16] = 1e6   # f = 0
    a[..., 16:24] = -80  # f = 1 to the last bit
    a[..., 24:32] = 0.0  # a constant gate
    beta[24:32] = -9.0
    alpha[32:40] = -1e-3
    y, _ = m2.m2rnn_gated_scan_fwd(v, a, alpha, beta, h0)
    dy, dh = torch.randn_like(y), torch.randn_like(h0)
    got = m2.m2rnn_gated_scan_bwd(v, a, alpha, beta, y, dy, h0, dh)
    _, _, before, gates, E, Eb, _, ends = terms(v, a, alpha, beta, h0, None)
    args = [f64(x) for x in (v, a, alpha, beta)]
    ref, dl, _ = layer.gated_bwd(*args, f64(dy), f64(dh), f64(h0))
    # the error of the states where they grow: terms() takes 1 - f as it is, which is negative there
    Eb[..., 32:40] = np.abs(Eb[..., 32:40]) + 64 * U * 700 * np.abs(before[..., 32:40]).max()
    eV, eA, eL, eC = backward_bounds(args, Eb, before, gates, f64(dy), f64(dh), ends)
    # Where alpha < 0, 1 - f is one minus f as it is rounded (f > 1 is an exponential of one ulp, 2 u, whose argument is rounded twice,
    # 2 |x| u with |x| = |log f| below 0.01): 4 u f, which dv has times R.  R is at most R's bound over the memory of all later steps.
    R = np.abs(f64(dh))[:, 32:40]
    for t in range(699, -1, -1):
        r = R + np.abs(f64(dy)[:, t, 32:40])
        eV[:, t, 32:40] += 4 * U * gates[2][:, t, 32:40] * r
        R = gates[2][:, t, 32:40] * r
    near(got["dv"], ref["dv"], eV)
    near(got["da"], ref["da"], eA)
    near(got["dh0"], ref["dh0"], eC)
    near(got["dalpha"], ref["dalpha"], eL.sum((0, 1)) + 20 * U * np.abs(dl).sum((0, 1)) + 2 * U * np.abs(ref["dalpha"]))
    near(got["dbeta"], ref["dbeta"], eA.sum((0, 1)) + 20 * U * np.abs(ref["da"]).sum((0, 1)) + 2 * U * np.abs(ref["dbeta"]))
    assert not got["dv"][..., :8].any() and not got["da"][..., :8].any() and not got["dbeta"][:8].any()
    assert not got["da"][..., 8:16].any() and torch.equal(got["dv"][..., 8:16], dy[..., 8:16] + torch.cat(
        [torch.zeros_like(dy[:, 1:, 8:16]), dh[:, None, 8:16]], 1))
    assert bool(got["da"][..., 16:24].abs().max() < 1e-30) and bool(got["da"][..., 16:24].any())


@pytest.mark.parametrize("mask", [float("-inf"), -3.3895313892515355e38])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masked_single_steps(mask, dtype):
    """A token whose gate is masked leaves its state as it is, whatever v holds."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    v, a, alpha, beta, h = made(6, 1, 68, dtype, 13)
    v, a = v[:, 0].contiguous(), a[:, 0].contiguous()
    whole = m2.m2rnn_gated_scan_step(v, a, alpha, beta, h)
    for b, x in ((0, float("nan")), (2, float("inf")), (5, float("-inf"))):
        a[b] = mask
        v[b] = x
    out = m2.m2rnn_gated_scan_step(v, a, alpha, beta, h)
    for b in range(6):
        assert torch.equal(out[b], h[b] if b in (0, 2, 5) else whole[b])
    none = m2.m2rnn_gated_scan_step(v, a, alpha, beta)
    assert not none[[0, 2, 5]].any() and bool(torch.isfinite(none).all())
    alpha[3] = 0.0
    v[1, 3] = float("nan")
    assert torch.equal(m2.m2rnn_gated_scan_step(v, a, alpha, beta, h)[1, 3], h[1, 3])
