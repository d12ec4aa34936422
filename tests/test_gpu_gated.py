"""The gated recurrence of channels on the GPU against the fp64 oracle.

Tolerances, u = 2^-24, follow the recurrence.  A gate's exponent x = alpha softplus(a + beta) is off by (24 + |a + beta|) u of
itself (the sum's rounding, softplus, the product), which changes i = 1 - f by at most that share of i; a step's
operations round the state 8 times at most, the joins of 8-step stretches among them.  A join adds P h (from the state
that enters a stretch) and l (from its own inputs), each rounded by itself, and the two may cancel: what rounds is
bounded by m_t = f_t m_{t-1} + i |v|, m_0 = |h_0|, and not by |h_t|.  So the error of h_t is below
    e_t = f_t e_{t-1} + u ((24 + |z|) i (|v| + m_{t-1}) + 8 m_t),
summed below in fp64 beside the oracle, and the reverse recurrence's likewise (m of C: f (m + |dy|)).  Sums over batch and time: their terms'
errors, and 20 u of the terms' magnitudes (16 additions in fp32, the rest in fp64) and the last rounding.
"""
import numpy as np
import pytest

from _gpu import say, torch_cuda
from oracle import layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def made(B, T, D, dtype, seed, h0=True, far=False):
    """far: memories from one step to far beyond the sequence."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    beta = torch.rand(D, device="cuda", generator=g) * (16 if far else 6) - (14 if far else 6)
    return n(B, T, D).to(t), n(B, T, D).to(t), torch.rand(D, device="cuda", generator=g) * 15 + 1, beta, n(B, D) if h0 else None


def terms(v, a, alpha, beta, h0, lens):
    """The oracle's y, h_T, states before each step, gates, and the error bound of y."""
    v, a, alpha, beta, h0 = map(f64, (v, a, alpha, beta, h0))
    lens = None if lens is None else lens.cpu().numpy()
    y, hT, before = layer.gated_fwd(v, a, alpha, beta, h0, lens)
    s, sg, f, i = layer.gate(a, alpha, beta)
    z = np.where(np.isfinite(a), np.abs(a + beta), 0.0)
    e = np.zeros_like(hT)
    m = np.zeros_like(hT) if h0 is None else np.abs(h0)
    E, Eb = np.zeros_like(y), np.zeros_like(y)
    T = y.shape[1]
    n = np.full(y.shape[0], T) if lens is None else np.clip(lens, 0, T)
    for t in range(T):
        Eb[:, t] = e
        on = (t < n)[:, None] & (s[:, t] != 0)
        vv = np.where(on, v[:, t], 0.0)
        m1 = np.where(on, f[:, t] * m + i[:, t] * np.abs(vv), m)
        nxt = f[:, t] * e + U * ((24 + z[:, t]) * i[:, t] * (np.abs(vv) + m) + 8 * m1)
        e = np.where(on, nxt, e + 4 * U * m * (t % 8 == 0))
        m = m1
        E[:, t] = e
    return y, hT, before, (s, sg, f, i, z), E, Eb, e, n


def near(got, ref, tol):
    d = np.abs(f64(got) - ref)
    assert (d <= tol + 1e-38).all(), float((d / (tol + 1e-38)).max())


CASES = [  # B, T, D, dtype, lens, h0, far
    (1, 1, 4, "fp32", None, True, False), (2, 7, 8, "bf16", None, False, False), (3, 8, 100, "fp32", [8, 0, 3], True, False),
    (2, 9, 256, "bf16", None, True, True), (5, 63, 60, "fp32", [63, 1, 62, 0, 200], True, False),
    (2, 64, 260, "bf16", None, False, False), (1, 65, 1100, "fp32", None, True, True), (7, 129, 12, "bf16", None, True, False),
    (2, 200, 516, "bf16", [200, 64], False, True), (1, 513, 64, "fp32", None, True, True),
    (1, 1025, 2048, "bf16", None, False, False), (64, 70, 4, "fp32", None, True, False), (1, 2500, 8, "fp32", [2177], True, True),
    (33, 1, 2048, "bf16", None, True, False)]


@pytest.mark.parametrize("B,T,D,dtype,lens,h0,far", CASES)
def test_forward_and_backward(B, T, D, dtype, lens, h0, far):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("gated", B, T, D, dtype, lens, h0, far)
    args = made(B, T, D, dtype, B + T + D, h0, far)
    v, a, alpha, beta, s0 = args
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    y, hT = m2.m2rnn_gated_scan_fwd(*args, lens=n)
    ry, rh, before, (s, sg, f, i, z), E, Eb, e, ends = terms(*args, n)
    near(y, ry, E)
    near(hT, rh, e)
    for b, k in enumerate(ends):  # the last step's y, bit for bit
        assert torch.equal(hT[b], y[b, int(k) - 1] if k > 0 else hT[b] * 0 if s0 is None else s0[b])
    if lens is not None:
        for b, k in enumerate(ends):
            assert not y[b, int(k):].any()
    dy, dh = torch.randn_like(y), torch.randn(B, D, device="cuda")
    got = m2.m2rnn_gated_scan_bwd(*args[:4], y, dy, s0, dh, lens=n)
    V, A, AL, BE = map(f64, args[:4])
    ref, dl, R = layer.gated_bwd(V, A, AL, BE, f64(dy), f64(dh), f64(s0), None if n is None else n.cpu().numpy())
    eC, mC = np.zeros((B, D)), np.abs(f64(dh))
    eV, eA, eL = np.zeros_like(V), np.zeros_like(V), np.zeros_like(V)
    for t in range(T - 1, -1, -1):
        live = (t < ends)[:, None]
        r = mC + np.where(live, np.abs(f64(dy)[:, t]), 0.0)
        eR = eC + 2 * U * r
        eV[:, t] = i[:, t] * eR + U * (26 + z[:, t]) * i[:, t] * r
        C = f[:, t] * r
        eC = np.where(live, f[:, t] * eR + U * ((24 + z[:, t]) * i[:, t] * r + 8 * C), eC)
        mC = np.where(live, C, mC)
        span = np.abs(before[:, t] - V[:, t])
        eG = eC * span + C * (Eb[:, t] + 3 * U * (np.abs(before[:, t]) + np.abs(V[:, t])))
        eA[:, t] = live * np.abs(AL) * sg[:, t] * (eG + U * (20 + z[:, t]) * C * span)
        eL[:, t] = live * s[:, t] * (eG + U * (24 + z[:, t]) * C * span)
    live = (np.arange(T)[None, :] < ends[:, None])[..., None]
    near(got["dv"], ref["dv"], eV * live)
    near(got["da"], ref["da"], eA)
    near(got["dh0"], ref["dh0"], eC)
    near(got["dalpha"], ref["dalpha"], eL.sum((0, 1)) + 20 * U * np.abs(dl).sum((0, 1)) + 2 * U * np.abs(ref["dalpha"]))
    near(got["dbeta"], ref["dbeta"], eA.sum((0, 1)) + 20 * U * np.abs(ref["da"]).sum((0, 1)) + 2 * U * np.abs(ref["dbeta"]))
    # the same bits again, from dirty workspaces
    size = lambda q: torch.full((m2._size_query(q, B, T, D, m2._dtype_code(v)) + 16,), 255, dtype=torch.uint8, device="cuda")  # noqa: E731
    y2, h2 = m2.m2rnn_gated_scan_fwd(*args, lens=n, workspace=size("m2rnn_gated_scan_fwd_workspace_size"))
    g2 = m2.m2rnn_gated_scan_bwd(*args[:4], y, dy, s0, dh, lens=n, workspace=size("m2rnn_gated_scan_bwd_workspace_size"))
    assert torch.equal(y, y2) and torch.equal(hT, h2) and all(torch.equal(got[x], g2[x]) for x in got)
    # without the states' gradients
    g3 = m2.m2rnn_gated_scan_bwd(*args[:4], y, dy, s0, lens=n, want_dh0=False)
    assert g3["dh0"] is None
    ref3 = layer.gated_bwd(V, A, AL, BE, f64(dy), None, f64(s0), None if n is None else n.cpu().numpy())[0]
    near(g3["dv"], ref3["dv"], 2 * eV * live + 64 * U * np.abs(ref3["dv"]))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_steps_follow_the_scan(dtype):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    args = made(3, 20, 68, dtype, 5)
    y, hT = m2.m2rnn_gated_scan_fwd(*args)
    E = terms(*args, None)[4]
    h = args[4].clone()
    for t in range(20):
        out = m2.m2rnn_gated_scan_step(args[0][:, t].contiguous(), args[1][:, t].contiguous(), args[2], args[3], h, h_out=h)
        assert out is h
        near(h, f64(y[:, t]), 2 * E[:, t])
    first = m2.m2rnn_gated_scan_step(args[0][:, 0].contiguous(), args[1][:, 0].contiguous(), args[2], args[3])
    near(first, layer.gated_fwd(f64(args[0][:, :1]), f64(args[1][:, :1]), f64(args[2]), f64(args[3]))[0][:, 0],
         64 * U * np.abs(f64(args[0][:, 0])))


@pytest.mark.parametrize("mask", [float("-inf"), -3.3895313892515355e38])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_masked_steps_and_padding(mask, dtype):
    """Masked steps hold the state and padding is not looked at, whatever they hold; backward too."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    B, T, D = 3, 150, 72
    v, a, alpha, beta, h0 = made(B, T, D, dtype, 8)
    lens = torch.tensor([150, 77, 0], dtype=torch.int32, device="cuda")
    masked = torch.rand(B, T, device="cuda") < 0.3
    masked[0, 64:128] = True  # a whole chunk
    a[masked] = mask
    clean = v.clone()
    clean[masked] = 0.0
    junk = v.clone()
    junk[masked] = float("nan")
    ajunk = a.clone()
    for b, n in enumerate(lens.tolist()):
        junk[b, n:] = float("inf")
        ajunk[b, n:] = float("nan")
    y, hT = m2.m2rnn_gated_scan_fwd(junk, ajunk, alpha, beta, h0, lens=lens)
    args = (clean, a, alpha, beta, h0)
    ry, rh, _, _, E, _, e, _ = terms(*args, lens)
    near(y, ry, E)
    near(hT, rh, e)
    y0, h0_ = m2.m2rnn_gated_scan_fwd(*args, lens=lens)
    assert torch.equal(y, y0) and torch.equal(hT, h0_) and torch.equal(hT[2], h0[2])
    dy = torch.randn_like(y)
    dj = dy.clone()
    for b, n in enumerate(lens.tolist()):
        dj[b, n:] = float("nan")
    g = m2.m2rnn_gated_scan_bwd(clean, a, alpha, beta, y, dy, h0, lens=lens)
    gj = m2.m2rnn_gated_scan_bwd(junk, ajunk, alpha, beta, y, dj, h0, lens=lens)
    for x in g:
        assert torch.equal(g[x], gj[x]) and bool(torch.isfinite(g[x]).all()), x
    assert not g["dv"][masked].any() and not g["da"][masked].any()


def test_values_that_are_not_finite_stay_in_their_channel():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    v, a, alpha, beta, h0 = made(2, 300, 264, "fp32", 9)
    y, hT = m2.m2rnn_gated_scan_fwd(v, a, alpha, beta, h0)
    for what, value in ((v, float("nan")), (v, float("inf")), (a, float("nan"))):
        x = what.clone()
        x[1, 137, 5] = value
        args = (x, a) if what is v else (v, x)
        yb, hb = m2.m2rnn_gated_scan_fwd(*args, alpha, beta, h0)
        same = torch.ones_like(y, dtype=torch.bool)
        same[1, 137:, 5] = False
        assert torch.equal(yb[same], y[same]) and not torch.isfinite(yb[1, 137:, 5]).any()
        keep = torch.ones_like(hT, dtype=torch.bool)
        keep[1, 5] = False
        assert torch.equal(hb[keep], hT[keep]) and not torch.isfinite(hb[1, 5])


def test_far_gates():
    """alpha = 0, gates that are 0 or 1, a constant gate next to 1 over a long sequence, growing states (alpha < 0)."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    v, a, alpha, beta, h0 = made(2, 700, 64, "fp32", 11)
    alpha[:8] = 0.0
    a[..., 8:16] = 1e6   # f = 0
    a[..., 16:24] = -80  # f = 1 to the last bit
    a[..., 24:32] = 0.0  # a constant gate
    beta[24:32] = -9.0
    alpha[32:40] = -1e-3
    args = (v, a, alpha, beta, h0)
    y, hT = m2.m2rnn_gated_scan_fwd(*args)
    ry, rh, _, _, E, _, e, _ = terms(*args, None)
    grow = np.zeros(64, dtype=bool)
    grow[32:40] = True
    near(y[..., ~torch.tensor(grow, device="cuda")], ry[..., ~grow], E[..., ~grow])
    d = np.abs(f64(y) - ry)[..., grow]
    assert (d <= 1e-4 * np.abs(ry)[..., grow].max()).all()
    assert torch.equal(y[..., :8], h0[:, None, :8].expand(-1, 700, -1))
    assert torch.equal(y[..., 8:16], v[..., 8:16])


def test_empty():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    h0 = torch.randn(3, 8, device="cuda")
    y, hT = m2.m2rnn_gated_scan_fwd(z(3, 0, 8), z(3, 0, 8), z(8), z(8), h0)
    assert y.shape == (3, 0, 8) and torch.equal(hT, h0)
    g = m2.m2rnn_gated_scan_bwd(z(3, 0, 8), z(3, 0, 8), z(8), z(8), y, y, h0, h0)
    assert torch.equal(g["dh0"], h0) and not g["dalpha"].any() and not g["dbeta"].any()
    g = m2.m2rnn_gated_scan_bwd(z(0, 5, 8), z(0, 5, 8), z(8), z(8), z(0, 5, 8), z(0, 5, 8))
    assert not g["dalpha"].any() and g["dv"].shape == (0, 5, 8)


def test_refusals():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    v, a, alpha, beta, h0 = made(2, 8, 16, "fp32", 1)
    with pytest.raises(TypeError):
        m2.m2rnn_gated_scan_fwd(v, a.bfloat16(), alpha, beta)
    with pytest.raises(TypeError):
        m2.m2rnn_gated_scan_fwd(v, a, alpha.double(), beta)
    with pytest.raises(ValueError):
        m2.m2rnn_gated_scan_fwd(v.transpose(0, 1), a, alpha, beta)
    with pytest.raises(ValueError):
        m2.m2rnn_gated_scan_fwd(v, a, alpha, beta, h0[:1])
    with pytest.raises(TypeError):
        m2.m2rnn_gated_scan_fwd(v, a, alpha, beta, lens=torch.tensor([8, 8], device="cuda"))
    with pytest.raises(m2.M2RNNError):
        m2.m2rnn_gated_scan_fwd(v, a, alpha, beta, h0, h_T=h0)
    with pytest.raises(m2.M2RNNError):
        m2.m2rnn_gated_scan_fwd(*(x[..., :6].contiguous() for x in (v, a, alpha, beta)))
