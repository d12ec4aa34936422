"""Arrays whose elements are numbered past 2^31 (and launches of more than 2^32 threads, were they not cut):
the end of a large call against the same rows in a call of their own.  Where each row is computed by
itself the two agree bit for bit; the scan over a long sequence is compared within its error bound."""
import pytest

from _gpu import say, torch_cuda

pytestmark = pytest.mark.gpu


def test_scan_of_a_long_sequence():
    import matrix_state_nonlinear_m2rnn_amd as m2
    torch = torch_cuda()
    T, N, K, V, tail = 1 << 17, 128, 16, 128, 300
    say(f"scan T={T} N={N}")
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*s, std=1.0, dtype=torch.float32):
        return torch.empty(s, dtype=dtype, device="cuda").normal_(0, std, generator=g)
    q, k = normal(1, T, 1, K, std=K ** -0.5, dtype=torch.bfloat16), normal(1, T, 1, K, std=K ** -0.5, dtype=torch.bfloat16)
    v, a = normal(1, T, N, V, dtype=torch.bfloat16), normal(1, T, N)
    alpha, beta, w_r = normal(N).abs() + 0.5, normal(N) - 3.0, normal(N, V)
    assert v.numel() >= 1 << 31

    def run(f, part, H0=None):
        x = [f(t[:, part]) for t in (q, k, v)]
        return m2.m2rnn_ssm_fwd(*x, a[:, part], alpha, beta, f(w_r), H0)
    same = lambda t: t  # noqa: E731
    y, H = run(same, slice(0, T))
    y_end, H_end = y[:, -tail:].clone(), H
    del y
    _, H0 = run(same, slice(0, T - tail))
    y1, H1 = run(same, slice(T - tail, T), H0)
    # each side is within ops roundings of the sum of its terms' absolute values, ops as in the scan's own tests
    _, A0 = run(torch.abs, slice(0, T - tail))
    ya, Ha = run(torch.abs, slice(T - tail, T), A0)
    ops = K + V + 64 + 4 * (T // 64) + 96
    for x, x1, xa in ((y_end, y1, ya), (H_end, H1, Ha)):
        assert torch.isfinite(x).all()
        assert bool(((x - x1).abs() <= 2 * ops * 2.0 ** -24 * xa + 1e-30).all())


def test_scan_backward_of_many_states():
    import matrix_state_nonlinear_m2rnn_amd as m2
    torch = torch_cuda()
    B, N, K, V = 1 << 13, 32, 128, 128
    say(f"scan backward B={B} N={N} K={K} V={V}")
    g = torch.Generator(device="cuda").manual_seed(2)

    def normal(*s, dtype=torch.float32):
        return torch.empty(s, dtype=dtype, device="cuda").normal_(0, 1, generator=g)
    q, k, v = (normal(B, 1, N, d, dtype=torch.bfloat16) for d in (K, K, V))
    a, alpha, beta, w_r = normal(B, 1, N), normal(N).abs(), normal(N), normal(N, V)
    ckpt, dy = normal(B, N, 1, K, V), normal(B, 1, N, V)
    assert ckpt.numel() >= 1 << 32
    out = m2.m2rnn_ssm_bwd(q, k, v, a, alpha, beta, w_r, ckpt, dy)
    e = slice(B - 2, B)
    end = m2.m2rnn_ssm_bwd(q[e], k[e], v[e], a[e], alpha, beta, w_r, ckpt[e], dy[e])
    for n in ("dq", "dk", "dv", "da", "dH0"):
        assert torch.equal(out[n][e], end[n]), n
    assert all(torch.isfinite(out[n]).all() for n in ("dalpha", "dbeta", "dw_r"))


def test_scan_step_of_many_states():
    import matrix_state_nonlinear_m2rnn_amd as m2
    torch = torch_cuda()
    B, N, K, V = 1 << 12, 32, 128, 128
    say(f"scan step B={B} N={N} K={K} V={V}")
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*s):
        return torch.empty(s, device="cuda").normal_(0, 1, generator=g)
    q, k, v, a = normal(B, N, K), normal(B, N, K), normal(B, N, V), normal(B, N)
    alpha, beta, w_r, H = normal(N).abs(), normal(N), normal(N, V), normal(B, N, K, V)
    assert H.numel() >= 1 << 31
    y, H1 = m2.m2rnn_ssm_step(q, k, v, a, alpha, beta, w_r, H)
    e = slice(B - 3, B)
    y_end, H_end = m2.m2rnn_ssm_step(q[e], k[e], v[e], a[e], alpha, beta, w_r, H[e])
    assert torch.equal(y[e], y_end) and torch.equal(H1[e], H_end)


def test_qk_norm_rope_of_many_tokens():
    import matrix_state_nonlinear_m2rnn_amd as m2
    torch = torch_cuda()
    T, Nq, Nk, K = (1 << 26) + 5, 2, 1, 16
    say(f"q/k norm T={T}")
    g = torch.Generator(device="cuda").manual_seed(4)

    def normal(*s, dtype=torch.bfloat16):
        return torch.empty(s, dtype=dtype, device="cuda").normal_(0, 1, generator=g)
    q, k, gq, gk = normal(1, T, Nq, K), normal(1, T, Nk, K), normal(K, dtype=torch.float32), normal(K, dtype=torch.float32)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    freq = torch.tensor([1e4 ** (-i / 8) for i in range(8)], dtype=torch.float64, device="cuda")
    assert q.numel() > 1 << 31
    qo, ko = m2.m2rnn_qk_norm_rope_fwd(q, k, gq, gk, pos, freq)
    e = slice(T - 70, T)
    qe, ke = m2.m2rnn_qk_norm_rope_fwd(q[:, e], k[:, e], gq, gk, pos[:, e].clone(), freq)
    assert torch.equal(qo[:, e], qe) and torch.equal(ko[:, e], ke)
    dqo, dko = qo.float(), ko.float()
    del qo, ko
    out = m2.m2rnn_qk_norm_rope_bwd(q, k, gq, gk, pos, freq, dqo, dko)
    end = m2.m2rnn_qk_norm_rope_bwd(q[:, e], k[:, e], gq, gk, pos[:, e].clone(), freq, dqo[:, e], dko[:, e])
    assert torch.equal(out["dq"][:, e], end["dq"]) and torch.equal(out["dk"][:, e], end["dk"])


def test_conv_window_of_a_long_prompt():
    import matrix_state_nonlinear_m2rnn_amd as m2
    torch = torch_cuda()
    T, C = (1 << 20) + 7, 2052
    say(f"conv T={T} C={C}")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    w = torch.empty(C, 4, device="cuda").normal_(0, 1, generator=g)
    assert x.numel() > 1 << 31
    u, win = m2.m2rnn_conv4_silu_fwd_state(x, w)
    assert torch.equal(win, x[:, -3:])
    ue, wine = m2.m2rnn_conv4_silu_fwd_state(x[:, -90:], w, win=x[:, -93:-90].clone())
    assert torch.equal(u[:, -90:], ue) and torch.equal(win, wine)


def test_clip_of_one_large_tensor():
    import matrix_state_nonlinear_m2rnn_amd as m2
    torch = torch_cuda()
    n = (1 << 31) + 12345
    say(f"clip n={n}")
    t = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    norm = m2.m2rnn_grad_clip([t], 1.0)
    assert float(norm) == float(torch.tensor(float(n), dtype=torch.float64).sqrt().float())
    want = float((1.0 / norm.double()).float().to(torch.bfloat16))
    assert float(t.min()) == want and float(t.max()) == want
