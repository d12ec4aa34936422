"""Refusals of the q/k norm with rotation, the gradient norm and clipping, and the conv window's entry
points: every invalid call returns its documented status before anything is enqueued."""
import ctypes

import matrix_state_nonlinear_m2rnn_amd as m2

P = ctypes.c_void_p
F = ctypes.c_float


def qk(B=1, T=2, Nq=2, Nk=1, K=64, R=64, dtype=0, eps=1e-6, bwd=False, bad=None, nbytes=1 << 40):
    n = ("q", "k", "gq", "gk", "pos", "freq")
    a = {x: P(256) for x in n + ("q_out", "k_out", "dqo", "dko", "dq", "dk", "dgq", "dgk", "ws")}
    a.update(bad or {})
    head = [B, T, Nq, Nk, K, R, 0, dtype] + [a[x] for x in n] + [F(eps)]
    if bwd:
        return m2.lib().m2rnn_qk_norm_rope_bwd(*head, *[a[x] for x in ("dqo", "dko", "dq", "dk", "dgq", "dgk", "ws")],
                                               nbytes, None)
    return m2.lib().m2rnn_qk_norm_rope_fwd(*head, a["q_out"], a["k_out"], None)


def test_qk_norm_rope():
    for bwd in (False, True):
        assert qk(B=-1, bwd=bwd) == m2.M2RNN_EINVAL
        assert qk(dtype=4, bwd=bwd) == m2.M2RNN_EINVAL
        assert qk(R=72, bwd=bwd) == m2.M2RNN_EINVAL                   # more than the head
        assert qk(eps=-1.0, bwd=bwd) == m2.M2RNN_EINVAL
        assert qk(eps=float("nan"), bwd=bwd) == m2.M2RNN_EINVAL
        assert qk(K=24, R=8, bwd=bwd) == m2.M2RNN_EUNSUPPORTED
        assert qk(K=272, bwd=bwd) == m2.M2RNN_EUNSUPPORTED
        assert qk(R=12, bwd=bwd) == m2.M2RNN_EUNSUPPORTED
        for x in ("q", "k", "gq", "gk", "pos", "freq"):
            assert qk(bad={x: None}, bwd=bwd) == m2.M2RNN_EINVAL, x
            assert qk(bad={x: P(258)}, bwd=bwd) == m2.M2RNN_EINVAL, x
    assert qk(bad={"q_out": None}) == m2.M2RNN_EINVAL
    assert qk(bad={"dgk": None}, bwd=True) == m2.M2RNN_EINVAL
    assert qk(bad={"ws": None}, bwd=True) == m2.M2RNN_EWORKSPACE
    n = ctypes.c_size_t(0)
    assert m2.lib().m2rnn_qk_norm_rope_bwd_workspace_size(1, 2, 2, 1, 64, ctypes.byref(n)) == 0
    assert n.value >= 2 * 64 * 4 and qk(bwd=True, nbytes=n.value - 1) == m2.M2RNN_EWORKSPACE
    assert qk(B=0, bad={"q": None}) == m2.M2RNN_OK


class Tensor(ctypes.Structure):
    _fields_ = [("data", P), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int64)]


def tensors(*specs):
    return (Tensor * len(specs))(*[Tensor(*s) for s in specs])


def test_grad_lists():
    L = m2.lib()
    n = ctypes.c_size_t(0)
    ok = tensors((4096, 1000, 0), (1 << 20, 5, 1))
    assert L.m2rnn_grad_norm_workspace_size(ok, 2, ctypes.byref(n)) == 0 and n.value == 16
    assert L.m2rnn_grad_norm_workspace_size(ok, 2, None) == m2.M2RNN_EINVAL
    norm, ws = P(256), P(512)
    for bad in (tensors((4096, -1, 0)), tensors((4096, 5, 3)), tensors((None, 5, 0)), tensors((4098, 5, 0)),
                tensors((4097, 5, 1))):
        assert L.m2rnn_grad_norm(bad, 1, norm, ws, 1 << 20, None) == m2.M2RNN_EINVAL
        assert L.m2rnn_grad_clip(bad, 1, None, norm, F(1.0), None) == m2.M2RNN_EINVAL
    assert L.m2rnn_grad_norm(ok, -1, norm, ws, 16, None) == m2.M2RNN_EINVAL
    assert L.m2rnn_grad_norm(None, 1, norm, ws, 16, None) == m2.M2RNN_EINVAL
    assert L.m2rnn_grad_norm(ok, 2, None, ws, 16, None) == m2.M2RNN_EINVAL
    assert L.m2rnn_grad_norm(ok, 2, norm, ws, 15, None) == m2.M2RNN_EWORKSPACE
    assert L.m2rnn_grad_norm(ok, 2, norm, None, 16, None) == m2.M2RNN_EWORKSPACE
    for m in (-1.0, float("nan")):
        assert L.m2rnn_grad_clip(ok, 2, None, norm, F(m), None) == m2.M2RNN_EINVAL
    assert L.m2rnn_grad_clip(ok, 2, None, None, F(1.0), None) == m2.M2RNN_EINVAL
    # memory written twice, or written while another tensor is read from it
    twice = tensors((4096, 1000, 0), (4096, 1000, 0))
    assert L.m2rnn_grad_clip(twice, 2, None, norm, F(1.0), None) == m2.M2RNN_EINVAL
    part = tensors((4096, 1000, 0), (8092, 10, 0))
    assert L.m2rnn_grad_clip(part, 2, None, norm, F(1.0), None) == m2.M2RNN_EINVAL
    # the norm within what is scaled
    assert L.m2rnn_grad_clip(ok, 2, None, P(4096 + 8), F(1.0), None) == m2.M2RNN_EINVAL
    assert L.m2rnn_grad_clip(ok, 2, None, P((1 << 20) + 8), F(1.0), None) == m2.M2RNN_EINVAL
    outs = lambda *a: (P * len(a))(*a)  # noqa: E731
    assert L.m2rnn_grad_clip(ok, 2, outs(1 << 21, (1 << 21) + 3996), norm, F(1.0), None) == m2.M2RNN_EINVAL
    assert L.m2rnn_grad_clip(ok, 2, outs(1 << 20, 1 << 22), norm, F(1.0), None) == m2.M2RNN_EINVAL  # onto the other
    assert L.m2rnn_grad_clip(ok, 2, outs(4100, 1 << 22), norm, F(1.0), None) == m2.M2RNN_EINVAL     # onto itself, shifted
    assert L.m2rnn_grad_clip(ok, 2, outs(4098 + (1 << 22), 1 << 23), norm, F(1.0), None) == m2.M2RNN_EINVAL  # alignment
    assert L.m2rnn_grad_clip(ok, 0, None, norm, F(1.0), None) == m2.M2RNN_OK


def test_norm_within_the_gradients():
    L = m2.lib()
    ok = tensors((4096, 1000, 0), (1 << 20, 6, 1), (None, 0, 0))
    for at in (4096, 4096 + 3996, 1 << 20, (1 << 20) + 8):
        assert L.m2rnn_grad_norm(ok, 3, P(at), P(512), 1 << 20, None) == m2.M2RNN_EINVAL, at


def test_conv_window():
    L = m2.lib()
    p, q = P(1 << 12), P(1 << 20)

    def state(B=1, T=8, C=8, dtype=0, x=p, w=p, lens=None, win=p, u=p, wo=q):
        return L.m2rnn_conv4_silu_fwd_state(B, T, C, dtype, x, w, None, lens, win, u, wo, None)

    def step(B=1, C=8, dtype=0, x=p, w=p, win=p, u=p, wo=q):
        return L.m2rnn_conv4_silu_step(B, C, dtype, x, w, None, win, u, wo, None)
    for f in (state, step):
        assert f(B=-1) == m2.M2RNN_EINVAL
        assert f(C=6) == m2.M2RNN_EUNSUPPORTED
        assert f(dtype=3) == m2.M2RNN_EINVAL
        assert f(x=None) == m2.M2RNN_EINVAL
        assert f(w=None) == m2.M2RNN_EINVAL
        assert f(u=None) == m2.M2RNN_EINVAL
        assert f(wo=None) == m2.M2RNN_EINVAL
        assert f(x=P(20)) == m2.M2RNN_EINVAL
        assert f(win=P(1 << 20), wo=P((1 << 20) + 32)) == m2.M2RNN_EINVAL
        assert f(B=0) == m2.M2RNN_OK
    assert state(win=q, wo=q) == m2.M2RNN_EINVAL
    assert state(lens=P(258)) == m2.M2RNN_EINVAL


def test_conv_sizes_that_no_launch_holds():
    """Steps are numbered with ints, up to two chunks past the last one, and a launch holds fewer than 2^32 threads."""
    L = m2.lib()
    p, q = P(1 << 12), P(1 << 20)
    calls = {
        "fwd": lambda B, T, C: L.m2rnn_conv4_silu_fwd(B, T, C, 1, p, p, None, q, None),
        "state": lambda B, T, C: L.m2rnn_conv4_silu_fwd_state(B, T, C, 1, p, p, None, None, None, q, q, None),
        "bwd": lambda B, T, C: L.m2rnn_conv4_silu_bwd(B, T, C, 1, p, p, None, p, q, q, None, p, 1 << 40, None),
        "step": lambda B, T, C: L.m2rnn_conv4_silu_step(B, C, 1, p, p, None, None, q, q, None),
    }
    last = (1 << 31) - 1
    for name in ("fwd", "state", "bwd"):
        for T in (last, last - 63, last - 255):
            assert calls[name](1, T, 4) == m2.M2RNN_EUNSUPPORTED, (name, T)
            assert calls[name](0, T, 4) == m2.M2RNN_EUNSUPPORTED, (name, T)
        assert calls[name](1, 1 << 30, 4096) == m2.M2RNN_EUNSUPPORTED, name  # 2^27 waves or more
    assert calls["step"](1 << 24, 1, 1024) == m2.M2RNN_EUNSUPPORTED         # 2^32 threads
    assert calls["step"](1 << 31, 1, 4) == m2.M2RNN_EUNSUPPORTED
    for name in ("fwd", "state"):
        assert calls[name](0, last - 256, 4) == m2.M2RNN_OK                 # nothing to do, nothing launched
