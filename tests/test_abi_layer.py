"""The C ABI of the layer's entry, the gated recurrence and the orthogonalised update on the CPU: invalid calls are
rejected with the documented status before anything is enqueued, and empty ones do nothing."""
import ctypes

import pytest

import matrix_state_nonlinear_m2rnn_amd as m2

OK, EINVAL, EUNS, EWS = m2.M2RNN_OK, m2.M2RNN_EINVAL, m2.M2RNN_EUNSUPPORTED, m2.M2RNN_EWORKSPACE
MB = 1 << 20


def p(x):
    return ctypes.c_void_p(x) if x else None


def norm(rows=4, D=64, xt=1, x=MB, rt=0, res=2 * MB, gamma=3 * MB, eps=1e-6, h=4 * MB, ot=1, group=0, out=5 * MB, scale=0):
    return m2.lib().m2rnn_add_norm_fwd(rows, D, xt, p(x), rt, p(res), p(gamma), eps, p(h), ot, group, p(out), p(scale), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(D=0), EINVAL), (dict(D=6), EUNS), (dict(D=16388), EUNS), (dict(rows=1 << 31), EUNS),
    (dict(xt=2), EINVAL), (dict(rt=2), EINVAL), (dict(ot=3), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(x=0), EINVAL), (dict(gamma=0), EINVAL), (dict(out=0), EINVAL), (dict(res=0), EINVAL),  # h without a residual
    (dict(ot=2), EINVAL),  # no scale
    (dict(ot=1, group=64), EINVAL), (dict(ot=2, group=64, D=128, scale=6 * MB), EUNS), (dict(ot=2, group=128, scale=6 * MB), EUNS),
    (dict(x=MB + 8), EINVAL), (dict(scale=6 * MB + 2, ot=2), EINVAL),
    (dict(h=2 * MB + 16), EINVAL), (dict(h=MB), EINVAL),  # x has another type than the stream
    (dict(out=MB), EINVAL), (dict(out=4 * MB + 1008), EINVAL), (dict(out=3 * MB), EINVAL),
    (dict(ot=2, scale=5 * MB), EINVAL), (dict(ot=2, scale=4 * MB), EINVAL),
    (dict(rows=0), OK), (dict(rows=0, x=0, out=0, res=0, h=0), OK)])
def test_add_norm_fwd_arguments(kw, status):
    assert norm(**kw) == status


def norm_bwd(rows=4, D=64, ht=0, h=MB, gamma=2 * MB, eps=1e-6, dout=3 * MB, dh=4 * MB, dx=5 * MB, dg=6 * MB, ws=7 * MB, n=MB):
    return m2.lib().m2rnn_add_norm_bwd(rows, D, ht, p(h), p(gamma), eps, p(dout), p(dh), p(dx), p(dg), p(ws), n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), EINVAL), (dict(D=10), EUNS), (dict(ht=2), EINVAL), (dict(eps=-1.0), EINVAL), (dict(h=0), EINVAL),
    (dict(gamma=0), EINVAL), (dict(dout=0), EINVAL), (dict(dx=0), EINVAL), (dict(dg=0), EINVAL), (dict(dh=4 * MB + 4), EINVAL),
    (dict(dx=MB), EINVAL), (dict(dx=3 * MB + 16), EINVAL), (dict(dg=MB + 16), EINVAL), (dict(dg=5 * MB), EINVAL),
    (dict(ws=0), EWS), (dict(n=16), EWS), (dict(ws=7 * MB + 4), EWS)])
def test_add_norm_bwd_arguments(kw, status):
    assert norm_bwd(**kw) == status


def gated(B=2, T=70, D=64, dt=0, v=MB, a=2 * MB, alpha=3 * MB, beta=4 * MB, lens=0, h0=5 * MB, y=6 * MB, hT=7 * MB, ws=8 * MB, n=MB):
    return m2.lib().m2rnn_gated_scan_fwd(B, T, D, dt, p(v), p(a), p(alpha), p(beta), p(lens), p(h0), p(y), p(hT), p(ws), n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), EINVAL), (dict(T=-1), EINVAL), (dict(D=0), EINVAL), (dict(D=6), EUNS), (dict(D=(1 << 24) + 4), EUNS),
    (dict(T=(1 << 31) + 1), EUNS), (dict(B=1 << 30), EUNS), (dict(B=1, T=1 << 31, D=1024), EUNS), (dict(dt=2), EINVAL),
    (dict(v=0), EINVAL), (dict(a=0), EINVAL), (dict(alpha=0), EINVAL), (dict(beta=0), EINVAL), (dict(y=0), EINVAL),
    (dict(v=MB + 8), EINVAL), (dict(lens=9 * MB + 2), EINVAL), (dict(y=MB), EINVAL), (dict(hT=5 * MB), EINVAL),
    (dict(hT=6 * MB + 64), EINVAL), (dict(ws=0), EWS), (dict(n=64), EWS), (dict(B=0), OK)])
def test_gated_scan_fwd_arguments(kw, status):
    assert gated(**kw) == status


def gated_bwd(B=2, T=70, D=64, dt=0, v=MB, a=2 * MB, alpha=3 * MB, beta=4 * MB, lens=0, h0=5 * MB, y=6 * MB, dy=7 * MB,
              dhT=8 * MB, dv=9 * MB, da=10 * MB, dal=11 * MB, dbe=12 * MB, dh0=13 * MB, ws=14 * MB, n=MB):
    return m2.lib().m2rnn_gated_scan_bwd(B, T, D, dt, *map(p, (v, a, alpha, beta, lens, h0, y, dy, dhT, dv, da, dal, dbe, dh0,
                                                               ws)), n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), EINVAL), (dict(D=6), EUNS), (dict(dt=2), EINVAL), (dict(v=0), EINVAL), (dict(y=0), EINVAL), (dict(dy=0), EINVAL),
    (dict(dv=0), EINVAL), (dict(da=0), EINVAL), (dict(dal=0), EINVAL), (dict(dbe=0), EINVAL), (dict(dy=7 * MB + 4), EINVAL),
    (dict(dv=7 * MB), EINVAL), (dict(da=9 * MB + 16), EINVAL), (dict(dbe=11 * MB), EINVAL), (dict(dh0=5 * MB), EINVAL),
    (dict(ws=0), EWS), (dict(n=64), EWS)])
def test_gated_scan_bwd_arguments(kw, status):
    assert gated_bwd(**kw) == status


def test_gated_scan_step_arguments():
    def step(B=2, D=64, dt=0, v=MB, a=2 * MB, alpha=3 * MB, beta=4 * MB, h=5 * MB, out=6 * MB):
        return m2.lib().m2rnn_gated_scan_step(B, D, dt, p(v), p(a), p(alpha), p(beta), p(h), p(out), None)
    assert step(D=6) == EUNS and step(dt=2) == EINVAL and step(v=0) == EINVAL and step(out=0) == EINVAL
    assert step(out=MB) == EINVAL and step(out=5 * MB + 16) == EINVAL and step(h=5 * MB + 4) == EINVAL
    assert step(B=0) == OK


def orth(batch=2, m=64, n=64, dt=0, g=MB, steps=5, coefs=True, eps=1e-7, out=2 * MB, ws=16 * MB, bytes_=64 * MB):
    c = (ctypes.c_float * 15)() if coefs else None
    return m2.lib().m2rnn_orthogonalize(batch, m, n, dt, p(g), steps, c, eps, p(out), p(ws), bytes_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), EINVAL), (dict(m=-1), EINVAL), (dict(dt=2), EINVAL), (dict(steps=0), EINVAL), (dict(steps=65), EUNS),
    (dict(coefs=False), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(m=65537), EUNS),
    (dict(batch=65536), EUNS), (dict(batch=1000, m=16384, n=16384), EUNS), (dict(g=0), EINVAL), (dict(out=0), EINVAL),
    (dict(g=MB + 4), EINVAL), (dict(out=MB + 64), EINVAL), (dict(ws=0, m=300), EWS), (dict(bytes_=64, m=300), EWS), (dict(ws=16 * MB + 4, m=300), EWS),
    (dict(batch=0), OK), (dict(n=0), OK)])
def test_orthogonalize_arguments(kw, status):
    assert orth(**kw) == status


def test_workspace_queries():
    L, n = m2.lib(), ctypes.c_size_t(0)
    assert L.m2rnn_add_norm_bwd_workspace_size(4, 64, None) == EINVAL
    assert L.m2rnn_add_norm_bwd_workspace_size(4, 6, ctypes.byref(n)) == EUNS
    assert L.m2rnn_gated_scan_fwd_workspace_size(2, 70, 64, 7, ctypes.byref(n)) == EINVAL
    assert L.m2rnn_gated_scan_bwd_workspace_size(2, 70, 64, 0, None) == EINVAL
    assert L.m2rnn_gated_scan_bwd_workspace_size(0, 70, 64, 0, ctypes.byref(n)) == OK
    assert L.m2rnn_orthogonalize_workspace_size(3, 0, 5, 0, ctypes.byref(n)) == OK and n.value == 0


def test_binding_refuses_before_the_device():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        m2.m2rnn_add_norm_fwd(x, torch.ones(8))  # not on a GPU
    with pytest.raises(ValueError):
        m2.m2rnn_add_norm_fwd(x, torch.ones(4))
    with pytest.raises(ValueError):
        m2.m2rnn_gated_scan_fwd(x, x, torch.ones(8), torch.ones(8))
    with pytest.raises(ValueError):
        m2.m2rnn_orthogonalize(torch.zeros(8))
