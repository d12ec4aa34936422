"""The residual's addition with the RMSNorm on the GPU against the fp64 oracle.

Tolerances, u = 2^-24.  h is one fp32 addition, rounded to the stream's type: u (and half a bf16 step, 2^-8) of |res + x|.
The other outputs are compared with the formula of the kernel's own h.  The squares' sum has 64 terms in a lane and at
most 8 levels above, so 1/rms is off by 36 u of the sum and 6 u of its own operations, and an output by 48 u (two
products more), plus half a bf16 step where it is stored so.  e4m3: the scale 52 u; out times scale is off by half a step,
2^-4 of the value, or 2^-10 of the scale below the smallest normal number, and 2^-18 of the value for ties that fall
the other way.  Backward: dx = r p - m (r h) + dh; r p 48 u, dh 2 u, and m from a sum of products whose error is at most
80 u of the sum of their magnitudes, plus 90 u of the term itself.  dgamma: up to 64 terms in a lane and 64 lanes, 180 u of the
sum of the magnitudes, and its last rounding.
"""
import numpy as np
import pytest

from _gpu import say, torch_cuda
from oracle import layer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def half(name):
    return {"fp32": 0.0, "bf16": 2.0 ** -8}[name]


def dt(name):
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def f64(t):
    return t.double().cpu().numpy()


def made(rows, D, x, res, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    X = (torch.randn(rows, D, device="cuda", generator=g) * scale).to(dt(x))
    R = None if res == "none" else (torch.randn(rows, D, device="cuda", generator=g) * 3 * scale).to(dt(res))
    return X, R, torch.randn(D, device="cuda", generator=g) * 0.3 + 1


def check_fwd(X, R, gamma, eps, out, group, o, s, h):
    import torch
    x = f64(X)
    if R is None:
        assert h is X
    else:
        ref = f64(R) + x
        e = half("bf16" if R.dtype == torch.bfloat16 else "fp32")
        assert h.dtype == R.dtype and (np.abs(f64(h) - ref) <= (e + 1.01 * U) * np.abs(ref) + 1e-44).all()
    ref = layer.norm_fwd(f64(h), f64(gamma), eps)
    assert o.dtype == dt(out) and o.shape == X.shape
    if out != "e4m3":
        assert s is None
        assert (np.abs(f64(o) - ref) <= (48 * U + 1.001 * half(out)) * np.abs(ref) + 1e-44).all()
        return
    g = group or X.shape[-1]
    parts = ref.reshape(-1, X.shape[-1] // g, g)
    sr = np.maximum(np.abs(parts).max(-1) / 448.0, 2.0 ** -126)
    sk = f64(s).reshape(sr.shape)
    assert (np.abs(sk - sr) <= 52 * U * sr).all()
    got = f64(o.float()).reshape(parts.shape) * sk[..., None]
    assert (np.abs(got - parts) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(parts) + 2.0 ** -10 * sk[..., None] * (1 + 2.0 ** -18)).all()


SHAPES = [(1, 4), (3, 16), (70, 12), (5, 20), (33, 64), (9, 100), (7, 256), (4, 260), (2050, 128), (2100, 512), (2049, 1100),
          (3, 1100), (2053, 2048), (130, 2048), (2051, 4096), (2, 4100), (6, 8192), (3, 16384)]


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("x,res,out", [("bf16", "fp32", "bf16"), ("bf16", "bf16", "e4m3"), ("fp32", "none", "fp32"),
                                       ("fp32", "bf16", "e4m3"), ("bf16", "none", "bf16")])
def test_forward(rows, D, x, res, out):
    torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    for group in ([0, 128] if out == "e4m3" and D % 128 == 0 else [0]):
        say("add_norm", rows, D, x, res, out, group)
        X, R, gamma = made(rows, D, x, res, rows + D)
        check_fwd(X, R, gamma, 1e-6, out, group, *m2.m2rnn_add_norm_fwd(X, gamma, R, 1e-6, out_dtype=dt(out), group=group))


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("h,stream", [("fp32", True), ("bf16", True), ("fp32", False)])
def test_backward(rows, D, h, stream):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("add_norm bwd", rows, D, h, stream)
    H, dout, gamma = made(rows, D, h, "fp32", 7 * rows + D)
    dh = torch.randn_like(dout) if stream else None
    got = m2.m2rnn_add_norm_bwd(H, gamma, dout, dh, 1e-6)
    hh, gg, dd = f64(H), f64(gamma), f64(dout)
    dx, dg = layer.norm_bwd(hh, gg, 1e-6, dd, f64(dh) if stream else None)
    r = 1.0 / np.sqrt((hh * hh).mean(-1, keepdims=True) + 1e-6)
    p = gg * dd
    tol = U * (48 * np.abs(r * p) + 90 * np.abs(r ** 3 * hh * (p * hh).mean(-1, keepdims=True))
               + 80 * r ** 3 * np.abs(hh) * np.abs(p * hh).mean(-1, keepdims=True) + (2 * np.abs(f64(dh)) if stream else 0.0))
    assert (np.abs(f64(got["dx"]) - dx) <= tol + 1e-44).all()
    assert (np.abs(f64(got["dgamma"]) - dg) <= 180 * U * np.abs(dd * hh * r).sum(0) + 2 * U * np.abs(dg)).all()
    again = m2.m2rnn_add_norm_bwd(H, gamma, dout, dh, 1e-6)
    assert torch.equal(again["dx"], got["dx"]) and torch.equal(again["dgamma"], got["dgamma"])
    # in place on either gradient
    out = {"dx": dout.clone(), "dgamma": torch.empty_like(gamma)}
    m2.m2rnn_add_norm_bwd(H, gamma, out["dx"], dh, 1e-6, out=out)
    assert torch.equal(out["dx"], got["dx"])
    if stream:
        out = {"dx": dh.clone(), "dgamma": torch.empty_like(gamma)}
        m2.m2rnn_add_norm_bwd(H, gamma, dout, out["dx"], 1e-6, out=out)
        assert torch.equal(out["dx"], got["dx"])


@pytest.mark.parametrize("D", [64, 1100, 2048, 8192])
def test_stream_in_place_and_leading_axes(D):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    X, R, gamma = made(12, D, "fp32", "fp32", D)
    o, s, h = m2.m2rnn_add_norm_fwd(X.view(3, 4, D), gamma, R.view(3, 4, D), out_dtype=torch.float8_e4m3fn)
    assert o.shape == (3, 4, D) and s.shape == (3, 4, 1)
    S = R.clone()
    o2, _, h2 = m2.m2rnn_add_norm_fwd(X, gamma, S, h=S, out_dtype=torch.float8_e4m3fn)
    assert h2 is S and torch.equal(S, h.view(12, D)) and torch.equal(o2.float(), o.float().view(12, D))
    Y = X.clone()
    m2.m2rnn_add_norm_fwd(Y, gamma, R, h=Y)
    assert torch.equal(Y, S)
    with pytest.raises(m2.M2RNNError):
        m2.m2rnn_add_norm_fwd(X, gamma, R, out=X)


@pytest.mark.parametrize("D", [64, 1024, 2048, 16384])
@pytest.mark.parametrize("rows", [5, 2060])
def test_values_at_the_edges(D, rows):
    """Rows of zeros, tiny and huge rows; rows with values that are not finite leave the other rows their bits."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    if rows * D > 1 << 23:
        rows = 300
    X, _, gamma = made(rows, D, "fp32", "none", 3)
    group = 128 if D % 128 == 0 else 0
    X[1] = 0.0
    X[2] *= 1e-30
    X[3] *= 1e15
    calls = [(torch.float32, 0), (torch.float8_e4m3fn, 0), (torch.float8_e4m3fn, group)]
    good = [m2.m2rnn_add_norm_fwd(X, gamma, out_dtype=t, group=g) for t, g in calls]
    o, _, _ = good[0]
    check_fwd(X, None, gamma, 1e-6, "fp32", 0, o, None, X)
    check_fwd(X, None, gamma, 1e-6, "e4m3", group, good[2][0], good[2][1], X)
    assert not o[1].any() and not good[1][0][1].float().any() and float(good[1][1][1, 0]) == 2.0 ** -126
    bad = X.clone()
    bad[0, D // 2] = float("nan")
    bad[4, 1] = float("inf")
    for (t, g), (o, s, _) in zip(calls, good):
        ob, sb, _ = m2.m2rnn_add_norm_fwd(bad, gamma, out_dtype=t, group=g)
        keep = [i for i in range(rows) if i not in (0, 4)]
        assert torch.equal(ob.float()[keep], o.float()[keep])
        assert not torch.isfinite(ob.float()[0]).any() and bool(torch.isnan(ob.float()[4, 1]))
        if s is not None:
            assert torch.equal(sb[keep], s[keep]) and bool(torch.isnan(sb[0]).all())
    # eps = 0 on a row of zeros is 0/0
    assert bool(torch.isnan(m2.m2rnn_add_norm_fwd(X, gamma, eps=0.0)[0][1]).all())


def test_refusals():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    x, g = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    for kw, err in ((dict(out_dtype=torch.float16), TypeError), (dict(group=32, out_dtype=torch.float8_e4m3fn), ValueError),
                    (dict(group=128), ValueError), (dict(h=x), ValueError), (dict(scale=x), ValueError),
                    (dict(res=x.half()), TypeError), (dict(res=x[:2]), ValueError), (dict(res=x.cpu()), ValueError)):
        with pytest.raises(err):
            m2.m2rnn_add_norm_fwd(x, g, **kw)
    with pytest.raises(ValueError):
        m2.m2rnn_add_norm_fwd(x.t(), torch.ones(4, device="cuda"))
    with pytest.raises(TypeError):
        m2.m2rnn_add_norm_bwd(x, g, x.bfloat16())
