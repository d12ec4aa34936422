"""The layer's entry with a residual, its backward and the gated recurrence's backward on tensors past 2^31 elements."""
import numpy as np
import pytest

from _gpu import say, torch_cuda
from oracle import layer
from test_gpu_layer_calls import rng, same

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def room(torch, gb):
    if torch.cuda.get_device_properties(0).total_memory < gb << 30:
        pytest.skip(f"needs {gb} GB")
    torch.cuda.empty_cache()


@pytest.mark.parametrize("stream", ["fp32", "bf16"])
def test_norm_with_a_residual_and_backward(stream):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    room(torch, 80)
    say("large offsets: norm with a residual", stream)
    n = rng(43)
    rows, D = 262144 + 64, 8192  # 2.15e9 elements, 4097 times the same 64 rows
    t = torch.float32 if stream == "fp32" else torch.bfloat16
    blocks = rows // 64
    part = dict(x=n(64, D).bfloat16(), res=n(64, D).to(t), dout=n(64, D), dh=n(64, D))
    gamma = 1 + 0.1 * n(D)
    x, res = (part[k].repeat(blocks, 1) for k in ("x", "res"))
    small = m2.m2rnn_add_norm_fwd(part["x"], gamma, part["res"])
    out, _, h = m2.m2rnn_add_norm_fwd(x, gamma, res, h=res)
    assert h is res
    for k in (0, blocks // 2, blocks - 1):  # a row's sums have one order, whatever the number of rows
        at = slice(64 * k, 64 * k + 64)
        assert same([out[at], h[at]], [small[0], small[2]])
    del x, out
    dout, dh = (part[k].repeat(blocks, 1) for k in ("dout", "dh"))
    one = m2.m2rnn_add_norm_bwd(small[2], gamma, part["dout"], part["dh"])
    g = m2.m2rnn_add_norm_bwd(h, gamma, dout, dh, out={"dx": dh, "dgamma": torch.empty_like(gamma)})
    assert g["dx"] is dh
    for k in (0, blocks // 2, blocks - 1):
        assert torch.equal(dh[64 * k: 64 * k + 64], one["dx"])
    H, G, P = (z.double().cpu().numpy() for z in (small[2], gamma, part["dout"]))
    ref = blocks * layer.norm_bwd(H, G, 1e-6, P)[1]
    # as in test_gpu_norm.py: up to 64 terms in a lane, 180 u of the sum of the magnitudes
    terms = blocks * np.abs(P * layer.norm_fwd(H, np.ones(D), 1e-6)).sum(0)
    assert (np.abs(g["dgamma"].double().cpu().numpy() - ref) <= 180 * U * terms + U * np.abs(ref)).all()


def test_gated_backward():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    room(torch, 120)
    say("large offsets: gated recurrence's backward")
    n = rng(47)
    B, T, D, K = 3, 360000, 2048, 19200  # 2.2e9 elements; K: whole groups of chunks of either direction
    v, a = (torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dy = torch.empty(B, T, D, device="cuda")
    for t in (v, a, dy):  # the same sequence three times, of the same 6000 steps over and over
        t.view(B, 60, 6000, D)[:] = n(6000, D).to(t.dtype)
    alpha, beta = n(D).abs() + 1.0, n(D) - 1.0
    y, _ = m2.m2rnn_gated_scan_fwd(v, a, alpha, beta)
    g = m2.m2rnn_gated_scan_bwd(v, a, alpha, beta, y, dy)
    cut = lambda t: t[2:, -K:].contiguous()  # noqa: E731
    # chunks and groups count from the end, so the last K steps by themselves take the same sums; the first of them has another state before
    h0 = y[2:, -K - 1].contiguous()
    s = m2.m2rnn_gated_scan_bwd(cut(v), cut(a), alpha, beta, cut(y), cut(dy), h0)
    for name in ("dv", "da"):
        assert torch.equal(g[name][2:, -K:], s[name])
        assert torch.equal(g[name][0], g[name][2])
    assert torch.equal(g["dh0"][0], g["dh0"][2])
    # dbeta = sum da, dalpha = sum da softplus / (alpha sigma), from the da that were written: 20 u of the terms' magnitudes, as in
    # test_gpu_gated.py, and (26 + |z|) u for each factor of dalpha's terms
    da, db, ma, mb = (torch.zeros(D, dtype=torch.float64, device="cuda") for _ in range(4))
    for k in range(0, T, 6000):
        w = g["da"][0, k:k + 6000].double()
        z = a[0, k:k + 6000].double() + beta.double()
        q = w * torch.nn.functional.softplus(z, threshold=1e9) / (alpha.double() * torch.sigmoid(z))
        db += w.sum(0)
        mb += w.abs().sum(0)
        da += q.sum(0)
        ma += (q.abs() * (20 + 2 * (26 + z.abs()))).sum(0)
    assert bool(((g["dbeta"].double() - B * db).abs() <= B * 20 * U * mb + 2 * U * B * db.abs()).all())
    assert bool(((g["dalpha"].double() - B * da).abs() <= B * U * ma + 2 * U * B * da.abs()).all())
