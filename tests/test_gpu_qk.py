"""The norm of queries and keys per head with the position rotation, on the GPU against its fp64 oracle.

Tolerances count roundings to fp32 (2^-24 of the value each).  Forward: the sum of squares (8 in a lane,
5 across lanes, mean, eps) halves into r, plus its root and quotient: 10; x r gamma: 2; a sine or
cosine: the reduced angle and its series within 4 of 1; the products and their difference 3.  So
24 of (|a| + |b|) for a pair (a, b) of the normalised head; bf16 outputs add half a step, 2^-8 of the
value.  Backward: gn is within 8 of (|ga| + |gb|); dx = r p - r^3 x dot / K adds r^3 (30) and dot's
14: 64 of r |p| + r^3 |x| sum |p x| / K.  dgamma sums one term per row: (rows + 64).
"""
import numpy as np
import pytest

from oracle import qk

from _gpu import say, torch_cuda

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(B, T, Nq, Nk, K, R, dtype, seed, far=True):
    import torch
    r = np.random.default_rng(seed)

    def rounded(x):
        t = torch.tensor(x, dtype=torch.float32)
        return (t.to(torch.bfloat16) if dtype == "bf16" else t).float().numpy()
    return dict(q=rounded(r.normal(0, 2, (B, T, Nq, K))), k=rounded(r.normal(0, 0.5, (B, T, Nk, K))),
                gq=r.normal(1, 0.2, K).astype(np.float32), gk=r.normal(1, 0.2, K).astype(np.float32),
                pos=(r.integers(0, 1 << 20, (B, T)) if far else np.arange(B * T).reshape(B, T)).astype(np.int32),
                freq=10000.0 ** (-np.arange(0, R, 2, dtype=np.float64) / max(R, 1)),
                dq=r.normal(0, 1, (B, T, Nq, K)).astype(np.float32), dk=r.normal(0, 1, (B, T, Nk, K)).astype(np.float32))


def on_gpu(d, dtype):
    import torch
    return {n: torch.from_numpy(np.ascontiguousarray(x)).cuda().to(torch.bfloat16 if dtype == "bf16" and n in "qk" else
                                                                   torch.from_numpy(x).dtype) for n, x in d.items()}


def pair_sum(x, R, inter):
    """|a| + |b| of each feature's pair (|x| where it is not turned)."""
    a, b = qk.pairs(x.shape[-1], R, inter)
    s = np.abs(x)
    out = s.copy()
    out[..., a] = out[..., b] = s[..., a] + s[..., b]
    return out


def within(name, got, ref, tol):
    x = got.double().cpu().numpy()
    assert np.all(np.isfinite(x)), name
    worst = float(np.max(np.abs(x - ref) / (tol + 1e-37))) if ref.size else 0.0
    say(name, "worst error over its bound: %.3g" % worst)
    assert worst <= 1.0, (name, worst)


CASES = [
    # B, T, Nq, Nk, K, R: single tokens, every lane count, odd K and head counts, part of the head, no keys
    (1, 1, 1, 1, 16, 16), (3, 1, 5, 1, 64, 64), (2, 37, 4, 2, 64, 32), (1, 7, 32, 8, 128, 128), (2, 5, 3, 3, 80, 40),
    (1, 33, 2, 1, 256, 256), (2, 3, 7, 7, 48, 24), (1, 130, 9, 3, 32, 8), (1, 4, 6, 2, 96, 96), (2, 9, 4, 0, 64, 64),
    (2, 9, 0, 4, 112, 56), (1, 5, 3, 2, 64, 0), (1, 3000, 2, 1, 16, 8),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(case, inter, dtype):
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    B, T, Nq, Nk, K, R = case
    say("qk norm rope", case, inter, dtype)
    eps = 1e-6
    d = make(*case, dtype, seed=sum(case))
    t = on_gpu(d, dtype)
    args = (t["q"], t["k"], t["gq"], t["gk"], t["pos"], t["freq"])
    qo, ko = m2.m2rnn_qk_norm_rope_fwd(*args, eps, interleaved=inter)
    g = m2.m2rnn_qk_norm_rope_bwd(*args, t["dq"], t["dk"], eps, interleaved=inter)
    torch.cuda.synchronize()
    assert qo.dtype == t["q"].dtype
    for x, gamma, out, do, dx, dg in (("q", "gq", qo, "dq", g["dq"], g["dgamma_q"]),
                                      ("k", "gk", ko, "dk", g["dk"], g["dgamma_k"])):
        r = 1.0 / np.sqrt(np.mean(d[x].astype(np.float64) ** 2, axis=-1, keepdims=True) + eps)
        ref = qk.norm_rope_fwd(d[x], d[gamma], d["pos"], d["freq"], eps, inter)
        tol = 24 * U * pair_sum(d[gamma] * d[x] * r, R, inter)
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        within(x + " out", out, ref, tol)
        rdx, rdg = qk.norm_rope_bwd(d[x], d[gamma], d["pos"], d["freq"], eps, inter, d[do])
        p = np.abs(d[gamma]) * pair_sum(d[do].astype(np.float64), R, inter)
        within("d" + x, dx, rdx, 64 * U * (r * p + r ** 3 * np.abs(d[x]) * np.mean(p * np.abs(d[x]), -1, keepdims=True)))
        rows = B * T * d[x].shape[2]
        within("dgamma " + x, dg, rdg, (rows + 64) * U * np.sum(p / np.abs(d[gamma]) * np.abs(d[x]) * r, axis=(0, 1, 2)))


def test_far_and_negative_positions():
    """Positions up to the end of int32: the angle of the first pair is the position itself."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    d = make(1, 6, 2, 2, 32, 32, "f32", seed=1)
    d["pos"] = np.array([[0, -1, -(1 << 31), (1 << 31) - 1, 123456789, -7]], dtype=np.int32)
    t = on_gpu(d, "f32")
    qo, _ = m2.m2rnn_qk_norm_rope_fwd(t["q"], t["k"], t["gq"], t["gk"], t["pos"], t["freq"], 1e-6)
    ref = qk.norm_rope_fwd(d["q"], d["gq"], d["pos"], d["freq"], 1e-6, False)
    r = 1.0 / np.sqrt(np.mean(d["q"].astype(np.float64) ** 2, axis=-1, keepdims=True) + 1e-6)
    # two fp64 roundings of an angle of 2^31 are 2^-21 each; the oracle's own angle has one of them
    within("q out", qo, ref, (24 * U + 3 * 2.0 ** -22) * pair_sum(d["gq"] * d["q"] * r, 32, False))


def test_rows_of_zeros_and_empty_batches():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    d = make(1, 4, 2, 2, 64, 64, "f32", seed=2)
    d["q"][:, 1] = 0.0
    t = on_gpu(d, "f32")
    args = (t["q"], t["k"], t["gq"], t["gk"], t["pos"], t["freq"])
    qo, ko = m2.m2rnn_qk_norm_rope_fwd(*args, 1e-6)
    g = m2.m2rnn_qk_norm_rope_bwd(*args, t["dq"], t["dk"], 1e-6)
    assert not qo[:, 1].any() and torch.isfinite(g["dq"]).all()
    e = {n: (x[:, :0].contiguous() if x.dim() > 1 else x) for n, x in t.items()}
    args = (e["q"], e["k"], e["gq"], e["gk"], e["pos"], e["freq"])
    qo, ko = m2.m2rnn_qk_norm_rope_fwd(*args)
    assert qo.shape == (1, 0, 2, 64)
    g = m2.m2rnn_qk_norm_rope_bwd(*args, e["dq"], e["dk"])
    assert not g["dgamma_q"].any() and not g["dgamma_k"].any()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("eps,scale", [(0.0, 1.0), (1e-30, 1.0), (1e-30, 1e15), (1e-6, 1e15), (1e-30, 1e-12), (1.0, 1e-18)])
def test_magnitudes_and_small_eps(eps, scale, inter):
    """Heads of 1e15 and of 1e-12, rows of zeros (padding) beside them where eps allows them, and eps = 0 with
    head counts that leave a wave's last lanes without a head: the same bounds as above."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("qk magnitudes", eps, scale, inter)
    eps = float(np.float32(eps))
    for B, T, Nq, Nk, K, R in ((2, 9, 5, 2, 64, 32), (1, 7, 3, 0, 16, 16), (1, 6, 1, 2, 112, 56)):
        d = make(B, T, Nq, Nk, K, R, "f32", seed=K)
        for x in ("q", "k"):
            d[x] = (d[x] * np.float32(scale)).astype(np.float32)
            if eps > 0:
                d[x][:, 1:3] = 0.0
        t = on_gpu(d, "f32")
        args = (t["q"], t["k"], t["gq"], t["gk"], t["pos"], t["freq"])
        qo, ko = m2.m2rnn_qk_norm_rope_fwd(*args, eps, interleaved=inter)
        g = m2.m2rnn_qk_norm_rope_bwd(*args, t["dq"], t["dk"], eps, interleaved=inter)
        for x, gamma, out, do, dx, dg in (("q", "gq", qo, "dq", g["dq"], g["dgamma_q"]),
                                          ("k", "gk", ko, "dk", g["dk"], g["dgamma_k"])):
            r = 1.0 / np.sqrt(np.mean(d[x].astype(np.float64) ** 2, axis=-1, keepdims=True) + eps)
            ref = qk.norm_rope_fwd(d[x], d[gamma], d["pos"], d["freq"], eps, inter)
            within(x + " out", out, ref, 24 * U * pair_sum(d[gamma] * d[x] * r, R, inter))
            rdx, rdg = qk.norm_rope_bwd(d[x], d[gamma], d["pos"], d["freq"], eps, inter, d[do])
            p = np.abs(d[gamma]) * pair_sum(d[do].astype(np.float64), R, inter)
            within("d" + x, dx, rdx,
                   64 * U * (r * p + r ** 3 * np.abs(d[x]) * np.mean(p * np.abs(d[x]), -1, keepdims=True)))
            rows = B * T * d[x].shape[2]
            within("dgamma " + x, dg, rdg,
                   (rows + 64) * U * np.sum(p / np.abs(d[gamma]) * np.abs(d[x]) * r, axis=(0, 1, 2)))


def test_scale_gradients_that_cancel():
    """Two million tokens, the second half's gradients with the other sign.  A term x r of dgamma meets six roundings, its sum
    in a lane is of 64 terms, half of each sign: so of 32 terms at most.  The bound is six standard deviations of roundings of
    2^-24 of their values, evenly distributed."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    T, K = 1 << 21, 16
    say("qk cancelling sums", T)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.empty(1, T, 1, K, device="cuda").normal_(generator=g).abs() + 1.0
    k = torch.empty(1, T, 0, K, device="cuda")
    gamma = torch.ones(K, device="cuda")
    dq = torch.ones_like(q)
    dq[:, T // 2:] = -1.0
    pos = torch.zeros(1, T, dtype=torch.int32, device="cuda")
    d = m2.m2rnn_qk_norm_rope_bwd(q, k, gamma, gamma, pos, torch.empty(0, dtype=torch.float64, device="cuda"), dq, k, 0.0)
    x = q.double()[0, :, 0]
    terms = x / x.pow(2).mean(-1, keepdim=True).sqrt()
    ref = terms[:T // 2].sum(0) - terms[T // 2:].sum(0)
    tol = 6 * U * torch.sqrt((terms ** 2).sum(0) * (6 ** 2 + 32 ** 2) / 3) + U * ref.abs()
    worst = float(((d["dgamma_q"].double() - ref).abs() / tol).max())
    say("dgamma worst error over its bound: %.3g" % worst)
    assert worst <= 1.0


def test_graph_and_stream():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    t = on_gpu(make(2, 70, 4, 2, 64, 64, "bf16", seed=3), "bf16")
    args = (t["q"], t["k"], t["gq"], t["gk"], t["pos"], t["freq"])
    qo, ko = m2.m2rnn_qk_norm_rope_fwd(*args)
    ref = m2.m2rnn_qk_norm_rope_bwd(*args, t["dq"], t["dk"])
    out = {n: torch.empty_like(x) for n, x in ref.items()}
    q2, k2 = torch.empty_like(qo), torch.empty_like(ko)
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()

    def work(stream=None):
        m2.m2rnn_qk_norm_rope_fwd(*args, q_out=q2, k_out=k2, stream=stream)
        m2.m2rnn_qk_norm_rope_bwd(*args, t["dq"], t["dk"], out=out, workspace=ws, stream=stream)

    def same():
        torch.cuda.synchronize()
        assert torch.equal(q2, qo) and torch.equal(k2, ko)
        assert all(torch.equal(out[n], ref[n]) for n in ref)
    work(stream=s)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        work()
    for _ in range(3):
        for x in (q2, k2, *out.values()):
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        same()
