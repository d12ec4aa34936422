"""The selective state space scan on the GPU (prompt, training pair, single token) against its fp64
oracle.

Tolerance.  The kernels compute in fp32: products of exactly split operands accumulated in fp32 on
the MFMA, decays from fp64 sums of logarithms.  An output that is a sum of terms x is within
ops * 2^-24 * sum |x| of the exact one, ops the roundings that one term passes through.  A term meets:
the accumulation of its chunk (L), of the contractions over K and V, one product and one sum per
later chunk and segment (2 ceil(T / L) + 2 segments, at most 64), and for its factors: softplus
(4), the decay 2^x (x's rounding to fp32 and the hardware's exponential: 2, times |x| 2^-x ln 2 < 1,
so 2) up to three times, D_j twice, the reference point of the decay, the split's remainder,
sigma (4) and the last sum: below 32.  So ops = K + V + L + 4 ceil(T / L) + 96.  sum |x| is the oracle
run on absolute values (the decays keep their signs).  Sums over (b, t) add their tree's depth,
at most 64 + log: within the same count.
"""
import ctypes

import numpy as np
import pytest

from oracle import ssm

from _gpu import say, torch_cuda

pytestmark = pytest.mark.gpu

GRADS = ("dq", "dk", "dv", "da", "dalpha", "dbeta", "dw_r", "dH0")


def make(B, T, N, G, K, V, dtype, seed, with_H0=True, alpha=None, beta=None, a_std=1.0):
    import torch
    r = np.random.default_rng(seed)

    def rounded(x):
        x = torch.tensor(x, dtype=torch.float32)
        return (x.to(torch.bfloat16) if dtype == "bf16" else x).float().numpy()
    d = dict(q=rounded(r.normal(0, K ** -0.5, (B, T, G, K))), k=rounded(r.normal(0, K ** -0.5, (B, T, G, K))),
             v=rounded(r.normal(0, 1, (B, T, N, V))), a=r.normal(0, a_std, (B, T, N)).astype(np.float32),
             alpha=(r.uniform(0.1, 8.0, N) if alpha is None else np.full(N, alpha)).astype(np.float32),
             beta=(r.normal(-2, 2, N) if beta is None else np.full(N, beta)).astype(np.float32),
             w_r=r.normal(0, 0.3, (N, V)).astype(np.float32))
    d["H0"] = r.normal(0, 1, (B, N, K, V)).astype(np.float32) if with_H0 else None
    d["dy"] = r.normal(0, 1, (B, T, N, V)).astype(np.float32)
    d["dH_T"] = r.normal(0, 1, (B, N, K, V)).astype(np.float32)
    return d


def on_gpu(d, dtype):
    import torch
    out = {}
    for n, x in d.items():
        t = None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
        out[n] = t.to(torch.bfloat16) if n in ("q", "k", "v") and dtype == "bf16" else t
    return out


def oracle_in(d):
    return [d[x] for x in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0")]


def bounds(d, dtype, lens, back):
    """The tolerances of y, H_T and, if asked, the gradients (see the module's docstring)."""
    T, K, V = d["q"].shape[1], d["q"].shape[3], d["v"].shape[3]
    L = 64 if dtype == "bf16" else 32
    eps = (K + V + L + 4 * -(-T // L) + 96) * 2.0 ** -24
    m = {n: (x if x is None or n in ("a", "alpha", "beta") else np.abs(x)) for n, x in d.items()}
    y, HT = ssm.fwd(*oracle_in(m), lens=lens)
    tol = {"y": eps * y, "H_T": eps * HT}
    if back:
        g = ssm.bwd(*oracle_in(m), m["dy"], m["dH_T"], lens=lens, signs=-1.0)
        tol.update({n: eps * np.abs(g[n]) for n in GRADS})
    return tol


def check(got, ref, tol):
    for n, r in ref.items():
        x = got[n].double().cpu().numpy()
        assert np.all(np.isfinite(x)), n
        worst = float(np.max(np.abs(x - r) / (tol[n] + 1e-30))) if r.size else 0.0
        say(n, "worst error over its bound: %.3g" % worst)
        assert worst <= 1.0, (n, worst)


def run(t, lens=None, back=True, ws=None):
    import torch
    import matrix_state_nonlinear_m2rnn_amd as m2
    args = [t[x] for x in ("q", "k", "v", "a", "alpha", "beta", "w_r")]
    if not back:
        y, HT = m2.m2rnn_ssm_fwd(*args, t["H0"], lens=lens)
        return {"y": y, "H_T": HT}
    y, HT, ckpt = m2.m2rnn_ssm_fwd_ckpt(*args, t["H0"], lens=lens)
    g = m2.m2rnn_ssm_bwd(*args, ckpt, t["dy"], t["dH_T"], lens=lens)
    torch.cuda.synchronize()
    return {"y": y, "H_T": HT, **g}


SIZES = [
    # B, T, N, Nqk, K, V: one step, the chunk's edges, odd lengths, shared and grouped query/keys, every V, padded K
    (1, 1, 1, 1, 16, 16), (2, 2, 2, 1, 16, 32), (1, 31, 3, 3, 32, 16), (2, 64, 2, 2, 64, 64), (1, 65, 5, 1, 64, 16),
    (1, 129, 2, 2, 64, 128), (2, 100, 6, 2, 48, 16), (1, 257, 4, 2, 128, 64), (1, 700, 2, 1, 80, 32),
    (1, 190, 3, 3, 128, 128), (3, 33, 9, 1, 16, 16), (1, 1100, 1, 1, 64, 64), (1, 96, 6, 3, 112, 32),
    (64, 1030, 1, 1, 16, 16),  # thousands of chunks: the partial sums take the tree
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES)
def test_scan_and_gradients(size, dtype):
    torch_cuda()
    say("ssm", size, dtype)
    d = make(*size, dtype, seed=sum(size))
    ref = dict(zip(("y", "H_T"), ssm.fwd(*oracle_in(d))))
    ref.update(ssm.bwd(*oracle_in(d), d["dy"], d["dH_T"]))
    tol = bounds(d, dtype, None, True)
    t = on_gpu(d, dtype)
    got = run(t)
    check(got, ref, tol)
    # the forward without checkpoints is the same forward
    plain = run(t, back=False)
    assert (plain["y"] == got["y"]).all() and (plain["H_T"] == got["H_T"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size,lens", [((4, 130, 4, 2, 32, 32), [130, 1, 64, 0]), ((3, 70, 5, 1, 64, 16), [-3, 500, 33]),
                                       ((2, 200, 2, 2, 128, 64), [5, 128])])
def test_padded_batch(size, lens, dtype):
    """Steps past a sequence's end hold NaN and infinities: nothing of them is read; y and the gradients
    there are zeros."""
    torch = torch_cuda()
    say("ssm padded", size, lens, dtype)
    d = make(*size, dtype, seed=7)
    B, T = size[:2]
    ls = np.array(lens)
    past = np.arange(T)[None, :] >= np.clip(ls, 0, T)[:, None]
    ref = dict(zip(("y", "H_T"), ssm.fwd(*oracle_in(d), lens=ls)))
    ref.update(ssm.bwd(*oracle_in(d), d["dy"], d["dH_T"], lens=ls))
    tol = bounds(d, dtype, ls, True)
    for n, bad in (("q", np.nan), ("k", np.inf), ("v", np.nan), ("a", -np.inf), ("dy", np.nan)):
        d[n] = np.array(d[n])
        d[n][past] = bad
    got = run(on_gpu(d, dtype), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check(got, ref, tol)
    at = torch.from_numpy(past).cuda()
    for n in ("y", "dq", "dk", "dv", "da"):
        assert not got[n][at].any(), n


@pytest.mark.parametrize("alpha,beta,a_std", [(0.0, 0.0, 1.0), (40.0, 3.0, 2.0), (1.0, -30.0, 1.0), (1000.0, 60.0, 1.0),
                                              (-0.02, 0.0, 1.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_from_none_to_all(alpha, beta, a_std, dtype):
    """f = 1 throughout, f that forgets at once, steps of 1e-13, f that underflows, f above 1."""
    torch_cuda()
    say("ssm decays", alpha, beta, dtype)
    d = make(2, 150, 3, 3, 32, 32, dtype, seed=11, alpha=alpha, beta=beta, a_std=a_std)
    ref = dict(zip(("y", "H_T"), ssm.fwd(*oracle_in(d))))
    g = ssm.bwd(*oracle_in(d), d["dy"], d["dH_T"])
    ref.update(g)
    tol = bounds(d, dtype, None, True)
    check(run(on_gpu(d, dtype)), ref, tol)


@pytest.mark.parametrize("lowest", [-float("inf"), -3.4028234663852886e38])
def test_steps_masked_through_their_gate(lowest):
    """a at the type's lowest value: D = 0 and f = 1, so the step leaves the state as it is, and the gradients
    of what it would have written (k, v through the state, a) are zeros."""
    torch = torch_cuda()
    say(f"masked steps {lowest}")
    d = make(2, 150, 4, 2, 32, 32, "f32", 77)
    off = np.random.default_rng(3).random((2, 150, 4)) < 0.4
    off[0, :, 0] = True                       # a head with every step masked
    off[1, 64:128] = True                     # whole chunks
    d["a"][off] = lowest
    t = on_gpu(d, "f32")
    import matrix_state_nonlinear_m2rnn_amd as m2
    x = [t[n] for n in ("q", "k", "v", "a", "alpha", "beta", "w_r")]
    y, H, ckpt = m2.m2rnn_ssm_fwd_ckpt(*x, t["H0"])
    g = m2.m2rnn_ssm_bwd(*x, ckpt, t["dy"], t["dH_T"])
    assert torch.equal(H[0, 0], t["H0"][0, 0])
    at = torch.from_numpy(off).cuda()
    assert bool((g["da"][at] == 0).all())
    assert bool((g["dk"][1, 64:128] == 0).all())
    # dv there is w_r (.) dy alone
    assert torch.equal(g["dv"][1, 64:128], t["w_r"] * t["dy"][1, 64:128])
    for n, z in [("y", y), ("H", H)] + list(g.items()):
        assert bool(torch.isfinite(z).all()), n
    y1, H1 = m2.m2rnn_ssm_step(*(z[:, 70].contiguous() if z.dim() > 2 else z for z in x), t["H0"])
    assert torch.equal(H1[1], t["H0"][1]) and bool(torch.isfinite(y1).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 1, 1, 16, 16), (3, 4, 2, 48, 32), (2, 6, 1, 128, 128), (5, 2, 2, 64, 64)])
def test_steps_follow_the_scan(size, dtype):
    """A prompt, then single tokens in place, against the oracle's one scan; each step also out of place."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    B, N, G, K, V = size
    P, S = 37, 4
    say("ssm steps", size, dtype)
    d = make(B, P + S, N, G, K, V, dtype, seed=5)
    ref = ssm.fwd(*oracle_in(d))
    tol = bounds(d, dtype, None, False)
    t = on_gpu(d, dtype)
    pre = {n: (x[:, :P].contiguous() if n in ("q", "k", "v", "a") else x) for n, x in t.items()}
    y, H = m2.m2rnn_ssm_fwd(*[pre[x] for x in ("q", "k", "v", "a", "alpha", "beta", "w_r")], pre["H0"])
    ys = [y]
    for i in range(P, P + S):
        args = [t[x][:, i].contiguous() if x in ("q", "k", "v", "a") else t[x]
                for x in ("q", "k", "v", "a", "alpha", "beta", "w_r")]
        y1, H1 = m2.m2rnn_ssm_step(*args, H)
        y2, H2 = m2.m2rnn_ssm_step(*args, H, H_out=H)
        assert H2 is H and torch.equal(H1, H) and torch.equal(y1, y2)
        ys.append(y2[:, None])
    check({"y": torch.cat(ys, 1), "H_T": H}, dict(zip(("y", "H_T"), ref)), tol)
    y0, H0 = m2.m2rnn_ssm_step(*args)  # from zeros
    y1, H1 = m2.m2rnn_ssm_step(*args, torch.zeros_like(H))
    assert torch.equal(y0, y1) and torch.equal(H0, H1)


def test_empty_sequences_and_batches():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    d = make(2, 0, 4, 2, 32, 16, "f32", seed=3)
    got = run(on_gpu(d, "f32"))
    h0 = torch.from_numpy(d["H0"]).cuda()
    assert torch.equal(got["H_T"], h0) and torch.equal(got["dH0"], torch.from_numpy(d["dH_T"]).cuda())
    assert got["y"].shape == (2, 0, 4, 16)
    for n in ("dalpha", "dbeta", "dw_r"):
        assert not got[n].any()
    d = make(0, 5, 4, 2, 32, 16, "f32", seed=3)
    got = run(on_gpu(d, "f32"))
    for n in ("dalpha", "dbeta", "dw_r"):
        assert not got[n].any()
    y, H = m2.m2rnn_ssm_step(*[on_gpu(d, "f32")[x][:, 0].contiguous() if x in "qkva" else on_gpu(d, "f32")[x]
                               for x in ("q", "k", "v", "a", "alpha", "beta", "w_r")])
    assert y.shape == (0, 4, 16)


def test_graph_streams_and_dirty_workspaces():
    """Captured and replayed calls, a call on another stream with a workspace of its own, and a
    workspace that holds NaN give the eager bits."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    d = make(1, 700, 4, 2, 64, 16, "bf16", seed=21)
    t = on_gpu(d, "bf16")
    args = [t[x] for x in ("q", "k", "v", "a", "alpha", "beta", "w_r")]
    ref = {n: x.clone() for n, x in run(t).items()}
    dims = m2.Dims(1, 700, 4, 64, 16, 2)
    n = ctypes.c_size_t(0)

    def ws(name):
        assert getattr(m2.lib(), name)(ctypes.byref(dims), m2.DTYPE_BF16, ctypes.byref(n)) == 0
        return torch.full((n.value,), 255, dtype=torch.uint8, device="cuda")
    fw, bw = ws("m2rnn_ssm_fwd_workspace_size"), ws("m2rnn_ssm_bwd_workspace_size")
    out = {x: torch.empty_like(ref[x]) for x in GRADS}
    y, HT = torch.empty_like(ref["y"]), torch.empty_like(ref["H_T"])
    ckpt = torch.full((1, 4, 11, 64, 16), float("nan"), device="cuda")

    def work(stream=None):
        m2.m2rnn_ssm_fwd_ckpt(*args, t["H0"], y=y, H_T=HT, ckpt=ckpt, workspace=fw, stream=stream)
        m2.m2rnn_ssm_bwd(*args, ckpt, t["dy"], t["dH_T"], out=out, workspace=bw, stream=stream)

    def same(tag):
        torch.cuda.synchronize()
        for name, r in ref.items():
            x = y if name == "y" else HT if name == "H_T" else out[name]
            assert torch.equal(x, r), (tag, name)
    work()
    same("dirty workspace")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for x in (y, HT, *out.values()):
        x.fill_(float("nan"))
    torch.cuda.synchronize()
    work(stream=s)
    same("stream")
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        work()
    for rep in range(3):
        for x in (y, HT, ckpt, *out.values()):
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        same(rep)


def test_two_calls_at_once():
    """Training pairs issued together on two streams, each with its binding-made workspaces and outputs, give the
    bits of their solo runs."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("ssm two streams")
    sets = [on_gpu(make(2, 1500, 6, g, 64, V, "bf16", seed=40 + V), "bf16") for g, V in ((1, 16), (3, 64))]
    solo = [run(t) for t in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for t, s, o in zip(sets, streams, got):
            x = [t[n] for n in ("q", "k", "v", "a", "alpha", "beta", "w_r")]
            y, H, ckpt = m2.m2rnn_ssm_fwd_ckpt(*x, t["H0"], stream=s)
            o.append(({"y": y, "H_T": H}, m2.m2rnn_ssm_bwd(*x, ckpt, t["dy"], t["dH_T"], stream=s), ckpt))
    torch.cuda.synchronize()
    for ref, runs in zip(solo, got):
        for fwd, bwd, _ in runs:
            for n, r in ref.items():
                assert torch.equal(fwd.get(n, bwd.get(n)), r), n
