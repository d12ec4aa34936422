"""The selective scan's layer as it is used, every piece on the GPU through the C ABI:

    training   q, k, v = conv4+SiLU(x_q, x_k, x_v); q, k normalised per head and turned by position;
               y = selective scan; out = RMSNorm(y (.) SiLU(gz)); and back, then all parameter gradients
               clipped by their global norm;
    serving    a padded batch of prompts, then token by token, against one scan over everything.

Each piece has its own tests at its own tolerance; these check that they compose.  Budget: a term passes
through at most 500 roundings of 2^-24 in a piece; in a 2-norm over many elements they add up as
sqrt(500) 2^-24 = 1.4e-6; five pieces follow each other, and sums with cancelling signs lose a factor
of three: 2e-5.
"""
import numpy as np
import pytest

from oracle import block, qk, ssm

from _gpu import rel_l2, say, torch_cuda

pytestmark = pytest.mark.gpu

EPS = 1e-6


def layer_inputs(B, T, N, G, K, V, seed):
    r = np.random.default_rng(seed)
    f32 = lambda a: np.asarray(a, dtype=np.float32)  # noqa: E731
    d = {"a": r.normal(0, 1, (B, T, N)), "alpha": r.uniform(0.2, 4.0, N), "beta": r.normal(-2, 1, N),
         "w_r": r.normal(0, 0.3, (N, V)), "gq": r.normal(1, 0.1, K), "gk": r.normal(1, 0.1, K),
         "gz": r.normal(0, 2.0, (B, T, N, V)), "gamma": r.normal(1, 0.1, (N, V)), "dout": r.normal(0, 1, (B, T, N, V))}
    for x, C in (("q", G * K), ("k", G * K), ("v", N * V)):
        d["x" + x], d["w" + x], d["b" + x] = r.normal(0, 1, (B, T, C)), r.normal(0, 0.5, (C, 4)), r.normal(0, 0.1, C)
    d = {n: f32(x) for n, x in d.items()}
    d["pos"] = np.broadcast_to(np.arange(T, dtype=np.int32) + 1000, (B, T)).copy()
    d["freq"] = 10000.0 ** (-np.arange(0, K, 2, dtype=np.float64) / K)
    return d


PARAMS = ("dwq", "dwk", "dwv", "dbq", "dbk", "dbv", "dgq", "dgk", "dalpha", "dbeta", "dw_r", "dgamma")


def oracle_layer(d, B, T, N, G, K, V):
    u = {x: block.conv4_silu_fwd(d["x" + x], d["w" + x], d["b" + x]) for x in "qkv"}
    uq, uk, uv = u["q"].reshape(B, T, G, K), u["k"].reshape(B, T, G, K), u["v"].reshape(B, T, N, V)
    q = qk.norm_rope_fwd(uq, d["gq"], d["pos"], d["freq"], EPS, False)
    k = qk.norm_rope_fwd(uk, d["gk"], d["pos"], d["freq"], EPS, False)
    args = (q, k, uv, d["a"], d["alpha"], d["beta"], d["w_r"])
    y, HT = ssm.fwd(*args)
    g = {"y": y, "H_T": HT, "out": block.out_norm_fwd(y, d["gz"], d["gamma"], EPS)}
    gn = block.out_norm_bwd(y, d["gz"], d["gamma"], EPS, d["dout"])
    gs = ssm.bwd(*args, None, gn["dy"])
    g.update({n: gs[n] for n in ("da", "dalpha", "dbeta", "dw_r")}, dgz=gn["dgz"], dgamma=gn["dgamma"])
    duq, g["dgq"] = qk.norm_rope_bwd(uq, d["gq"], d["pos"], d["freq"], EPS, False, gs["dq"])
    duk, g["dgk"] = qk.norm_rope_bwd(uk, d["gk"], d["pos"], d["freq"], EPS, False, gs["dk"])
    for x, du in (("q", duq), ("k", duk), ("v", gs["dv"])):
        c = block.conv4_silu_bwd(d["x" + x], d["w" + x], d["b" + x], du.reshape(B, T, -1))
        g["dx" + x], g["dw" + x], g["db" + x] = c["dx"], c["dw"], c["dbias"]
    return g


def gpu_layer(t, B, T, N, G, K, V):
    import matrix_state_nonlinear_m2rnn_amd as m2
    u = {x: m2.m2rnn_conv4_silu_fwd(t["x" + x], t["w" + x], t["b" + x]) for x in "qkv"}
    uq, uk, uv = u["q"].view(B, T, G, K), u["k"].view(B, T, G, K), u["v"].view(B, T, N, V)
    rope = (uq, uk, t["gq"], t["gk"], t["pos"], t["freq"])
    q, k = m2.m2rnn_qk_norm_rope_fwd(*rope, EPS)
    args = (q, k, uv, t["a"], t["alpha"], t["beta"], t["w_r"])
    y, HT, ckpt = m2.m2rnn_ssm_fwd_ckpt(*args)
    g = {"y": y, "H_T": HT, "out": m2.m2rnn_out_norm_fwd(y, t["gz"], t["gamma"], EPS)}
    gn = m2.m2rnn_out_norm_bwd(y, t["gz"], t["gamma"], t["dout"], EPS)
    gs = m2.m2rnn_ssm_bwd(*args, ckpt, gn["dy"])
    g.update({n: gs[n] for n in ("da", "dalpha", "dbeta", "dw_r")}, dgz=gn["dgz"], dgamma=gn["dgamma"])
    gr = m2.m2rnn_qk_norm_rope_bwd(*rope, gs["dq"], gs["dk"], EPS)
    g["dgq"], g["dgk"] = gr["dgamma_q"], gr["dgamma_k"]
    for x, du in (("q", gr["dq"]), ("k", gr["dk"]), ("v", gs["dv"])):
        c = m2.m2rnn_conv4_silu_bwd(t["x" + x], t["w" + x], t["b" + x], du.view(B, T, -1))
        g["dx" + x], g["dw" + x], g["db" + x] = c["dx"], c["dw"], c["dbias"]
    norm = m2.m2rnn_grad_clip([g[n] for n in PARAMS], 1.0)
    return g, norm


@pytest.mark.parametrize("size", [(2, 70, 4, 2, 32, 16), (1, 130, 2, 2, 64, 64), (2, 33, 6, 1, 16, 32)])
def test_training_step(size):
    torch = torch_cuda()
    say("ssm layer", size)
    d = layer_inputs(*size, seed=sum(size))
    ref = oracle_layer(d, *size)
    norm = np.sqrt(sum(float(np.sum(ref[n] ** 2)) for n in PARAMS))
    assert norm > 1.0  # so that the step is clipped
    for n in PARAMS:
        ref[n] = ref[n] / norm
    t = {n: torch.from_numpy(x).cuda() for n, x in d.items()}
    got, gnorm = gpu_layer(t, *size)
    assert abs(float(gnorm) - norm) <= 2e-5 * norm
    for n, r in ref.items():
        e = rel_l2(got[n].cpu().numpy(), r)
        say(n, e)
        assert e <= 2e-5, (n, e)

    # the whole step captured: every replay gives the eager step's bits
    keep = {n: x.clone() for n, x in got.items()}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cap, cnorm = gpu_layer(t, *size)
    for _ in range(3):
        for x in cap.values():
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cnorm, gnorm)
        for n, x in keep.items():
            assert torch.equal(cap[n], x), n


def test_serving_a_padded_batch():
    """Prompts of unequal lengths, then tokens; the oracle scans each sequence whole."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    B, P, S, N, G, K, V = 3, 50, 5, 4, 2, 32, 16
    lens = [50, 7, 31]
    say("ssm serving", lens)
    d = layer_inputs(B, P + S, N, G, K, V, seed=77)
    t = {n: torch.from_numpy(x).cuda() for n, x in d.items()}
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def block_of(rows, win, H, lens=None):
        """One piece of every sequence: rows [B, length] of its tokens (a list of index arrays)."""
        at = torch.from_numpy(np.stack(rows)).cuda()
        pick = lambda x: torch.gather(x, 1, at.view(B, -1, *[1] * (x.dim() - 2)).expand(-1, -1, *x.shape[2:]))  # noqa: E731
        token = at.shape[1] == 1 and lens is None
        u, nxt = {}, {}
        for x in "qkv":
            xs = pick(t["x" + x])
            if token:
                u[x], nxt[x] = m2.m2rnn_conv4_silu_step(xs[:, 0].contiguous(), t["w" + x], t["b" + x], win[x])
            else:
                u[x], nxt[x] = m2.m2rnn_conv4_silu_fwd_state(xs, t["w" + x], t["b" + x], win[x], lens=lens)
        n = at.shape[1]
        pos = at.to(torch.int32) + 1000
        q, k = m2.m2rnn_qk_norm_rope_fwd(u["q"].view(B, n, G, K), u["k"].view(B, n, G, K), t["gq"], t["gk"], pos, t["freq"],
                                         EPS)
        gate = (t["alpha"], t["beta"], t["w_r"])
        if token:
            y, H = m2.m2rnn_ssm_step(q[:, 0].contiguous(), k[:, 0].contiguous(), u["v"].view(B, N, V),
                                     pick(t["a"])[:, 0].contiguous(), *gate, H)
            return y[:, None], nxt, H
        y, H = m2.m2rnn_ssm_fwd(q, k, u["v"].view(B, n, N, V), pick(t["a"]).contiguous(), *gate, H, lens=lens)
        return y, nxt, H
    y, win, H = block_of([np.arange(P)] * B, {x: None for x in "qkv"}, None, L)
    ys = [[y[b, :lens[b]]] for b in range(B)]
    for s in range(S):
        y, win, H = block_of([np.array([n + s]) for n in lens], win, H)
        for b in range(B):
            ys[b].append(y[b])
    torch.cuda.synchronize()
    for b in range(B):
        n = lens[b] + S
        one = {x: (v[b:b + 1, :n] if v.ndim >= 3 and v.shape[:2] == (B, P + S) else v) for x, v in d.items()}
        one["pos"] = d["pos"][b:b + 1, :n]
        u = {x: block.conv4_silu_fwd(one["x" + x], d["w" + x], d["b" + x]) for x in "qkv"}
        q, k = (qk.norm_rope_fwd(u[x].reshape(1, n, G, K), d["g" + x], one["pos"], d["freq"], EPS, False) for x in "qk")
        ref, HT = ssm.fwd(q, k, u["v"].reshape(1, n, N, V), one["a"], d["alpha"], d["beta"], d["w_r"])
        got = torch.cat(ys[b]).cpu().numpy()
        assert rel_l2(got, ref[0]) <= 2e-5 and rel_l2(H[b].cpu().numpy(), HT[0]) <= 2e-5
        say("sequence", b, rel_l2(got, ref[0]), rel_l2(H[b].cpu().numpy(), HT[0]))


def test_tokens_from_a_captured_graph():
    """A token's calls captured once, the windows, the state and the position advanced in place: each replay
    is the next token, bit for bit what the eager calls give."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    B, S, N, G, K, V = 3, 6, 4, 2, 32, 16
    say("ssm tokens, captured")
    d = layer_inputs(B, S, N, G, K, V, seed=78)
    t = {n: torch.from_numpy(x).cuda() for n, x in d.items()}
    xs = [{x: t["x" + x][:, s].contiguous() for x in "qkv"} | {"a": t["a"][:, s].contiguous()} for s in range(S)]

    def fresh_state():
        return ({x: torch.zeros(B, 3, t["x" + x].shape[2], device="cuda") for x in "qkv"},
                torch.zeros(B, N, K, V, device="cuda"), torch.full((B, 1), 500, dtype=torch.int32, device="cuda"))

    def token(x, win, H, pos):
        u = {c: m2.m2rnn_conv4_silu_step(x[c], t["w" + c], t["b" + c], win[c], win_out=win[c])[0] for c in "qkv"}
        q, k = m2.m2rnn_qk_norm_rope_fwd(u["q"].view(B, 1, G, K), u["k"].view(B, 1, G, K), t["gq"], t["gk"], pos,
                                         t["freq"], EPS)
        y, _ = m2.m2rnn_ssm_step(q.view(B, G, K), k.view(B, G, K), u["v"].view(B, N, V), x["a"], t["alpha"],
                                 t["beta"], t["w_r"], H, H_out=H)
        pos += 1
        return y
    win, H, pos = fresh_state()
    want = []
    for x in xs:
        y = token(x, win, H, pos)
        want.append((y.clone(), H.clone(), {c: win[c].clone() for c in "qkv"}))
    torch.cuda.synchronize()

    win, H, pos = fresh_state()
    now = {c: torch.empty_like(x) for c, x in xs[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        y = token(now, win, H, pos)
    for s in range(S):
        for c, x in xs[s].items():
            now[c].copy_(x)
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[s][0]) and torch.equal(H, want[s][1]), s
        assert all(torch.equal(win[c], want[s][2][c]) for c in "qkv"), s
    assert int(pos[0, 0]) == 500 + S
