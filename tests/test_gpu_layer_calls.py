"""The layer's entry, the gated recurrence and the orthogonalised update as a program calls them: a training step and serving of
the layer against fp64, streams of their own, captured graphs, several calls at once, tensors past 2^31 elements."""
import numpy as np
import pytest

from _gpu import say, torch_cuda
from oracle import layer

pytestmark = pytest.mark.gpu


def rng(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, device="cuda", generator=g)


def flat(t):
    import torch
    if isinstance(t, torch.Tensor):
        return [t]
    return [x for u in (t.values() if isinstance(t, dict) else t) if u is not None for x in flat(u)]


def bits(t):
    import torch
    return t.view(torch.uint8) if t.dtype is torch.float8_e4m3fn else t


def same(a, b):
    import torch
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(flat(a), flat(b)))


def calls():
    """name -> a function of a random source that gives (call, its inputs)."""
    import torch
    import matrix_state_nonlinear_m2rnn_amd as m2
    B = torch.bfloat16

    def gated(n, dt=None, B_=2, T=700, D=512):
        v, a = n(B_, T, D), n(B_, T, D)
        if dt:
            v, a = v.to(dt), a.to(dt)
        return [v, a, n(D).abs() + 0.5, n(D) - 3.0]

    def gated_bwd(n):
        args = gated(n)
        y, _ = m2.m2rnn_gated_scan_fwd(*args)
        return m2.m2rnn_gated_scan_bwd, [*args, y, n(2, 700, 512)]

    def q8(*args, stream=None):
        return m2.m2rnn_add_norm_fwd(*args, out_dtype=torch.float8_e4m3fn, group=128, stream=stream)
    return dict(
        norm=lambda n: (m2.m2rnn_add_norm_fwd, [n(4096, 1024), n(1024), n(4096, 1024)]),
        norm_q8=lambda n: (q8, [n(4096, 1024).to(B), n(1024), n(4096, 1024).to(B)]),
        norm_bwd=lambda n: (m2.m2rnn_add_norm_bwd, [n(4096, 1024), n(1024), n(4096, 1024), n(4096, 1024)]),
        gated=lambda n: (m2.m2rnn_gated_scan_fwd, gated(n)),
        gated_bf16=lambda n: (m2.m2rnn_gated_scan_fwd, gated(n, B)),
        gated_bwd=gated_bwd,
        gated_step=lambda n: (m2.m2rnn_gated_scan_step, [n(1024, 1024), n(1024, 1024), n(1024).abs(), n(1024), n(1024, 1024)]),
        orth=lambda n: (m2.m2rnn_orthogonalize, [n(2, 300, 700)]),
        orth_small=lambda n: (m2.m2rnn_orthogonalize, [n(256, 64, 64)]),
        orth_thin=lambda n: (m2.m2rnn_orthogonalize, [n(8, 16, 8192)]))


NAMES = ["norm", "norm_q8", "norm_bwd", "gated", "gated_bf16", "gated_bwd", "gated_step", "orth", "orth_small", "orth_thin"]


def busy(m):
    for _ in range(20):
        m @ m


@pytest.mark.parametrize("name", NAMES)
def test_dropped_inputs_and_results_on_a_stream_of_their_own(name):
    torch = torch_cuda()
    say("own stream", name)
    m = torch.zeros(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    f, args = calls()[name](rng(5))
    ref = [t.clone() for t in flat(f(*args))]
    shapes = [(t.shape, t.dtype) for t in flat(args)]
    del args
    torch.cuda.synchronize()
    for _ in range(2):  # the second time round the allocator holds blocks of these sizes
        f, args = calls()[name](rng(5))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            busy(m)
        got = f(*args, stream=s)
        del args
        other = [torch.empty(shape, dtype=dt, device="cuda").fill_(77) for shape, dt in shapes]
        torch.cuda.synchronize()
        assert same(got, ref), "an input's memory was handed out while the call still read it"
        busy(m)
        copies = [t.clone() for t in flat(got)]
        sizes = [(t.shape, t.dtype) for t in flat(got)]
        del got
        with torch.cuda.stream(s):
            mine = [torch.empty(shape, dtype=torch.uint8, device="cuda").fill_(77) for shape, dt in sizes]
        torch.cuda.synchronize()
        assert same(copies, ref), "a result's memory was handed out while the caller's stream still read it"
        del other, mine, copies


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    torch = torch_cuda()
    say("graph", name)
    f, args = calls()[name](rng(7))
    ref = [t.clone() for t in flat(f(*args))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f(*args)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f(*args)
    for _ in range(4):
        for t in flat(out):
            bits(t).fill_(7)
        f(*args)  # the program's own eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(out, ref)


@pytest.mark.parametrize("name", ["gated", "gated_bwd", "orth", "orth_thin"])
def test_several_streams_at_once(name):
    """Calls on four streams at once, each with its own workspace, give what they give alone."""
    torch = torch_cuda()
    say("streams", name)
    made = [calls()[name](rng(11 + k)) for k in range(4)]
    refs = [[t.clone() for t in flat(f(*args))] for f, args in made]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [f(*args, stream=s) for (f, args), s in zip(made, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, refs):
            assert same(a, b)


def test_workspaces_are_checked():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    n = rng(3)
    v, a, al, be = n(2, 200, 64), n(2, 200, 64), n(64), n(64)
    with pytest.raises(ValueError):
        m2.m2rnn_gated_scan_fwd(v, a, al, be, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        m2.m2rnn_orthogonalize(n(300, 300), workspace=torch.empty(1 << 24, dtype=torch.uint8))
    with pytest.raises(ValueError):
        m2.m2rnn_add_norm_bwd(n(8, 64), n(64), n(8, 64), workspace=torch.empty(4, device="cuda"))


def test_training_step_of_a_layer():
    """residual + norm, projections, the gated recurrence, output gate + norm, and back; the gradients clipped, the matrices'
    updates orthogonalised: against torch's autograd and the oracle in fp64, in the 2-norm.  Everything is fp32 here, so the
    bound is some tens of fp32 roundings carried through the layer: 1e-5; five steps' amplification of at most 485 of the
    weak directions makes it 1e-3 for the update."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    n = rng(21)
    B, T, D, E = 3, 150, 96, 128
    x, res, gamma = n(B, T, D), 2 * n(B, T, D), 1 + 0.1 * n(D)
    W, gz, g2 = n(3 * E, D) * D ** -0.5, n(B, T, E), 1 + 0.1 * n(E)
    alpha, beta, h0, dout, dh = n(E).abs() + 0.5, n(E) - 2.0, n(B, E), n(B, T, E), 0.1 * n(B, T, D)
    lens = torch.tensor([150, 97, 1], dtype=torch.int32, device="cuda")
    live = (torch.arange(T, device="cuda")[None] < lens[:, None])[..., None].float()
    dout = dout * live

    xn, _, h = m2.m2rnn_add_norm_fwd(x, gamma, res, 1e-6)
    p = (xn.view(-1, D) @ W[:2 * E].t()).view(B, T, 2 * E)
    v, a = p[..., :E].contiguous(), p[..., E:].contiguous()
    y, hT = m2.m2rnn_gated_scan_fwd(v, a, alpha, beta, h0, lens=lens)
    out = m2.m2rnn_out_norm_fwd(y, gz, g2, 1e-5)
    gn = m2.m2rnn_out_norm_bwd(y, gz, g2, dout, 1e-5)
    gr = m2.m2rnn_gated_scan_bwd(v, a, alpha, beta, y, gn["dy"], h0, lens=lens)
    dp = torch.cat([gr["dv"], gr["da"]], -1).view(-1, 2 * E)
    dW = dp.t() @ xn.view(-1, D)
    back = m2.m2rnn_add_norm_bwd(h, gamma, (dp @ W[:2 * E]).view(B, T, D), dh, 1e-6)
    grads = [dW, gr["dalpha"], gr["dbeta"], back["dgamma"], gn["dgamma"]]
    before = [g.clone() for g in grads]
    norm = m2.m2rnn_grad_clip(grads, 1.0)
    up = m2.m2rnn_orthogonalize(dW)

    leaf = {k: t.double().cpu().requires_grad_(True) for k, t in dict(x=x, res=res, gamma=gamma, W=W[:2 * E], alpha=alpha,
                                                                    beta=beta, h0=h0, g2=g2).items()}
    hh = leaf["res"] + leaf["x"]
    rx = leaf["gamma"] * hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + 1e-6)
    q = rx @ leaf["W"].t()
    s, ys = leaf["h0"], []
    for t in range(T):
        f = torch.exp(-leaf["alpha"] * torch.nn.functional.softplus(q[:, t, E:] + leaf["beta"], threshold=1e9))
        on = (t < lens.cpu())[:, None]
        s = torch.where(on, f * s + (1 - f) * q[:, t, :E], s)
        ys.append(torch.where(on, s, 0.0 * s))
    ry = torch.stack(ys, 1)
    u = ry * torch.nn.functional.silu(gz.double().cpu())
    ro = leaf["g2"] * u / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-5)
    ((ro * dout.double().cpu()).sum() + (hh * dh.double().cpu()).sum()).backward()

    def near(got, ref, tol, what):
        d, r = got.double().cpu() - ref.detach(), ref.detach()
        assert float(d.norm()) <= tol * float(r.norm()), (what, float(d.norm() / r.norm()))
    near(y, ry, 1e-5, "y")
    near(hT, s, 1e-5, "h_T")
    near(out, ro, 1e-5, "out")
    near(back["dx"], leaf["x"].grad, 1e-5, "dx")
    near(back["dx"], leaf["res"].grad, 1e-5, "dres")
    near(gr["dh0"], leaf["h0"].grad, 1e-5, "dh0")
    for g, k in zip(before, ("W", "alpha", "beta", "gamma", "g2")):
        near(g, leaf[k].grad, 2e-5, k)
    total = float(sum((leaf[k].grad ** 2).sum() for k in ("W", "alpha", "beta", "gamma", "g2")) ** 0.5)
    assert abs(float(norm) - total) <= 1e-5 * total
    ref = layer.orthogonalize(leaf["W"].grad.numpy() / max(total, 1.0), 5, (3.4445, -4.7750, 2.0315), 1e-7)
    assert np.linalg.norm(up.double().cpu().numpy() - ref) <= 1e-3 * np.linalg.norm(ref)


def test_serving_of_a_padded_batch():
    """Prompts of a padded batch through the 8-bit norm and the recurrence, then tokens one at a time: the same as the whole
    sequences in one call, and padding of any content is not looked at."""
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    n = rng(31)
    B, T, E = 4, 90, 256
    lens = torch.tensor([90, 33, 64, 0], dtype=torch.int32, device="cuda")
    gamma, alpha, beta = 1 + 0.1 * n(E), n(E).abs() + 0.5, n(E) - 2.0
    x, stream, a = n(B, T + 5, E).bfloat16(), n(B, T + 5, E), n(B, T + 5, E).bfloat16()
    out, scale, h = m2.m2rnn_add_norm_fwd(x, gamma, stream, out_dtype=torch.float8_e4m3fn, group=128)
    v = (out.float().view(B, T + 5, 2, 128) * scale[..., None]).view(B, T + 5, E).bfloat16()
    whole = []  # each sequence alone: its prompt, then five tokens (the last five rows)
    for b in range(B):
        k = int(lens[b])
        take = lambda t: torch.cat([t[b:b + 1, :k], t[b:b + 1, T:]], 1).contiguous()  # noqa: E731
        whole.append(m2.m2rnn_gated_scan_fwd(take(v), take(a), alpha, beta))
    pv, pa = v[:, :T].clone(), a[:, :T].clone()
    for b in range(B):
        pv[b, int(lens[b]):] = float("nan")
        pa[b, int(lens[b]):] = float("inf")
    y, state = m2.m2rnn_gated_scan_fwd(pv, pa, alpha, beta, lens=lens)
    for t in range(5):
        row = lambda z: z[:, T + t].contiguous()  # noqa: E731
        o1, s1, h1 = m2.m2rnn_add_norm_fwd(row(x), gamma, row(stream), out_dtype=torch.float8_e4m3fn, group=128)
        assert same([o1, s1, h1], [row(out), row(scale), row(h)])
        m2.m2rnn_gated_scan_step(row(v), row(a), alpha, beta, state, h_out=state)
        for b in range(B):
            # each step adds a few roundings of values of order one, on either side
            assert float((state[b] - whole[b][0][0, int(lens[b]) + t]).abs().max()) <= 64 * 2.0 ** -24 * 4
    for b in range(B):
        k = int(lens[b])
        assert not y[b, k:].any()
        assert float((y[b, :k] - whole[b][0][0, :k]).abs().max() if k else 0.0) <= 64 * 2.0 ** -24 * 4


def test_offsets_past_2_31():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    say("large offsets: norm")
    n = rng(41)
    rows, D = 262145 + 7, 8192  # 2.15e9 elements
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda")
    some = n(64, D).bfloat16()
    x.view(-1)[: (rows // 64) * 64 * D].view(-1, 64, D)[:] = some
    x[-20:] = some[:20]
    gamma = 1 + 0.1 * n(D)
    out, scale, _ = m2.m2rnn_add_norm_fwd(x, gamma, out_dtype=torch.float8_e4m3fn, group=128)
    small, sc, _ = m2.m2rnn_add_norm_fwd(x[-64:].contiguous(), gamma, out_dtype=torch.float8_e4m3fn, group=128)
    assert same([out[-64:], scale[-64:]], [small, sc])
    del x, out, scale
    say("large offsets: gated recurrence")
    B, T, D = 3, 360000, 2048  # 2.2e9 elements
    v = torch.empty(B, T, D, dtype=torch.bfloat16, device="cuda")
    a = torch.empty_like(v)
    piece = n(6000, D).bfloat16()
    gate = n(6000, D).bfloat16()
    v.view(B, 60, 6000, D)[:] = piece
    a.view(B, 60, 6000, D)[:] = gate
    alpha, beta = n(D).abs() + 1.0, n(D) - 1.0  # memories far shorter than a piece
    y, hT = m2.m2rnn_gated_scan_fwd(v, a, alpha, beta)
    ref, _ = m2.m2rnn_gated_scan_fwd(v[:1, :18000].contiguous(), a[:1, :18000].contiguous(), alpha, beta)
    # the pieces' ends after the first two have the same past, as far as it reaches
    for b in (0, 2):
        assert float((y[b, -3000:] - ref[0, -3000:]).abs().max()) <= 64 * 2.0 ** -24 * 5
    assert torch.equal(hT, y[:, -1])
    del v, a, y


def test_sizes_of_one_and_many():
    torch = torch_cuda()
    import matrix_state_nonlinear_m2rnn_amd as m2
    n = rng(51)
    # more rows than a launch has workgroups, narrow and wide
    for rows, D in ((300001, 4), (70001, 24), (5000, 128)):
        x, gamma = n(rows, D), 1 + 0.1 * n(D)
        o, _, _ = m2.m2rnn_add_norm_fwd(x, gamma)
        ref = layer.norm_fwd(x.double().cpu().numpy(), gamma.double().cpu().numpy(), 1e-6)
        assert float(np.abs(o.double().cpu().numpy() - ref).max()) <= 48 * 2.0 ** -24 * float(np.abs(ref).max())
        g = m2.m2rnn_add_norm_bwd(x, gamma, x)
        dg = layer.norm_bwd(x.double().cpu().numpy(), gamma.double().cpu().numpy(), 1e-6, x.double().cpu().numpy())[1]
        assert float(np.abs(g["dgamma"].double().cpu().numpy() - dg).max()) <= 180 * 2.0 ** -24 * float(np.abs(dg).max())
    # thousands of matrices, and one of a single column
    g = n(5000, 8, 12)
    o = m2.m2rnn_orthogonalize(g)
    assert torch.equal(m2.m2rnn_orthogonalize(g[4321].contiguous()), o[4321])
    c = n(1, 4097, 1)
    o = m2.m2rnn_orthogonalize(c).double()
    s = 1.0
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    # one singular value: the unit vector times its image, with a few roundings a step
    assert float((o - s * c.double() / c.double().norm()).norm()) <= 5 * 32 * 2.0 ** -24
