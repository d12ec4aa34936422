"""The cases that the operators next to the M²RNN recurrence are measured on, with their plain forms.

Operators: the selective state space scan (per head: D_t = softplus(a_t + beta), f_t = exp(-alpha D_t),
H_t = f_t H_{t-1} + D_t k_t v_t^T, y_t = H_t^T q_t + w_r v_t) with its causal conv4 + SiLU, for prompts,
training and single tokens; the norm of queries and keys per head with the position rotation; the
global gradient norm over many tensors with clipping.
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # Prefill of a 16K-token context at the headline head shape.
        {"name": "scan_16k", "op": "scan", "B": 2, "T": 16384, "N": 32, "Nqk": 32, "K": 64, "V": 64, "dtype": "bf16",
         "ragged": False},
        # A padded batch of prompts at the pages' head shape: one query/key for 128 heads.
        {"name": "scan_shared_ragged", "op": "scan", "B": 4, "T": 4096, "N": 128, "Nqk": 1, "K": 64, "V": 16,
         "dtype": "bf16", "ragged": True},
        # A short prompt in fp32 that continues a conversation: conv windows and state in and out.
        {"name": "prompt_fp32", "op": "prompt", "B": 1, "T": 509, "N": 16, "Nqk": 16, "K": 128, "V": 128,
         "dtype": "fp32", "ragged": False},
        # A training step of the layer at the repository's training shape (forward, checkpoints, backward).
        {"name": "train_4k", "op": "train", "B": 4, "T": 4096, "N": 16, "Nqk": 16, "K": 64, "V": 64, "dtype": "bf16"},
        # The same at the pages' head shape, with the shared query/key's gradients summed over the heads.
        {"name": "train_shared", "op": "train", "B": 4, "T": 4096, "N": 128, "Nqk": 1, "K": 64, "V": 16,
         "dtype": "bf16"},
        # Serving: one token for each of 128 sequences.
        {"name": "step_b128", "op": "step", "B": 128, "N": 32, "Nqk": 32, "K": 64, "V": 64, "dtype": "bf16"},
        # Serving: one token of one sequence through conv and scan, where the latency counts.
        {"name": "token_b1", "op": "token", "B": 1, "N": 128, "Nqk": 1, "K": 64, "V": 16, "dtype": "fp32"},
        # q/k norm + rotation of a 16K-token prefill.
        {"name": "rope_16k", "op": "rope", "B": 2, "T": 16384, "Nq": 32, "Nk": 32, "K": 64, "R": 64, "inter": False,
         "dtype": "bf16"},
        # The same for one token of each of 128 sequences at far positions, grouped keys, part of the head rotated.
        {"name": "rope_token", "op": "rope", "B": 128, "T": 1, "Nq": 32, "Nk": 8, "K": 128, "R": 64, "inter": True,
         "dtype": "fp32"},
        # Its backward at a training shape.
        {"name": "rope_bwd", "op": "rope_bwd", "B": 4, "T": 4096, "Nq": 16, "Nk": 16, "K": 128, "R": 128,
         "inter": False, "dtype": "bf16"},
        # Clipping the gradients of one small layer (many small tensors, odd sizes).
        {"name": "clip_small", "op": "clip", "layers": 4, "N": 4, "K": 16, "V": 16, "width": 129, "dtype": "fp32"},
        # Clipping a whole model's gradients.
        {"name": "clip_model", "op": "clip", "layers": 24, "N": 32, "K": 64, "V": 64, "width": 2048, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng, most):
    N = _log_int(rng, 1, max(1, most))
    div = [d for d in range(1, N + 1) if N % d == 0]
    return N, rng.choice([1, N, rng.choice(div)])


def draw(rng):
    op = rng.choice(["scan", "scan", "prompt", "train", "train", "step", "token", "rope", "rope_bwd", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("scan", "prompt", "train"):
        K, V = rng.choice([16, 32, 48, 64, 96, 128]), rng.choice([16, 32, 64, 128])
        if op == "prompt":
            dtype = "fp32"
        # at most about a quarter of the largest listed case's state work
        most = (1 << 31) // (K * V) if op == "train" and dtype == "bf16" else (1 << 30) // (K * V)
        T = _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, max(1, min(8, most // T)))
        N, Nqk = _heads(rng, max(1, min(64, most // (T * B))))
        c = {"op": op, "B": B, "T": T, "N": N, "Nqk": Nqk, "K": K, "V": V, "dtype": dtype}
        if op != "train":
            c["ragged"] = rng.random() < 0.4
        return c
    if op in ("step", "token"):
        K, V = rng.choice([16, 32, 48, 64, 96, 128]), rng.choice([16, 32, 64, 128])
        N, Nqk = _heads(rng, 64)
        B = _log_int(rng, 1, max(1, min(256, (1 << 24) // (N * K * V))))
        return {"op": op, "B": B, "N": N, "Nqk": Nqk, "K": K, "V": V, "dtype": dtype if op == "step" else "fp32"}
    if op in ("rope", "rope_bwd"):
        K = rng.choice([16, 32, 64, 80, 96, 128, 256])
        R = rng.choice([K, K // 2])
        Nq = _log_int(rng, 1, 64)
        Nk = rng.choice([1, Nq, max(1, Nq // 4)])
        T = _log_int(rng, 1, 16384)
        B = _log_int(rng, 1, max(1, min(128, (1 << 25) // (T * Nq * K))))
        return {"op": op, "B": B, "T": T, "Nq": Nq, "Nk": Nk, "K": K, "R": R, "inter": rng.random() < 0.5, "dtype": dtype}
    V = rng.choice([16, 32, 64, 128])
    return {"op": "clip", "layers": _log_int(rng, 1, 16), "N": _log_int(rng, 1, 32), "K": rng.choice([16, 64, 128]),
            "V": V, "width": _log_int(rng, 33, 1537), "dtype": dtype}


def _clip_shapes(c):
    """The parameters of `layers` layers: projections, the recurrence's weights, conv taps, norm scales, gates."""
    N, K, V, D = c["N"], c["K"], c["V"], c["width"]
    C = 2 * K + N * V
    layer = [(C, D), (D, N * V), (4 * D, D), (D, 4 * D), (N, V, V), (N, V), (C, 4), (C,), (N * V,), (D,), (N,), (N,)]
    return layer * c["layers"]


# ---------------------------------------------------------------- inputs

def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


class _Gen:
    def __init__(self, seed):
        self.dev = _dev()
        self.g = torch.Generator(device=self.dev)
        self.g.manual_seed(seed)

    def normal(self, shape, std=1.0, mean=0.0, dtype=torch.float32):
        x = torch.empty(shape, dtype=torch.float32, device=self.dev)
        x.normal_(mean, std, generator=self.g)
        return x.to(dtype)

    def uniform(self, shape, lo=0.0, hi=1.0):
        x = torch.empty(shape, dtype=torch.float32, device=self.dev)
        return x.uniform_(lo, hi, generator=self.g)

    def ints(self, lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=self.g, device=self.dev, dtype=torch.int32)


def _gates(r, N):
    """alpha in [1, 16], beta = softplus^-1 of a step size spread over [1e-3, 1e-1] (its logarithm)."""
    d0 = torch.exp(r.uniform((N,), math.log(1e-3), math.log(1e-1)))
    return r.uniform((N,), 1.0, 16.0), d0 + torch.log(-torch.expm1(-d0))


def prepare(case, seed):
    c, r = case, _Gen(seed)
    s = {"c": c}
    op = c["op"]
    if op in ("scan", "prompt", "train", "step", "token"):
        B, N, G, K, V, dt = c["B"], c["N"], c["Nqk"], c["K"], c["V"], _dtype(c)
        lead = (B, c["T"]) if "T" in c else (B,)
        s["a"] = r.normal(lead + (N,))
        s["alpha"], s["beta"] = _gates(r, N)
        s["w_r"] = r.normal((N, V), 0.1 ** 0.5)
        if op in ("prompt", "token"):  # the convolution's inputs: its outputs are q, k, v
            for x, C, std in (("q", G * K, 1.0), ("k", G * K, 1.0), ("v", N * V, 1.0)):
                s["x" + x] = r.normal(lead + (C,), std, dtype=dt)
                s["w" + x] = r.normal((C, 4), 0.5)
                s["b" + x] = r.normal((C,), 0.1)
                s["win" + x] = r.normal((B, 3, C), std, dtype=dt)
        else:
            s["q"] = r.normal(lead + (G, K), K ** -0.5, dtype=dt)
            s["k"] = r.normal(lead + (G, K), K ** -0.5, dtype=dt)
            s["v"] = r.normal(lead + (N, V), dtype=dt)
        if op != "train":
            s["H0"] = r.normal((B, N, K, V), 0.3)
        else:
            s["dy"] = r.normal(lead + (N, V))
        s["lens"] = r.ints(max(1, c["T"] // 4), c["T"] + 1, (B,)) if c.get("ragged") else None
    elif op in ("rope", "rope_bwd"):
        B, T, K, R, dt = c["B"], c["T"], c["K"], c["R"], _dtype(c)
        s["q"] = r.normal((B, T, c["Nq"], K), 1.3, dtype=dt)
        s["k"] = r.normal((B, T, c["Nk"], K), 0.7, dtype=dt)
        s["gq"], s["gk"] = r.normal((K,), 0.1, 1.0), r.normal((K,), 0.1, 1.0)
        # each sequence begins at a position of its own, up to a million tokens in
        first = r.ints(0, 1 << 20, (B, 1)) if T == 1 else r.ints(0, 1 << 14, (B, 1))
        s["pos"] = (first + torch.arange(T, device=r.dev, dtype=torch.int32)[None, :]).contiguous()
        s["freq"] = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=r.dev) / R)
        if op == "rope_bwd":
            s["gqo"], s["gko"] = r.normal((B, T, c["Nq"], K)), r.normal((B, T, c["Nk"], K))
    else:
        # gradients of very unequal sizes, as layers have them
        shapes = _clip_shapes(c)
        s["g"] = [r.normal(sh, 10.0 ** -(1 + i % 5), dtype=_dtype(c)) for i, sh in enumerate(shapes)]
        # the clipped gradients go to one flat buffer, each tensor at a multiple of 128 elements
        at = [0]
        for g in s["g"]:
            at.append(at[-1] + (g.numel() + 127) // 128 * 128)
        s["flat"] = torch.zeros(at[-1], dtype=_dtype(c), device=r.dev)
        s["out"] = [s["flat"][i:i + g.numel()].view(g.shape) for i, g in zip(at, s["g"])]
        s["max_norm"] = 1.0
    return s


# ---------------------------------------------------------------- plain forms (32 bits; 64 for angles and long sums)

L = 64


def _softplus(z):
    return torch.clamp(z, min=0) + torch.log1p(torch.exp(-torch.abs(z)))


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _live(lens, T, dev):
    """[B, T] truth values: the steps within each sequence's length."""
    return torch.arange(T, device=dev)[None, :] < lens[:, None]


def _conv(x, w, b, win, lens):
    """Causal conv4 + SiLU with the three inputs before the first step; the outputs and the next window."""
    x, win = x.float(), win.float()
    T = x.shape[1]
    xx = torch.cat([win, x], 1)
    pre = xx[:, 0:T] * w[:, 0] + xx[:, 1:T + 1] * w[:, 1] + xx[:, 2:T + 2] * w[:, 2] + xx[:, 3:T + 3] * w[:, 3] + b
    u = pre * _sigmoid(pre)
    if lens is None:
        return u, xx[:, T:]
    u = u * _live(lens, T, x.device)[:, :, None]
    at = lens[:, None].long() + torch.arange(3, device=x.device)[None, :]
    return u, torch.gather(xx, 1, at[:, :, None].expand(-1, -1, x.shape[2]))


def _chunks(x, T, nc):
    """[B, T, N, X] in 32 bits -> [B, N, nc, L, X], zeros past T."""
    x = x.float()
    if nc * L != T:
        x = torch.cat([x, x.new_zeros((x.shape[0], nc * L - T) + x.shape[2:])], 1)
    return x.view(x.shape[0], nc, L, x.shape[2], x.shape[3]).permute(0, 3, 1, 2, 4).contiguous()


def _laid_out(q, k, v, a, alpha, beta, lens):
    B, T, N = a.shape
    nc = (T + L - 1) // L
    rep = N // q.shape[2]
    q, k = (_chunks(x, T, nc).repeat_interleave(rep, 1) for x in (q, k))
    v = _chunks(v, T, nc)
    delta = _softplus(a + beta)
    if lens is not None:
        delta = delta * _live(lens, T, a.device)[:, :, None]
    delta = _chunks(delta[..., None], T, nc)[..., 0]  # [B,N,nc,L]
    lc = torch.cumsum(delta.double() * -alpha.double()[None, :, None, None], -1)  # ln of the decay within the chunk
    lower = torch.ones(L, L, dtype=torch.bool, device=a.device).tril()
    dec = torch.exp((lc[..., :, None] - lc[..., None, :]).masked_fill(~lower, -math.inf)).float()
    tot = torch.cumsum(lc[..., -1], -1)  # [B,N,nc]: ln of the decay up to each chunk's end
    return B, T, N, nc, q, k, v, delta, lc, dec, tot


def _back(x, T):
    """[B, N, nc, L, X] -> [B, T, N, X]."""
    B, N, nc, _, X = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(B, nc * L, N, X)[:, :T].contiguous()


def _entry_states(k, v, delta, lc, tot, H0):
    """The state that enters each chunk, and the last state."""
    B, N, nc, _, K = k.shape
    V = v.shape[-1]
    w = delta * torch.exp(lc[..., -1:] - lc).float()
    local = torch.matmul((k * w[..., None]).transpose(-1, -2).contiguous(), v).view(B, N, nc, K * V)
    before = torch.cat([tot.new_zeros(B, N, 1), tot], -1)  # ln of the decay up to each chunk's beginning; the end
    far = torch.exp(before[..., :, None] - tot[..., None, :])
    far = far.masked_fill(~torch.ones(nc + 1, nc, dtype=torch.bool, device=k.device).tril(-1), 0.0).float()
    H = torch.matmul(far, local)
    if H0 is not None:
        H = H + torch.exp(before).float()[..., None] * H0.view(B, N, 1, K * V)
    return H[:, :, :nc].view(B, N, nc, K, V), H[:, :, nc].view(B, N, K, V).contiguous()


def _scan(q, k, v, a, alpha, beta, w_r, H0, lens):
    B, T, N, nc, q, k, v, delta, lc, dec, tot = _laid_out(q, k, v, a, alpha, beta, lens)
    Hin, HT = _entry_states(k, v, delta, lc, tot, H0)
    P = torch.matmul(q, k.transpose(-1, -2).contiguous()) * dec * delta[..., None, :]
    y = torch.matmul(P, v) + torch.exp(lc).float()[..., None] * torch.matmul(q, Hin)
    y = _back(y + w_r[None, :, None, None, :] * v, T)
    if lens is not None:
        y = y * _live(lens, T, a.device)[:, :, None, None]
    return y, HT


def _train(s):
    c = s["c"]
    alpha, w_r = s["alpha"], s["w_r"]
    G = c["Nqk"]
    B, T, N, nc, q, k, v, delta, lc, dec, tot = _laid_out(s["q"], s["k"], s["v"], s["a"], alpha, s["beta"], None)
    K, V = q.shape[-1], v.shape[-1]
    u = _chunks(s["dy"], T, nc)
    Hin, HT = _entry_states(k, v, delta, lc, tot, None)
    QK = torch.matmul(q, k.transpose(-1, -2).contiguous())
    P = QK * dec
    e = torch.exp(lc).float()  # the decay from the chunk's beginning to each step
    w = torch.exp(lc[..., -1:] - lc).float()  # and from each step to the chunk's end
    y = _back(torch.matmul(P * delta[..., None, :], v) + e[..., None] * torch.matmul(q, Hin)
              + w_r[None, :, None, None, :] * v, T)
    # R that leaves each chunk: the sum over later chunks of their local parts, decayed back
    local = torch.matmul((q * e[..., None]).transpose(-1, -2).contiguous(), u).view(B, N, nc, K * V)
    before = torch.cat([tot.new_zeros(B, N, 1), tot[..., :-1]], -1)
    far = torch.exp(before[..., None, :] - tot[..., :, None])
    keep = torch.ones(nc, nc, dtype=torch.bool, device=q.device).triu(1)
    Rout = torch.matmul(far.masked_fill(~keep, 0.0).float(), local).view(B, N, nc, K, V)
    dH0 = torch.sum(torch.exp(before)[..., None] * local, 2).view(B, N, K, V)
    X = torch.matmul(u, v.transpose(-1, -2).contiguous()) * dec
    dq_in = e[..., None] * torch.matmul(u, Hin.transpose(-1, -2).contiguous())
    dk_in = w[..., None] * torch.matmul(v, Rout.transpose(-1, -2).contiguous())
    dq = torch.matmul(X * delta[..., None, :], k) + dq_in
    dk = delta[..., None] * (torch.matmul(X.transpose(-1, -2).contiguous(), q) + dk_in)
    dv = (delta[..., None] * (torch.matmul(P.transpose(-1, -2).contiguous(), u)
                              + w[..., None] * torch.matmul(k, Rout)) + w_r[None, :, None, None, :] * u)
    # g_t = <R_t, f_t H_{t-1}>: pairs (i >= t > j) within the chunk, and what enters or leaves it
    M = (QK * X).double()
    Md = M.tril(-1) * delta.double()[..., None, :]
    span = torch.flip(torch.cumsum(torch.flip(Md.sum(-1) - Md.sum(-2), [-1]), -1), [-1])
    a_in = (q * dq_in).double().sum(-1)
    b_in = (k * dk_in).double().sum(-1)
    bd = b_in * delta.double()
    through = torch.exp(lc[..., -1:]) * (Rout.double() * Hin.double()).sum((-1, -2))[..., None]
    g = span + torch.flip(torch.cumsum(torch.flip(a_in, [-1]), -1), [-1]) + torch.cumsum(bd, -1) - bd + through
    ddelta = M.tril().sum(-2) + b_in - alpha.double()[None, :, None, None] * g
    z = s["a"].double() + s["beta"].double()
    da = _back(ddelta[..., None], T)[..., 0] * _sigmoid(z)
    out = {"y": y, "H_T": HT, "da": da.float(), "dbeta": da.sum((0, 1)).float(),
           "dalpha": -(delta.double() * g).sum((0, 2, 3)).float(), "dv": _back(dv, T), "dH0": dH0.float(),
           "dw_r": (u.double() * v.double()).sum((0, 2, 3)).float()}
    for x, d in (("dq", dq), ("dk", dk)):
        out[x] = _back(d, T).view(B, T, G, N // G, K).sum(3)
    return out


def _step(q, k, v, a, alpha, beta, w_r, H):
    rep = v.shape[1] // q.shape[1]
    q, k, v = q.float().repeat_interleave(rep, 1), k.float().repeat_interleave(rep, 1), v.float()
    delta = _softplus(a + beta)
    H = torch.exp(-alpha * delta)[..., None, None] * H + (delta[..., None] * k)[..., None] * v[:, :, None, :]
    return (H * q[..., None]).sum(2) + w_r * v, H


def _turned(x, cos, sin, inter):
    """The first 2 * cos.shape[-1] features of each head, rotated in pairs; the others as they are."""
    h = cos.shape[-1]
    if inter:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * h:]], -1)


def _angles(s):
    t = s["pos"].double()[..., None] * s["freq"]
    return torch.cos(t).float()[:, :, None, :], torch.sin(t).float()[:, :, None, :]


def _rope(s):
    cos, sin = _angles(s)

    def one(x, gamma):
        xf = x.float()
        xn = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS) * gamma
        return _turned(xn, cos, sin, s["c"]["inter"]).to(x.dtype)
    return one(s["q"], s["gq"]), one(s["k"], s["gk"])


def _rope_bwd(s):
    cos, sin = _angles(s)

    def one(x, gamma, go):
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
        gn = _turned(go, cos, -sin, s["c"]["inter"])
        p = gamma * gn
        dx = r * p - xf * (r * r * r) * (p * xf).mean(-1, keepdim=True)
        return dx, (gn * xf * r).double().sum((0, 1, 2)).float()
    dq, dgq = one(s["q"], s["gq"], s["gqo"])
    dk, dgk = one(s["k"], s["gk"], s["gko"])
    return {"dq": dq, "dk": dk, "dgamma_q": dgq, "dgamma_k": dgk}


def _clip(s):
    sums = torch.stack([(g.float() * g.float()).sum(dtype=torch.float64) for g in s["g"]])
    norm = torch.sqrt(sums.sum())
    coef = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    for g, o in zip(s["g"], s["out"]):
        o.copy_(g.float() * coef)
    return norm.float(), s["flat"]


def run(state):
    s = state
    c = s["c"]
    op = c["op"]
    if own:
        import matrix_state_nonlinear_m2rnn_amd as m2
        gate = (s["a"], s["alpha"], s["beta"], s["w_r"]) if "a" in s else None
        if op == "scan":
            return m2.m2rnn_ssm_fwd(s["q"], s["k"], s["v"], *gate, s["H0"], lens=s["lens"])
        if op == "prompt":
            B, T, N, G, K, V = (c[x] for x in ("B", "T", "N", "Nqk", "K", "V"))
            (q, wq), (k, wk), (v, wv) = (m2.m2rnn_conv4_silu_fwd_state(s["x" + x], s["w" + x], s["b" + x], s["win" + x],
                                                                       lens=s["lens"]) for x in "qkv")
            y, H = m2.m2rnn_ssm_fwd(q.view(B, T, G, K), k.view(B, T, G, K), v.view(B, T, N, V), *gate, s["H0"],
                                    lens=s["lens"])
            return y, H, wq, wk, wv
        if op == "train":
            y, H, ckpt = m2.m2rnn_ssm_fwd_ckpt(s["q"], s["k"], s["v"], *gate)
            d = m2.m2rnn_ssm_bwd(s["q"], s["k"], s["v"], *gate, ckpt, s["dy"])
            return {"y": y, "H_T": H, **d}
        if op == "step":
            return m2.m2rnn_ssm_step(s["q"], s["k"], s["v"], *gate, s["H0"])
        if op == "token":
            B, N, G, K, V = (c[x] for x in ("B", "N", "Nqk", "K", "V"))
            (q, wq), (k, wk), (v, wv) = (m2.m2rnn_conv4_silu_step(s["x" + x], s["w" + x], s["b" + x], s["win" + x])
                                         for x in "qkv")
            y, H = m2.m2rnn_ssm_step(q.view(B, G, K), k.view(B, G, K), v.view(B, N, V), *gate, s["H0"])
            return y, H, wq, wk, wv
        if op == "rope":
            return m2.m2rnn_qk_norm_rope_fwd(s["q"], s["k"], s["gq"], s["gk"], s["pos"], s["freq"], EPS,
                                             interleaved=c["inter"])
        if op == "rope_bwd":
            return m2.m2rnn_qk_norm_rope_bwd(s["q"], s["k"], s["gq"], s["gk"], s["pos"], s["freq"], s["gqo"], s["gko"],
                                             EPS, interleaved=c["inter"])
        return m2.m2rnn_grad_clip(s["g"], s["max_norm"], out=s["out"]), s["flat"]
    if op == "scan":
        return _scan(s["q"], s["k"], s["v"], s["a"], s["alpha"], s["beta"], s["w_r"], s["H0"], s["lens"])
    if op == "prompt":
        B, T, N, G, K, V = (c[x] for x in ("B", "T", "N", "Nqk", "K", "V"))
        (q, wq), (k, wk), (v, wv) = (_conv(s["x" + x], s["w" + x], s["b" + x], s["win" + x], s["lens"]) for x in "qkv")
        y, H = _scan(q.view(B, T, G, K), k.view(B, T, G, K), v.view(B, T, N, V), s["a"], s["alpha"], s["beta"],
                     s["w_r"], s["H0"], s["lens"])
        return y, H, wq.contiguous(), wk.contiguous(), wv.contiguous()
    if op == "train":
        return _train(s)
    if op == "step":
        return _step(s["q"], s["k"], s["v"], s["a"], s["alpha"], s["beta"], s["w_r"], s["H0"])
    if op == "token":
        B, N, G, K, V = (c[x] for x in ("B", "N", "Nqk", "K", "V"))
        (q, wq), (k, wk), (v, wv) = (_conv(s["x" + x][:, None], s["w" + x], s["b" + x], s["win" + x], None) for x in "qkv")
        y, H = _step(q.view(B, G, K), k.view(B, G, K), v.view(B, N, V), s["a"], s["alpha"], s["beta"], s["w_r"], s["H0"])
        return y, H, wq.contiguous(), wk.contiguous(), wv.contiguous()
    if op == "rope":
        return _rope(s)
    if op == "rope_bwd":
        return _rope_bwd(s)
    return _clip(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    op = c["op"]
    if op in ("scan", "prompt", "train", "step", "token"):
        B, N, G, K, V = (c[x] for x in ("B", "N", "Nqk", "K", "V"))
        T = c.get("T", 1)
        e = 2 if c["dtype"] == "bf16" else 4
        rows, state = B * T, 4 * B * N * K * V
        byts = rows * ((2 * G * K + N * V) * e + 4 * N + 4 * N * V)
        flops = 5 * rows * N * K * V
        if op == "train":
            byts += rows * (4 * N * V + 4 * (2 * G * K + N * V) + 4 * N) + 2 * state
            flops += 12 * rows * N * K * V
        else:
            byts += 2 * state
        if op in ("prompt", "token"):
            C = 2 * G * K + N * V
            byts += 6 * B * C * e + 20 * C
            flops += 10 * rows * C
        return {"bytes": byts, "flops": flops}
    if op in ("rope", "rope_bwd"):
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * c["T"] * (c["Nq"] + c["Nk"]) * c["K"]
        return {"bytes": n * (2 * e if op == "rope" else e + 8) + 4 * c["B"] * c["T"], "flops": n * (8 if op == "rope" else 18)}
    n = sum(math.prod(sh) for sh in _clip_shapes(c))
    return {"bytes": n * 2 * (2 if c["dtype"] == "bf16" else 4), "flops": 3 * n}


# ---------------------------------------------------------------- the definitions, in 64 bits, step by step

def _softplus64(z):
    return torch.logaddexp(z, torch.zeros_like(z))


def _exact_conv(x, w, b, win, lens):
    x, w, b, win = x.double(), w.double(), b.double(), win.double()
    B, T, C = x.shape
    u = torch.empty_like(x)
    seen = torch.cat([win, x], 1)
    for t in range(T):
        pre = (seen[:, t:t + 4] * w.t()[None]).sum(1) + b
        u[:, t] = pre / (1.0 + torch.exp(-pre))
    nxt = torch.empty_like(win)
    for i in range(B):
        n = T if lens is None else int(lens[i])
        u[i, n:] = 0.0
        nxt[i] = seen[i, n:n + 3]
    return u, nxt


def _exact_scan(q, k, v, a, alpha, beta, w_r, H0, lens, keep=False):
    """y, the last state and, if kept, the state before each step."""
    B, T, N = a.shape
    rep = N // q.shape[2]
    q, k = (x.double().repeat_interleave(rep, 2) for x in (q, k))
    v, w_r = v.double(), w_r.double()
    D = _softplus64(a.double() + beta.double())
    f = torch.exp(-alpha.double() * D)
    if lens is not None:
        on = (torch.arange(T, device=a.device)[None] < lens[:, None])[..., None].double()
        D, f = D * on, f * on + (1.0 - on)
    K, V = q.shape[-1], v.shape[-1]
    H = torch.zeros(B, N, K, V, dtype=torch.float64, device=a.device) if H0 is None else H0.double().clone()
    y = torch.empty(B, T, N, V, dtype=torch.float64, device=a.device)
    states = torch.empty(T, B, N, K, V, dtype=torch.float64, device=a.device) if keep else None
    for t in range(T):
        if keep:
            states[t] = H
        H = f[:, t, :, None, None] * H + (D[:, t, :, None] * k[:, t])[..., None] * v[:, t, :, None, :]
        y[:, t] = (H * q[:, t, :, :, None]).sum(2) + w_r * v[:, t]
    if lens is not None:
        y = y * on[..., None]
    return (y, H, states, q, k, v, D, f) if keep else (y, H)


def _exact_train(s):
    c = s["c"]
    alpha, w_r = s["alpha"].double(), s["w_r"].double()
    y, HT, states, q, k, v, D, f = _exact_scan(s["q"], s["k"], s["v"], s["a"], s["alpha"], s["beta"], s["w_r"], None,
                                               None, keep=True)
    u = s["dy"].double()
    B, T, N, K = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    g, kRv = torch.empty_like(D), torch.empty_like(D)
    C = torch.zeros_like(HT)  # f_{t+1} R_{t+1}
    after = HT
    for t in range(T - 1, -1, -1):
        R = C + q[:, t, :, :, None] * u[:, t, :, None, :]
        Rv = (R * v[:, t, :, None, :]).sum(3)
        dq[:, t] = (after * u[:, t, :, None, :]).sum(3)
        dk[:, t] = D[:, t, :, None] * Rv
        dv[:, t] = D[:, t, :, None] * (R * k[:, t, :, :, None]).sum(2) + w_r * u[:, t]
        C = f[:, t, :, None, None] * R
        g[:, t] = (C * states[t]).sum((2, 3))
        kRv[:, t] = (k[:, t] * Rv).sum(2)
        after = states[t]
    da = (kRv - alpha * g) / (1.0 + torch.exp(-(s["a"].double() + s["beta"].double())))
    G = c["Nqk"]
    return {"y": y, "H_T": HT, "dq": dq.view(B, T, G, N // G, K).sum(3), "dk": dk.view(B, T, G, N // G, K).sum(3),
            "dv": dv, "da": da, "dalpha": -(D * g).sum((0, 1)), "dbeta": da.sum((0, 1)),
            "dw_r": (u * v).sum((0, 1)), "dH0": C}


def _exact_turn(x, s, sign):
    h, inter = s["freq"].numel(), s["c"]["inter"]
    z = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                    sign * s["pos"].double()[:, :, None, None] * s["freq"])
    lo, hi = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if inter else (slice(0, h), slice(h, 2 * h))
    turned = torch.complex(x[..., lo], x[..., hi]) * z
    out = x.clone()
    out[..., lo], out[..., hi] = turned.real, turned.imag
    return out


def _exact_rope(s):
    def one(x, gamma):
        x = x.double()
        return _exact_turn(x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * gamma.double(), s, 1.0)
    return one(s["q"], s["gq"]), one(s["k"], s["gk"])


def _exact_rope_bwd(s):
    def one(x, gamma, go):
        x, gamma = x.double(), gamma.double()
        n = torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
        gn = _exact_turn(go.double(), s, -1.0)
        p = gamma * gn
        return p / n - x * (p * x).mean(-1, keepdim=True) / n.pow(3), (gn * x / n).sum((0, 1, 2))
    (dq, dgq), (dk, dgk) = one(s["q"], s["gq"], s["gqo"]), one(s["k"], s["gk"], s["gko"])
    return {"dq": dq, "dk": dk, "dgamma_q": dgq, "dgamma_k": dgk}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    op = c["op"]
    gate = (s["a"], s["alpha"], s["beta"], s["w_r"]) if "a" in s else None
    if op == "scan":
        return _exact_scan(s["q"], s["k"], s["v"], *gate, s["H0"], s["lens"])
    if op in ("prompt", "token"):
        B, N, G, K, V = (c[x] for x in ("B", "N", "Nqk", "K", "V"))
        T, token = c.get("T", 1), op == "token"
        x = {n: s["x" + n][:, None] if token else s["x" + n] for n in "qkv"}
        (q, wq), (k, wk), (v, wv) = (_exact_conv(x[n], s["w" + n], s["b" + n], s["win" + n], s["lens"]) for n in "qkv")
        a = s["a"][:, None] if token else s["a"]
        y, H = _exact_scan(q.view(B, T, G, K), k.view(B, T, G, K), v.view(B, T, N, V), a, *gate[1:], s["H0"], s["lens"])
        return (y[:, 0] if token else y), H, wq, wk, wv
    if op == "train":
        return _exact_train(s)
    if op == "step":
        y, H = _exact_scan(*(s[x][:, None] for x in ("q", "k", "v", "a")), *gate[1:], s["H0"], None)
        return y[:, 0], H
    if op == "rope":
        return _exact_rope(s)
    if op == "rope_bwd":
        return _exact_rope_bwd(s)
    norm = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in s["g"]))
    coef = min(1.0, s["max_norm"] / norm)
    flat = torch.zeros_like(s["flat"], dtype=torch.float64)
    first = s["flat"].data_ptr()
    for g, o in zip(s["g"], s["out"]):
        i = (o.data_ptr() - first) // o.element_size()
        flat[i:i + g.numel()] = g.double().flatten() * coef
    return torch.tensor(norm, dtype=torch.float64), flat
