"""The cases that a linear layer's entry, its recurrence over channels and the update of its matrices are measured on,
with their plain forms.

Operators: the residual's addition with the RMSNorm of the sum (h = res + x, out = gamma h / sqrt(mean h^2 + eps)), its
output in 32, 16 or 8 bits with scales, and its gradient; the gated linear recurrence of channels
(f_t = exp(-alpha softplus(a_t + beta)), h_t = f_t h_{t-1} + (1 - f_t) v_t) for prompts, training and single tokens; the
orthogonalised update (X = G / (||G|| + eps), then X <- a X + (b A + c A A) X with A = X X^T, five times).
"""
import math

import torch

own = False

EPS = 1e-6
COEFS = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7


# ---------------------------------------------------------------- cases

def listed():
    return [
        # The entry of a layer in a 16K-token prefill: fp32 residual stream, bf16 branch, bf16 output for the projections.
        {"name": "norm_16k", "op": "norm", "rows": 32768, "D": 2048, "x": "bf16", "res": "fp32", "out": "bf16", "group": 0},
        # The same with a bf16 stream and an 8-bit output, one scale for every 128 features.
        {"name": "norm_e4m3", "op": "norm", "rows": 32768, "D": 2048, "x": "bf16", "res": "bf16", "out": "e4m3",
         "group": 128},
        # One token for each of 128 sequences, one scale a row: the latency counts.
        {"name": "norm_token", "op": "norm", "rows": 128, "D": 2048, "x": "bf16", "res": "fp32", "out": "e4m3", "group": 0},
        # The norm's backward at the training shape, with the gradient that comes down the residual stream.
        {"name": "norm_bwd", "op": "norm_bwd", "rows": 16384, "D": 2048, "h": "fp32", "stream": True},
        # The recurrence over a 16K-token context (prefill), as many channels as the headline has value columns.
        {"name": "gated_16k", "op": "gated", "B": 2, "T": 16384, "D": 2048, "dtype": "bf16", "ragged": False},
        # A padded batch in fp32 with an odd length and width that continues from states.
        {"name": "gated_ragged", "op": "gated", "B": 3, "T": 4093, "D": 1100, "dtype": "fp32", "ragged": True},
        # A training step of the recurrence (forward and backward) at the training shape.
        {"name": "gated_train", "op": "gated_train", "B": 4, "T": 4096, "D": 2048, "dtype": "bf16"},
        # Serving: one token for each of 128 sequences.
        {"name": "gated_token", "op": "gated_step", "B": 128, "D": 2048, "dtype": "bf16"},
        # The recurrence's matrices W of a model: 24 layers of 32 heads.
        {"name": "orth_heads", "op": "orth", "batch": 768, "m": 64, "n": 64, "dtype": "fp32"},
        # The query/key/value projection of a layer (2K + NV rows).
        {"name": "orth_qkv", "op": "orth", "batch": 1, "m": 2176, "n": 2048, "dtype": "fp32"},
        # The MLP's first matrix, in bf16.
        {"name": "orth_mlp", "op": "orth", "batch": 1, "m": 8192, "n": 2048, "dtype": "bf16"},
        # A few small odd ones.
        {"name": "orth_odd", "op": "orth", "batch": 6, "m": 129, "n": 515, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "gated", "gated", "gated_train", "gated_step", "orth", "orth", "orth"])
    if op in ("norm", "norm_bwd"):
        D = 128 * _log_int(rng, 1, 128) if rng.random() < 0.5 else 4 * _log_int(rng, 1, 4096)
        rows = _log_int(rng, 1, max(1, min(100000, (1 << 25) // D)))
        if op == "norm_bwd":
            return {"op": op, "rows": rows, "D": D, "h": rng.choice(["fp32", "bf16"]), "stream": rng.random() < 0.7}
        out = rng.choice(["fp32", "bf16", "e4m3", "e4m3"])
        return {"op": op, "rows": rows, "D": D, "x": rng.choice(["fp32", "bf16"]), "res": rng.choice(["fp32", "bf16", "none"]),
                "out": out, "group": 128 if out == "e4m3" and D % 128 == 0 and rng.random() < 0.6 else 0}
    if op == "gated_step":
        D = 4 * _log_int(rng, 1, 2048)
        return {"op": op, "B": _log_int(rng, 1, max(1, min(512, (1 << 20) // D))), "D": D, "dtype": rng.choice(["fp32", "bf16"])}
    if op in ("gated", "gated_train"):
        most = 1 << 25 if op == "gated" else 1 << 24
        T = _log_int(rng, 1, 32768)
        D = 4 * _log_int(rng, 1, max(1, min(2048, most // (4 * T))))
        B = _log_int(rng, 1, max(1, min(64, most // (T * D))))
        return {"op": op, "B": B, "T": T, "D": D, "dtype": rng.choice(["fp32", "bf16"]), "ragged": rng.random() < 0.5}
    m = _log_int(rng, 1, 4096)
    n = rng.choice([m, _log_int(rng, 1, 4096), _log_int(rng, 1, 4096)])
    batch = _log_int(rng, 1, max(1, min(512, (1 << 22) // (m * n))))
    return {"op": "orth", "batch": batch, "m": m, "n": n, "dtype": rng.choice(["fp32", "bf16"])}


# ---------------------------------------------------------------- inputs

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


class _Gen:
    def __init__(self, seed):
        self.dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
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


def prepare(case, seed):
    c, r = case, _Gen(seed)
    s = {"c": c}
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        rows, D = c["rows"], c["D"]
        s["gamma"] = r.normal((D,), 0.1, 1.0)
        # a residual stream has a few features far larger than the others
        big = torch.exp(r.normal((D,), 0.7))
        if op == "norm":
            s["x"] = r.normal((rows, D), 0.5, dtype=_TYPES[c["x"]])
            s["res"] = None if c["res"] == "none" else (r.normal((rows, D)) * big).to(_TYPES[c["res"]])
        else:
            s["h"] = (r.normal((rows, D)) * big).to(_TYPES[c["h"]])
            s["dout"] = r.normal((rows, D), 0.01)
            s["dh"] = r.normal((rows, D), 0.01) if c["stream"] else None
    elif op in ("gated", "gated_train", "gated_step"):
        B, D, dt = c["B"], c["D"], _TYPES[c["dtype"]]
        lead = (B,) if op == "gated_step" else (B, c["T"])
        s["v"], s["a"] = r.normal(lead + (D,), dtype=dt), r.normal(lead + (D,), dtype=dt)
        # alpha in [1, 16], beta = softplus^-1 of a step size spread over [1e-3, 1e-1] (its logarithm)
        d0 = torch.exp(r.uniform((D,), math.log(1e-3), math.log(1e-1)))
        s["alpha"], s["beta"] = r.uniform((D,), 1.0, 16.0), d0 + torch.log(-torch.expm1(-d0))
        s["h0"] = None if op == "gated_train" and not c.get("ragged") else r.normal((B, D), 0.3)
        s["lens"] = r.ints(0, c["T"] + 1, (B,)) if c.get("ragged") else None
        if op == "gated_train":
            s["dy"] = r.normal(lead + (D,))
            s["dh_T"] = r.normal((B, D)) if c.get("ragged") else None
    else:
        b, m, n = c["batch"], c["m"], c["n"]
        # a gradient: a few strong directions of falling strength over noise
        k = max(1, min(m, n) // 16)
        fall = torch.exp(-4.0 * torch.arange(k, device=r.dev) / k)
        g = torch.matmul(r.normal((b, m, k)) * fall, r.normal((b, k, n)))
        s["g"] = (1e-3 * (g + r.normal((b, m, n), 0.3))).to(_TYPES[c["dtype"]])
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits

def _norm(s):
    c = s["c"]
    h = s["x"] if s["res"] is None else (s["res"].float() + s["x"].float()).to(s["res"].dtype)
    hf = h.float()
    y = hf * torch.rsqrt((hf * hf).mean(-1, keepdim=True) + EPS) * s["gamma"]
    kept = None if s["res"] is None else h
    if c["out"] != "e4m3":
        return y.to(_TYPES[c["out"]]), None, kept
    g = c["group"] or c["D"]
    y = y.view(c["rows"], c["D"] // g, g)
    scale = torch.clamp(y.abs().amax(-1) / 448.0, min=2.0 ** -126)
    return (y / scale[..., None]).to(torch.float8_e4m3fn).view(c["rows"], c["D"]), scale, kept


def _norm_bwd(s):
    h, p = s["h"].float(), s["gamma"] * s["dout"]
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    hn = h * r
    dx = r * (p - hn * (p * hn).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"]
    return {"dx": dx, "dgamma": (s["dout"] * hn).sum(0, dtype=torch.float64).float()}


def _gate(s):
    """softplus(z), sigma(z) and i = 1 - f, which keeps its digits where f is next to 1."""
    z = s["a"].float() + s["beta"]
    t = torch.exp(-torch.abs(z))
    sp = torch.clamp(z, min=0) + torch.log1p(t)
    return sp, torch.where(z < 0, t, torch.ones_like(t)) / (1.0 + t), -torch.expm1(-s["alpha"] * sp)


def _live(s):
    T = s["c"]["T"]
    return (torch.arange(T, device=s["lens"].device)[None, :] < s["lens"][:, None])[..., None]


def _scan(i, b):
    """h_t = (1 - i_t) h_{t-1} + b_t from h = 0, by doubling: after the pass of span w each step holds the last 2w steps'."""
    T, w = i.shape[1], 1
    while w < T:
        h = b.clone()
        h[:, w:] = b[:, w:] + b[:, :-w] - i[:, w:] * b[:, :-w]
        b = h
        if 2 * w < T:
            j = i.clone()
            j[:, w:] = i[:, w:] + i[:, :-w] - i[:, w:] * i[:, :-w]
            i = j
        w *= 2
    return b


def _gated(s):
    i = _gate(s)[2]
    v = s["v"].float()
    if s["lens"] is not None:
        i = i * _live(s)
    b = i * v
    if s["h0"] is not None:
        b[:, 0] += (1.0 - i[:, 0]) * s["h0"]
    y = _scan(i, b)
    h_T = y[:, -1].clone()
    if s["lens"] is not None:
        y = y * _live(s)
    return y, h_T


def _gated_train(s):
    y, h_T = _gated(s)
    sp, sg, i = _gate(s)
    v, dy, alpha = s["v"].float(), s["dy"], s["alpha"]
    if s["lens"] is not None:
        live = _live(s)
        i, dy = i * live, dy * live
    # R_t = dy_t + f_{t+1} R_{t+1}: the same scan, backwards, its gates one step later
    b = dy.clone()
    if s["dh_T"] is not None:
        b[:, -1] += s["dh_T"]
    j = torch.cat([i[:, 1:], torch.zeros_like(i[:, :1])], 1)
    R = torch.flip(_scan(torch.flip(j, [1]), torch.flip(b, [1])), [1])
    h0 = torch.zeros_like(y[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([h0, y[:, :-1]], 1)
    f = torch.exp(-alpha * sp)
    if s["lens"] is not None:
        f = f * live
    G = f * R * (before - v)
    da = -alpha * sg * G
    return {"y": y, "h_T": h_T, "dv": i * R, "da": da, "dalpha": -(sp * G).sum((0, 1), dtype=torch.float64).float(),
            "dbeta": da.sum((0, 1), dtype=torch.float64).float(), "dh0": (1.0 - i[:, 0]) * R[:, 0]}


def _gated_step(s):
    i = _gate(s)[2]
    return s["h0"] + i * (s["v"].float() - s["h0"])


def _orth(s):
    a, b, c = COEFS
    X = s["g"].float()
    tall = X.shape[1] > X.shape[2]
    if tall:
        X = X.transpose(1, 2).contiguous()
    norm = torch.sqrt((X.double() * X.double()).sum((1, 2), keepdim=True)).float()
    X = X / (norm + NS_EPS)
    for _ in range(5):
        A = torch.matmul(X, X.transpose(1, 2).contiguous())
        X = a * X + torch.matmul(b * A + c * torch.matmul(A, A), X)
    if tall:
        X = X.transpose(1, 2).contiguous()
    return X.to(s["g"].dtype)


def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        import matrix_state_nonlinear_m2rnn_amd as m2
        if op == "norm":
            out, scale, h = m2.m2rnn_add_norm_fwd(s["x"], s["gamma"], s["res"], EPS, out_dtype=_TYPES[s["c"]["out"]],
                                                  group=s["c"]["group"])
            return out, scale, None if s["res"] is None else h
        if op == "norm_bwd":
            return m2.m2rnn_add_norm_bwd(s["h"], s["gamma"], s["dout"], s["dh"], EPS)
        if op == "orth":
            return m2.m2rnn_orthogonalize(s["g"], steps=5, coefs=COEFS, eps=NS_EPS)
        gate = (s["v"], s["a"], s["alpha"], s["beta"])
        if op == "gated":
            return m2.m2rnn_gated_scan_fwd(*gate, s["h0"], lens=s["lens"])
        if op == "gated_step":
            return m2.m2rnn_gated_scan_step(*gate, s["h0"])
        y, h_T = m2.m2rnn_gated_scan_fwd(*gate, s["h0"], lens=s["lens"])
        d = m2.m2rnn_gated_scan_bwd(*gate, y, s["dy"], s["h0"], s["dh_T"], lens=s["lens"])
        return {"y": y, "h_T": h_T, **d}
    return {"norm": _norm, "norm_bwd": _norm_bwd, "gated": _gated, "gated_train": _gated_train, "gated_step": _gated_step,
            "orth": _orth}[op](s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    op = c["op"]
    size = {"fp32": 4, "bf16": 2, "e4m3": 1, "none": 0}
    if op == "norm":
        scales = 4 * (c["D"] // (c["group"] or c["D"])) if c["out"] == "e4m3" else 0
        return {"bytes": c["rows"] * (c["D"] * (size[c["x"]] + 2 * size[c["res"]] + size[c["out"]]) + scales) + 4 * c["D"],
                "flops": 6 * c["rows"] * c["D"]}
    if op == "norm_bwd":
        n = c["rows"] * c["D"]
        return {"bytes": n * (size[c["h"]] + 8 + (4 if c["stream"] else 0)) + 8 * c["D"], "flops": 12 * n}
    if op == "orth":
        m, n = min(c["m"], c["n"]), max(c["m"], c["n"])
        # X X^T and A A are symmetric: half of each is enough
        step = m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n
        return {"bytes": 2 * c["batch"] * m * n * size[c["dtype"]], "flops": 5 * c["batch"] * step}
    e = size[c["dtype"]]
    n = c["B"] * c.get("T", 1) * c["D"]
    states = 4 * c["B"] * c["D"]
    if op == "gated_step":
        return {"bytes": n * 2 * e + 2 * states + 8 * c["D"], "flops": 12 * n}
    if op == "gated":
        return {"bytes": n * (2 * e + 4) + 2 * states + 8 * c["D"], "flops": 12 * n}
    return {"bytes": n * (2 * e + 16) + 2 * states + 16 * c["D"], "flops": 34 * n}


# ---------------------------------------------------------------- the definitions, in 64 bits, step by step

def _e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even: steps of 2^(e - 3), e the exponent, -6 at least."""
    e = torch.clamp(torch.frexp(x)[1] - 1, min=-6)
    step = torch.ldexp(torch.ones_like(x), e - 3)
    return torch.round(x / step) * step


def _exact_norm(s):
    c, x, gamma = s["c"], s["x"].double(), s["gamma"].double()
    # the stream is kept in its type, and the norm is of what is kept
    h = x if s["res"] is None else (s["res"].double() + x).float().to(s["res"].dtype).double()
    kept = None if s["res"] is None else s["res"].double() + x
    y = torch.empty_like(h)
    for i in range(0, c["rows"], 4096):
        part = h[i:i + 4096]
        y[i:i + 4096] = gamma * part / torch.sqrt(part.pow(2).sum(-1, keepdim=True) / c["D"] + EPS)
    if c["out"] != "e4m3":
        return y, None, kept
    parts = y.unflatten(-1, (-1, c["group"] or c["D"]))
    scale = torch.maximum(parts.abs().max(-1).values / 448.0, torch.full((), 2.0 ** -126, dtype=torch.float64, device=y.device))
    return _e4m3(parts / scale.unsqueeze(-1)).flatten(-2), scale, kept


def _exact_norm_bwd(s):
    h, gamma, g = s["h"].double(), s["gamma"].double(), s["dout"].double()
    n = torch.sqrt(h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + EPS)
    along = (gamma * g * h).sum(-1, keepdim=True) / h.shape[-1]
    dx = gamma * g / n - h * along / n.pow(3)
    return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dgamma": (g * h / n).sum(0)}


def _exact_gate(s, a):
    z = a.double() + s["beta"].double()
    sp = torch.logaddexp(z, torch.zeros_like(z))
    return sp, torch.exp(-s["alpha"].double() * sp)


def _exact_gated(s, keep=False):
    """y, the last state and, if kept, the state before each step."""
    B, T, D = s["v"].shape
    lens = [T] * B if s["lens"] is None else s["lens"].tolist()
    h = torch.zeros(B, D, dtype=torch.float64, device=s["v"].device) if s["h0"] is None else s["h0"].double()
    y = torch.zeros(B, T, D, dtype=torch.float64, device=h.device)
    before = torch.zeros_like(y) if keep else None
    on = torch.tensor([[t < n for n in lens] for t in range(T)], device=h.device)[..., None]
    for t in range(T):
        _, f = _exact_gate(s, s["a"][:, t])
        nxt = f * h + (1.0 - f) * s["v"][:, t].double()
        if keep:
            before[:, t] = h
        h = torch.where(on[t], nxt, h)
        y[:, t] = torch.where(on[t], h, torch.zeros_like(h))
    return (y, h, before, on) if keep else (y, h)


def _exact_gated_train(s):
    y, h, before, on = _exact_gated(s, keep=True)
    alpha, dy = s["alpha"].double(), s["dy"].double()
    C = torch.zeros_like(h) if s["dh_T"] is None else s["dh_T"].double()  # f_{t+1} R_{t+1}
    dv, da = torch.zeros_like(y), torch.zeros_like(y)
    dalpha = torch.zeros_like(alpha)
    for t in range(y.shape[1] - 1, -1, -1):
        sp, f = _exact_gate(s, s["a"][:, t])
        z = s["a"][:, t].double() + s["beta"].double()
        R = C + dy[:, t]
        df = R * (before[:, t] - s["v"][:, t].double())
        none = torch.zeros_like(R)
        dv[:, t] = torch.where(on[t], (1.0 - f) * R, none)
        da[:, t] = torch.where(on[t], -alpha * f * df / (1.0 + torch.exp(-z)), none)
        dalpha += torch.where(on[t], -sp * f * df, none).sum(0)
        C = torch.where(on[t], f * R, C)
    return {"y": y, "h_T": h, "dv": dv, "da": da, "dalpha": dalpha, "dbeta": da.sum((0, 1)), "dh0": C}


def _exact_orth(s):
    a, b, c = COEFS
    g = s["g"].double()
    out = torch.empty_like(g)
    for i in range(g.shape[0]):
        X = g[i] if g.shape[1] <= g.shape[2] else g[i].t().contiguous()
        X = X / (X.pow(2).sum().sqrt() + NS_EPS)
        eye = torch.eye(X.shape[0], dtype=torch.float64, device=X.device)
        for _ in range(5):
            A = X @ X.t()
            X = (a * eye + A @ (b * eye + c * A)) @ X
        out[i] = X if g.shape[1] <= g.shape[2] else X.t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gated_step":
        _, f = _exact_gate(s, s["a"])
        return f * s["h0"].double() + (1.0 - f) * s["v"].double()
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "gated": _exact_gated, "gated_train": _exact_gated_train,
            "orth": _exact_orth}[op](s)
