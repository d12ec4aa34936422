"""fp64 CPU oracle for the selective state space scan and its convolution window — TEST
INFRASTRUCTURE ONLY (see ``oracle/block.py``): plain numpy, step by step, no code shared with the GPU
path.

Per (b, n):  D_t = softplus(a_t + beta),  f_t = exp(-alpha D_t),
             H_t = f_t H_{t-1} + D_t k_t v_t^T,   y_t = H_t^T q_t + w_r (.) v_t,
with query/key j serving the heads j N/G .. (j + 1) N/G - 1, and nothing happening at or past
``lens[b]``.  The backward walks R_t = q_t dy_t^T + f_{t+1} R_{t+1} from dH_T.
"""
from __future__ import annotations

import numpy as np

from oracle.block import _f64, sigmoid, silu, softplus


def _prepared(q, k, v, a, alpha, beta, lens):
    q, k, v, a, alpha, beta = map(_f64, (q, k, v, a, alpha, beta))
    B, T, N = a.shape
    rep = N // q.shape[2]
    q, k = np.repeat(q, rep, axis=2), np.repeat(k, rep, axis=2)
    live = np.ones((B, T, 1))
    if lens is not None:
        live = (np.arange(T)[None, :] < np.clip(lens, 0, T)[:, None]).astype(np.float64)[..., None]
    on = live > 0
    q, k, v = (np.where(on[..., None], x, 0.0) for x in (q, k, v))
    a = np.where(on, a, 0.0)
    D = softplus(a + beta) * live
    f = np.exp(-alpha * D)
    return q, k, v, a, D, f, live


def fwd(q, k, v, a, alpha, beta, w_r, H0=None, lens=None, states=False):
    """y [B,T,N,V], H_T [B,N,K,V] (and the states before each step)."""
    q, k, v, a, D, f, live = _prepared(q, k, v, a, alpha, beta, lens)
    B, T, N, K = q.shape
    V = v.shape[-1]
    w_r = _f64(w_r)
    H = np.zeros((B, N, K, V)) if H0 is None else _f64(H0).copy()
    y = np.zeros((B, T, N, V))
    kept = []
    for t in range(T):
        kept.append(H)
        H = f[:, t, :, None, None] * H + (D[:, t, :, None] * k[:, t])[..., None] * v[:, t, :, None, :]
        y[:, t] = (np.einsum("bnkv,bnk->bnv", H, q[:, t]) + w_r * v[:, t]) * live[:, t, :, None]
    return (y, H, kept) if states else (y, H)


def bwd(q, k, v, a, alpha, beta, w_r, H0, dy, dH_T=None, lens=None, signs=1.0):
    """All gradients of sum <dy, y> + <dH_T, H_T>.  signs = -1 adds the decay's part of da and dalpha
    instead of subtracting it: with absolute values as inputs every gradient is then the sum of the
    magnitudes of its terms."""
    G = q.shape[2]
    _, HT, kept = fwd(q, k, v, a, alpha, beta, w_r, H0, lens, states=True)
    q, k, v, a, D, f, live = _prepared(q, k, v, a, alpha, beta, lens)
    alpha, beta, w_r = map(_f64, (alpha, beta, w_r))
    u = np.where(live[..., None] > 0, _f64(dy), 0.0)
    B, T, N, K = q.shape
    C = np.zeros_like(HT) if dH_T is None else _f64(dH_T).copy()
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    g, kRv = np.zeros_like(D), np.zeros_like(D)
    after = HT
    for t in range(T - 1, -1, -1):
        R = C + q[:, t, :, :, None] * u[:, t, :, None, :]
        Rv = np.einsum("bnkv,bnv->bnk", R, v[:, t])
        dq[:, t] = np.einsum("bnkv,bnv->bnk", after, u[:, t])
        dk[:, t] = D[:, t, :, None] * Rv
        dv[:, t] = D[:, t, :, None] * np.einsum("bnkv,bnk->bnv", R, k[:, t]) + w_r * u[:, t]
        C = f[:, t, :, None, None] * R
        g[:, t] = np.sum(C * kept[t], axis=(2, 3))
        kRv[:, t] = np.sum(k[:, t] * Rv, axis=-1)
        after = kept[t]
    da = (kRv - signs * alpha * g) * sigmoid(a + beta) * live
    return {"dq": dq.reshape(B, T, G, N // G, K).sum(3), "dk": dk.reshape(B, T, G, N // G, K).sum(3), "dv": dv,
            "da": da, "dalpha": -signs * (D * g * live).sum((0, 1)), "dbeta": da.sum((0, 1)),
            "dw_r": (u * v).sum((0, 1)), "dH0": C}


def conv4_silu_window(x, w, bias, win, lens=None):
    """Causal conv4 + SiLU of x [B,T,C] after the three inputs win [B,3,C] (oldest first; None: zeros):
    (u, the window after each sequence's last step)."""
    x, w, bias = map(_f64, (x, w, bias))
    B, T, C = x.shape
    win = np.zeros((B, 3, C)) if win is None else _f64(win)
    u, out = np.zeros((B, T, C)), np.zeros((B, 3, C))
    for b in range(B):
        n = T if lens is None else int(np.clip(lens[b], 0, T))
        seen = np.concatenate([win[b], x[b, :n]])
        for t in range(n):
            pre = np.sum(w.T * seen[t:t + 4], axis=0) + (0.0 if bias is None else bias)
            u[b, t] = silu(pre)
        out[b] = seen[n:n + 3]
    return u, out
