"""fp64 CPU oracle for the entry of a layer, the gated recurrence of channels and the orthogonalised update — TEST
INFRASTRUCTURE ONLY (see ``oracle/block.py``): plain numpy loops.

    h = res + x, out = gamma (.) h / sqrt(mean h^2 + eps)
    f_t = exp(-alpha softplus(a_t + beta)), h_t = f_t h_{t-1} + (1 - f_t) v_t
    X = G / (||G|| + eps), X <- a X + (b A + c A A) X with A = X X^T
"""
from __future__ import annotations

import numpy as np

from oracle.block import _f64


# ---------------------------------------------------------------- norm

def norm_fwd(h, gamma, eps):
    h = _f64(h)
    return _f64(gamma) * h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)


def norm_bwd(h, gamma, eps, dout, dh=None):
    """dx and dgamma for the loss sum <dout, out> + <dh, h>."""
    h, p = _f64(h), _f64(gamma) * _f64(dout)
    r = 1.0 / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
    dx = r * p - r ** 3 * h * np.mean(p * h, axis=-1, keepdims=True)
    if dh is not None:
        dx = dx + _f64(dh)
    return dx, np.sum(_f64(dout) * h * r, axis=tuple(range(h.ndim - 1)))


# ---------------------------------------------------------------- gated recurrence

def gate(a, alpha, beta):
    """softplus(z), sigma(z), f and 1 - f (without cancellation), z = a + beta."""
    z = _f64(a) + _f64(beta)
    s = np.maximum(z, 0.0) + np.log1p(np.exp(-np.abs(z)))
    s = np.where(np.isneginf(z), 0.0, s)
    sg = np.where(z < 0, np.exp(-np.abs(z)), 1.0) / (1.0 + np.exp(-np.abs(z)))
    x = np.where(s == 0.0, 0.0, _f64(alpha) * s)
    return s, sg, np.exp(-x), -np.expm1(-x)


def gated_fwd(v, a, alpha, beta, h0=None, lens=None):
    """y [B,T,D], h_T [B,D] and the state before each step."""
    v = _f64(v)
    B, T, D = v.shape
    s, _, f, i = gate(a, alpha, beta)
    h = np.zeros((B, D)) if h0 is None else _f64(h0).copy()
    y, before = np.zeros((B, T, D)), np.zeros((B, T, D))
    lens = np.full(B, T) if lens is None else np.clip(np.asarray(lens), 0, T)
    for t in range(T):
        before[:, t] = h
        on = (t < lens)[:, None] & (s[:, t] != 0.0)
        with np.errstate(invalid="ignore"):
            h = np.where(on, f[:, t] * h + i[:, t] * v[:, t], h)
        y[:, t] = np.where((t < lens)[:, None], h, 0.0)
    return y, h, before


def gated_bwd(v, a, alpha, beta, dy, dh_T=None, h0=None, lens=None):
    """dv, da, dalpha, dbeta, dh0 for the loss sum <dy, y> + <dh_T, h_T>, and the terms of the sums."""
    v, dy, al = _f64(v), _f64(dy), _f64(alpha)
    B, T, D = v.shape
    before = gated_fwd(v, a, alpha, beta, h0, lens)[2]
    s, sg, f, i = gate(a, alpha, beta)
    lens = np.full(B, T) if lens is None else np.clip(np.asarray(lens), 0, T)
    C = np.zeros((B, D)) if dh_T is None else _f64(dh_T).copy()
    dv, da, dl, Rs = (np.zeros((B, T, D)) for _ in range(4))
    for t in range(T - 1, -1, -1):
        live = (t < lens)[:, None]
        R = np.where(live, C + np.where(live, dy[:, t], 0.0), C)
        on = live & (s[:, t] != 0.0)
        C = np.where(on, f[:, t] * R, R)
        with np.errstate(invalid="ignore"):
            G = np.where(on, C * (before[:, t] - v[:, t]), 0.0)
        Rs[:, t] = np.where(live, R, 0.0)
        dv[:, t] = np.where(on, i[:, t] * R, 0.0)
        da[:, t] = -al * sg[:, t] * G
        dl[:, t] = -np.where(on, s[:, t], 0.0) * G
    return {"dv": dv, "da": da, "dalpha": dl.sum((0, 1)), "dbeta": da.sum((0, 1)), "dh0": C}, dl, Rs


# ---------------------------------------------------------------- orthogonalised update

def orthogonalize(g, steps, coefs, eps, noise=None):
    """The definition for one matrix.  noise(x, K): x with the roundings of a product over K terms put in."""
    X = _f64(g)
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / (np.sqrt(np.sum(X * X)) + eps)
    rows = [coefs] * steps if np.ndim(coefs) == 1 else list(coefs)
    put = noise or (lambda x, K: x)
    X = put(X, 0)
    for a, b, c in rows:
        A = put(X @ X.T, X.shape[1])
        B = put(b * A + c * (A @ A), A.shape[0])
        X = put(a * X + put(B @ X, A.shape[0]), 0)
    return X.T if tall else X
