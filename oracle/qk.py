"""fp64 CPU oracle for the norm of queries and keys per head with the position rotation — TEST
INFRASTRUCTURE ONLY (see ``oracle/block.py``): plain numpy.

    xn = gamma (.) x / sqrt(mean x^2 + eps) over a head's features; the pairs (p, p + R/2) of its first R
    features, or (2p, 2p + 1) interleaved, turned by pos * inv_freq[p].
"""
from __future__ import annotations

import numpy as np

from oracle.block import _f64


def pairs(K, R, interleaved):
    """Indices of the first and the second feature of each pair."""
    p = np.arange(R // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + R // 2)


def turn(x, pos, inv_freq, interleaved, sign=1.0):
    """x [B,T,N,K] with its pairs turned by sign * pos * inv_freq."""
    x, inv_freq = _f64(x), _f64(inv_freq)
    a, b = pairs(x.shape[-1], 2 * inv_freq.size, interleaved)
    t = sign * np.asarray(pos, dtype=np.float64)[:, :, None, None] * inv_freq
    out = x.copy()
    out[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
    out[..., b] = x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
    return out


def norm_rope_fwd(x, gamma, pos, inv_freq, eps, interleaved):
    x, gamma = _f64(x), _f64(gamma)
    return turn(gamma * x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps), pos, inv_freq, interleaved)


def norm_rope_bwd(x, gamma, pos, inv_freq, eps, interleaved, dout):
    """dx and dgamma for the loss sum <dout, out>."""
    x, gamma = _f64(x), _f64(gamma)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    gn = turn(dout, pos, inv_freq, interleaved, -1.0)
    p = gamma * gn
    return r * p - r ** 3 * x * np.mean(p * x, axis=-1, keepdims=True), np.sum(gn * x * r, axis=(0, 1, 2))
