"""CPU oracle for a hybrid's training and residual operators -- TEST
INFRASTRUCTURE ONLY (same rule as the rest of ``oracle``).

Plain numpy in float64, straight from the definitions:

  attention_backward   gradients of ``attention.attention`` for one sequence
  rms_norm_backward    gradients of x / sqrt(mean(x^2) + eps) * weight
  norm_rope_backward   gradients of ``attention.norm_rope``
  add_norm             the residual's addition and its RMS norm
  add_norm_backward    its gradients
"""
from __future__ import annotations

import math

import numpy as np

from .attention import rotate
from .layer import _f64


def attention_backward(q, k, v, d_o, window=0, scale=None):
    """One sequence, q, d_o [L, Hq, d], k, v [L, Hk, d].  Returns (dq, dk, dv)."""
    q, k, v, d_o = (_f64(t) for t in (q, k, v, d_o))
    L, Hq, d = q.shape
    G = Hq // k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    t, u = np.arange(L)[:, None], np.arange(L)[None]
    seen = (u <= t) & ((u > t - window) if window else True)
    for h in range(Hq):
        if L == 0:
            continue
        x = np.where(seen, scale * (q[:, h] @ k[:, h // G].T), -np.inf)
        p = np.exp(x - np.max(x, 1, keepdims=True))
        p /= np.sum(p, 1, keepdims=True)
        g = d_o[:, h] @ v[:, h // G].T                       # gradient of p
        e = p * (g - np.sum(p * g, 1, keepdims=True))        # gradient of x
        dq[:, h] = scale * (e @ k[:, h // G])
        dk[:, h // G] += scale * (e.T @ q[:, h])
        dv[:, h // G] += p.T @ d_o[:, h]
    return dq, dk, dv


def rms_norm_backward(x, weight, eps, dy):
    """(dx, d_weight summed over all rows); weight None: 1."""
    x, dy = _f64(x), _f64(dy)
    w = np.ones(x.shape[-1]) if weight is None else _f64(weight)
    rms = np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n = x / rms
    dx = (w * dy - n * np.mean(n * w * dy, -1, keepdims=True)) / rms
    return dx, np.sum((dy * n).reshape(-1, x.shape[-1]), 0)


def norm_rope_backward(x, weight, positions, inv_freq, dy, interleaved=False, factor=1.0, eps=1e-6):
    """(dx, d_weight or None without a norm).  A rotation's transpose turns back."""
    g = rotate(dy, -_f64(positions) if inv_freq is not None else positions, inv_freq, interleaved, factor)
    if weight is None:
        return g, None
    return rms_norm_backward(x, weight, eps, g)


def add_norm(x, res, weight, eps):
    """(y, r)."""
    r = _f64(x) + (0.0 if res is None else _f64(res))
    y = r / np.sqrt(np.mean(r * r, -1, keepdims=True) + eps)
    return (y if weight is None else y * _f64(weight)), r


def add_norm_backward(dy, r, weight, d_res_out, eps):
    """(d_r, d_weight)."""
    dr, dw = rms_norm_backward(r, weight, eps, dy)
    return (dr if d_res_out is None else dr + _f64(d_res_out)), dw
