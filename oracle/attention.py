"""CPU oracle for the softmax-attention layers of a hybrid -- TEST
INFRASTRUCTURE ONLY (same rule as the rest of ``oracle``).

Plain numpy in float64, straight from the definitions:

  rms_norm      y = x / sqrt(mean(x^2) + eps) * weight
  rotate        channel pairs turned by pos * inv_freq, half or interleaved
  attention     causal softmax attention of one sequence, full or windowed
  e4m3          values and rounding of OCP e4m3, by enumeration of its codes
  PagedCache    a paged cache of such codes, written token by token
"""
from __future__ import annotations

import math

import numpy as np

from .layer import _f64


def rms_norm(x, weight, eps):
    x = _f64(x)
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * _f64(weight)


def rotate(x, positions, inv_freq, interleaved, factor=1.0):
    """x [rows, H, d]; positions [rows]; the first 2 len(inv_freq) channels turn."""
    x = _f64(x).copy()
    if inv_freq is None:
        return x
    half = len(inv_freq)
    t = np.asarray(_f64(positions))[:, None] * _f64(inv_freq)
    c, s = (np.cos(t) * factor)[:, None], (np.sin(t) * factor)[:, None]
    ia = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    ib = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def norm_rope(x, weight, positions, inv_freq, interleaved=False, factor=1.0, eps=1e-6):
    x = _f64(x)
    return rotate(x if weight is None else rms_norm(x, weight, eps), positions, inv_freq,
                  interleaved, factor)


def attention(q, k, v, window=0, scale=None, causal_from=None):
    """One sequence: q [Lq, Hq, d] are its last Lq tokens, k, v [L, Hk, d].
    Returns (o, a, reach): o [Lq, Hq, d]; a the same sum over |v|; reach the
    largest scale * sum_i |q_i k_i| over the seen pairs (for error bounds).  A
    query that sees no key gives 0."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    Lq, Hq, d = q.shape
    L, Hk = k.shape[0], k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, a = np.zeros_like(q), np.zeros_like(q)
    reach = 0.0
    t = np.arange(L - Lq, L)[:, None]
    u = np.arange(L)[None]
    seen = (u <= t) & ((u > t - window) if window else True)
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // Hk)], v[:, h // (Hq // Hk)]
        if L == 0 or Lq == 0:
            continue
        x = np.where(seen, scale * (q[:, h] @ kh.T), -np.inf)
        top = np.max(x, 1, keepdims=True)
        p = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        z = np.sum(p, 1, keepdims=True)
        p = np.divide(p, z, out=np.zeros_like(p), where=z > 0)
        o[:, h], a[:, h] = p @ vh, p @ np.abs(vh)
        reach = max(reach, float(np.max(np.where(seen, abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T), 0.0))))
    return o, a, reach


def _e4m3_values():
    vals = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.nan if (c & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        vals[c] = -x if c & 128 else x
    return vals


E4M3 = _e4m3_values()
_POS = E4M3[:127]      # 0 .. 448, rising


def e4m3_code(x):
    """Codes of x rounded to the nearest value, ties to the even code; beyond
    448 the largest; NaN 0x7f (either sign)."""
    x = _f64(x)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    i = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo, hi = a - _POS[i - 1], _POS[i] - a
    c = np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i).astype(np.uint8)
    return np.where(np.isnan(x), 127, np.where(np.signbit(x), c | 128, c)).astype(np.uint8)


def page_scale(x):
    """Least 2^e >= max|x| / 448 over the finite values, e >= -100."""
    a = np.abs(_f64(x))
    top = float(np.max(np.where(np.isfinite(a), a, 0.0), initial=0.0))
    if top == 0.0:
        return 2.0 ** -100
    m, e = math.frexp(top / 448.0)        # top / 448 = m 2^e, m in [1/2, 1)
    return 2.0 ** max(-100, e - 1 if m == 0.5 else e)


class PagedCache:
    """Codes and scales of one of the two caches, written sequence by sequence."""

    def __init__(self, codes, scale, page_table):
        self.codes = np.array(codes, np.uint8)
        self.scale = np.array(scale, np.float64)
        self.table = np.array(page_table)
        self.P = self.codes.shape[2]

    def append(self, n, held, x):
        """x [tokens, H, d] behind `held` tokens of sequence n."""
        cap = self.table.shape[1] * self.P
        held = min(max(int(held), 0), cap)
        x = _f64(x)[:cap - held]
        t = 0
        while t < len(x):
            pos = held + t
            row = pos % self.P
            m = min(self.P - row, len(x) - t)
            page = int(self.table[n, pos // self.P])
            if 0 <= page < len(self.codes):
                for h in range(x.shape[1]):
                    new = x[t:t + m, h]
                    sc = page_scale(new)
                    old = self.scale[page, h]
                    if row:
                        sc = max(sc, old)
                        if sc > old:
                            self.codes[page, h, :row] = e4m3_code(E4M3[self.codes[page, h, :row]] * (old / sc))
                    self.scale[page, h] = sc
                    self.codes[page, h, row:row + m] = e4m3_code(new / sc)
            t += m

    def tokens(self, n, length):
        """[length, H, d] values of sequence n's tokens, and which lie on a page."""
        cap = self.table.shape[1] * self.P
        length = min(max(int(length), 0), cap)
        H, d = self.codes.shape[1], self.codes.shape[3]
        out, there = np.zeros((length, H, d)), np.zeros(length, bool)
        for t in range(length):
            page = int(self.table[n, t // self.P])
            if 0 <= page < len(self.codes):
                out[t] = E4M3[self.codes[page, :, t % self.P]] * self.scale[page][:, None]
                there[t] = True
        return out, there
