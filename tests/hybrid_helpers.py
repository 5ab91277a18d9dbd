"""Inputs, error bounds and runners shared by the tests of a hybrid's training and
residual operators.  Bounds are per element, from the roundings that the operators'
documentation allows; eps is fp32's half step."""
import math

import numpy as np
import torch

from attn_helpers import BF, F32, HALF, f64, gen, inv_freq, within  # noqa: F401
from oracle import attention as oa
from oracle import hybrid as oh

EPS = 2.0 ** -24


def attn_inputs(T, Hq, Hk, d, dtype, seed, pad=8):
    """q, k, v as column blocks of a projection's rows, d_o dense."""
    g = gen(seed)
    x = torch.randn(T, (Hq + 2 * Hk) * d + pad, generator=g).to(dtype)
    q = x[:, :Hq * d].unflatten(1, (Hq, d))
    k = x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    v = x[:, (Hq + Hk) * d:(Hq + 2 * Hk) * d].unflatten(1, (Hk, d))
    return q, k, v, torch.randn(T, Hq, d, generator=g).to(dtype)


def views(x, Hq, Hk, d):
    """The three column blocks of rows that lie like attn_inputs' projection."""
    return (x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)),
            x[:, (Hq + Hk) * d:(Hq + 2 * Hk) * d].unflatten(1, (Hk, d)))


def attn_grads(q, k, v, d_o, window, scale, dtype, grad=None):
    """The oracle's gradients of one sequence and their bounds.

    Weights p: a score's d + 4 fp32 roundings relative to sum |q k| twice (forward and
    here), its and the statistics' rounding as numbers (of size 1.5 reach + log2 n + 8),
    exp2 and log2 2^-22 each, sums of n terms; bf16: rounded once more for the products.
    D = d_o . o: o's own error (attn_bound's terms and its rounding; bf16: known to 16 bits,
    a step of 2^-15 at most), d products.
    e = p (d_o . v - D): those, and bf16's rounding.  Then sums of n (times the group's
    heads for dk, dv) products, and the output's rounding."""
    q, k, v, d_o = (f64(t) for t in (q, k, v, d_o))
    L, Hq, d = q.shape
    G = Hq // k.shape[1]
    c = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = oh.attention_backward(q, k, v, d_o, window, scale)
    b = HALF[BF] if dtype == BF else 0.0
    out = HALF[grad or dtype]
    bq, bk, bv = np.zeros_like(dq), np.zeros_like(dk), np.zeros_like(dv)
    t, u = np.arange(L)[:, None], np.arange(L)[None]
    seen = (u <= t) & ((u > t - window) if window else True)
    for h in range(Hq):
        kh, vh, qh, gh = k[:, h // G], v[:, h // G], q[:, h], d_o[:, h]
        x = np.where(seen, c * (qh @ kh.T), -np.inf)
        p = np.exp(x - np.max(x, 1, keepdims=True))
        p /= np.sum(p, 1, keepdims=True)
        reach = abs(c) * float(np.max(np.where(seen, np.abs(qh) @ np.abs(kh).T, 0.0)))
        n = float(np.max(np.sum(seen, 1)))
        rel = 4 * ((d + 4) * EPS * 1.5 * reach + EPS * (1.5 * reach + math.log2(n) + 8) + 2.0 ** -22) + 2 * (n + 16) * EPS
        a = p @ np.abs(vh)                                     # sum p |v|
        err_o = (rel + b) * a + (2.0 ** -15 if dtype == BF else HALF[dtype]) * np.abs(p @ vh)
        err_D = np.sum(np.abs(gh) * err_o, 1, keepdims=True) + (d + 8) * EPS * np.sum(np.abs(gh) * a, 1, keepdims=True)
        gp, ga = gh @ vh.T, np.abs(gh) @ np.abs(vh).T
        D = np.sum(p * gp, 1, keepdims=True)
        e = p * (gp - D)
        err_e = (rel + b + 4 * EPS) * np.abs(e) + p * ((d + 8) * EPS * ga + err_D + 4 * EPS * (np.abs(gp) + np.abs(D)))
        terms = (n + 16) * EPS
        bq[:, h] = abs(c) * ((err_e + terms * np.abs(e)) @ np.abs(kh))
        bk[:, h // G] += abs(c) * ((err_e + (L * G + 16) * EPS * np.abs(e)).T @ np.abs(qh))
        bv[:, h // G] += ((rel + b + (L * G + 16) * EPS) * p).T @ np.abs(gh)
    tiny = 1e-30
    return ((dq, bq + out * np.abs(dq) + tiny), (dk, bk + out * np.abs(dk) + tiny), (dv, bv + out * np.abs(dv) + tiny))


def check_attn(got, host, bounds, window, scale, dtype, grad=None, what=""):
    """got: (dq, dk, dv) of packed sequences that lie between `bounds`."""
    q, k, v, d_o = host
    for a, b in zip(bounds, bounds[1:]):
        if b <= a:
            continue
        refs = attn_grads(q[a:b], k[a:b], v[a:b], d_o[a:b], window, scale, dtype, grad)
        for name, x, (ref, bound) in zip(("dq", "dk", "dv"), got, refs):
            within(x[a:b], ref, bound, f"{what} {name} of tokens {a}..{b}")


def norm_grad_bound(x, w, eps, g, err_g, K=96):
    """Bounds of rms_norm_backward's dx (before its rounding) and d_weight, where g is off by err_g.
    Every sum over a row has fewer than K roundings to a term, and so have the products
    behind it; d_weight adds its rows one after another at worst."""
    x, w, g, err_g = (f64(t) if torch.is_tensor(t) else np.asarray(t, np.float64) for t in (x, w, g, err_g))
    rms = np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    n = np.abs(x) / rms
    gw, ew = np.abs(w * g), np.abs(w) * err_g
    dx = (ew + n * np.mean(n * ew, -1, keepdims=True) + K * EPS * (gw + 2 * n * np.mean(n * gw, -1, keepdims=True))) / rms
    rows = x.size // x.shape[-1]
    dw = (n * err_g + (rows + K) * EPS * np.abs(g) * n).reshape(-1, x.shape[-1]).sum(0)
    return dx + 1e-30, dw + 1e-30


def rope_grads(raw, weight, pos, freq, dy, inter, factor, eps, grad):
    """The oracle's (dx, bound), (d_weight, bound) of rows [rows, H, d]: turning back errs like
    turning does (rope_bound), relative to the largest pair."""
    raw, dy = f64(raw), f64(dy)
    f = None if freq is None else f64(freq)
    dx, dw = oh.norm_rope_backward(raw, weight, f64(pos) if pos is not None else np.zeros(len(raw)), f, dy, inter, factor, eps)
    R = np.sqrt(2.0) * np.max(np.abs(dy), -1, keepdims=True) * max(1.0, abs(factor))
    err = R * (8 * EPS + (2.0 ** -18 if grad == BF else 0.0)) * np.ones_like(dy)
    if weight is None:
        return (dx, err + HALF[grad] * np.abs(dx)), (None, None)
    g = oh.norm_rope_backward(raw, None, f64(pos) if pos is not None else np.zeros(len(raw)), f, dy, inter, factor)[0]
    bx, bw = norm_grad_bound(raw, weight, eps, g, err)
    return (dx, bx + HALF[grad] * np.abs(dx)), (dw, bw)
