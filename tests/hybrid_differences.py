"""Gradients against differences of the forward formula in 64 bits."""
import numpy as np
import torch

from attn_helpers import f64, gen
from hybrid_helpers import attn_grads
from oracle import attention as oa

STEP = 2.0 ** -14


def attention_differences(got, host, window, scale, dtype, grad):
    """(what, derivative, difference, slack) of L = sum(o d_o) of one sequence along directions that follow
    `got` = (dq, dk, dv) and the oracle's gradients head by head, weighted by token: there a gradient's share of L is the
    sum of its squares, so a part that is too much (along got) or missing (along the oracle's) shows in proportion.

    The slack is the gradients' own error by attn_grads' bounds, at its worst in every element, and the difference's:
    its third-order term, of h^2 of the first times the scores' change, and 2^-40 of sum |o d_o| over the step."""
    q, k, v, d_o = (f64(t) for t in host)
    refs = attn_grads(*host, window, scale, dtype, grad)
    size = float(np.sum(np.abs(oa.attention(q, k, v, window, scale)[0] * d_o)))
    weights = 2 * f64(torch.rand(2, len(q), generator=gen(len(q))))
    for i, name in enumerate(("dq", "dk", "dv")):
        g = f64(got[i]) if torch.is_tensor(got[i]) else got[i]
        for head in range(g.shape[1]):
            for w, along in [(w, a) for w in weights for a in (g, refs[i][0])]:
                u = np.zeros_like(g)
                u[:, head] = w[:, None] * along[:, head]
                u /= np.max(np.abs(u)) + 1e-300
                ends = []
                for h in (STEP, -STEP):
                    x = [q, k, v]
                    x[i] = x[i] + h * u
                    ends.append(float(np.sum(oa.attention(*x, window, scale)[0] * d_o)))
                want, have = (ends[0] - ends[1]) / (2 * STEP), float(np.sum(g * u))
                slack = float(np.sum(refs[i][1] * np.abs(u))) + 64 * STEP ** 2 * abs(want) + 2.0 ** -40 * size / STEP
                yield f"{name} of head {head}", have, want, slack


def check_attention_differences(got, host, window, scale, dtype, grad):
    for what, have, want, slack in attention_differences(got, host, window, scale, dtype, grad):
        assert abs(have - want) <= slack, f"{what}: {have:.6g}, difference {want:.6g}, slack {slack:.3g}"
