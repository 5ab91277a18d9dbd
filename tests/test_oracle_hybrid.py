"""Pins of the oracle of a hybrid's training operators: every gradient against
central differences of the forward oracle, and closed forms."""
import numpy as np
import pytest

from oracle import attention as oa
from oracle import hybrid as oh

H = 1e-6


def differences(f, x):
    """d f / d x by central differences (f a number)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + H
        up = f()
        x[i] = old - H
        g[i] = (up - f()) / (2 * H)
        x[i] = old
    return g


def close(a, b):
    # central differences: h^2 / 6 of the third derivative and 2^-52 / h of the value
    assert np.max(np.abs(a - b)) <= 1e-7 * max(1.0, np.max(np.abs(b))), np.max(np.abs(a - b))


@pytest.mark.parametrize("L,Hq,Hk,d,window,scale", [(5, 2, 1, 4, 0, None), (7, 3, 3, 4, 3, 0.7), (4, 4, 2, 8, 1, -0.5),
                                                    (1, 2, 2, 4, 0, None)])
def test_attention_backward_is_the_derivative(L, Hq, Hk, d, window, scale):
    rng = np.random.default_rng(L)
    q, k, v = rng.standard_normal((L, Hq, d)), rng.standard_normal((L, Hk, d)), rng.standard_normal((L, Hk, d))
    g = rng.standard_normal((L, Hq, d))
    f = lambda: float(np.sum(oa.attention(q, k, v, window, scale)[0] * g))  # noqa: E731
    for got, x in zip(oh.attention_backward(q, k, v, g, window, scale), (q, k, v)):
        close(got, differences(f, x))


def test_attention_backward_of_one_seen_token():
    """A window of one: o = v, so dv is the sum over the group and nothing reaches q and k."""
    rng = np.random.default_rng(0)
    q, g = rng.standard_normal((2, 6, 4, 8))
    k, v = rng.standard_normal((2, 6, 2, 8))
    dq, dk, dv = oh.attention_backward(q, k, v, g, window=1)
    assert np.all(np.abs(dq) < 1e-15) and np.all(np.abs(dk) < 1e-15)
    assert np.allclose(dv, g.reshape(6, 2, 2, 8).sum(2), atol=1e-15)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_norm_rope_backward_is_the_derivative(inter, normed):
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((2, 3, 2, 16))
    w = 1 + 0.3 * rng.standard_normal(16) if normed else None
    pos, freq = np.array([5, 0, 1000]), np.array([1.0, 0.3, 0.01])
    f = lambda: float(np.sum(oa.norm_rope(x, w, pos, freq, inter, 1.3, 1e-3) * g))  # noqa: E731
    dx, dw = oh.norm_rope_backward(x, w, pos, freq, g, inter, 1.3, 1e-3)
    close(dx, differences(f, x))
    if normed:
        close(dw, differences(f, w))


@pytest.mark.parametrize("with_res", [False, True])
def test_add_norm_backward_is_the_derivative(with_res):
    rng = np.random.default_rng(4)
    x, res, gy, gr = rng.standard_normal((4, 3, 16))
    w = 1 + 0.3 * rng.standard_normal(16)

    def f():
        y, r = oh.add_norm(x, res if with_res else None, w, 1e-3)
        return float(np.sum(y * gy) + np.sum(r * gr))

    _, r = oh.add_norm(x, res if with_res else None, w, 1e-3)
    dr, dw = oh.add_norm_backward(gy, r, w, gr, 1e-3)
    close(dr, differences(f, x))
    close(dw, differences(f, w))
    if with_res:
        close(dr, differences(f, res))


def test_a_norm_does_not_feel_its_rows_length():
    """With eps 0, y is the same for 2 r: the gradient has no part along r, and halves."""
    rng = np.random.default_rng(5)
    r, g = rng.standard_normal((2, 4, 32))
    a, dw = oh.add_norm_backward(g, r, None, None, 0.0)
    b, dw2 = oh.add_norm_backward(g, 2 * r, None, None, 0.0)
    assert np.max(np.abs(np.sum(a * r, -1))) < 1e-13
    assert np.allclose(a, 2 * b, atol=1e-15) and np.allclose(dw, dw2, atol=1e-14)
