"""Pins of the attention oracle: closed forms that need no implementation."""
import math

import numpy as np
import torch

from oracle import attention as oa


def test_e4m3_values_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    vals = codes.double().numpy()
    assert np.array_equal(np.isnan(vals), np.isnan(oa.E4M3))
    ok = ~np.isnan(vals)
    assert np.array_equal(vals[ok], oa.E4M3[ok])
    x = torch.randn(20000, generator=torch.Generator().manual_seed(0)) * torch.logspace(-4, 1.2, 20000)
    x = torch.cat([x, torch.tensor([448.0, -448.0, 0.0, -0.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])])
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oa.e4m3_code(x), want)
    assert oa.e4m3_code(np.array([np.inf, -np.inf, np.nan])).tolist() == [0x7e, 0xfe, 0x7f]


def test_page_scale_is_the_least_power_of_two():
    for top in (448.0, 448.0000001, 447.9, 1.0, 0.875, 0.8750001, 3e38, 1e-20):
        s = oa.page_scale(np.array([top, -top / 3, np.inf, np.nan]))
        assert top <= 448 * s and (top > 448 * s / 2 or s == 2.0 ** -100), top
        assert math.frexp(s)[0] == 0.5
    assert oa.page_scale(np.zeros(3)) == 2.0 ** -100
    assert oa.page_scale(np.array([1e-38])) == 2.0 ** -100


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 5, 3, 64))
    f = 1e4 ** (-np.arange(0, 32, 2) / 32)
    for inter in (False, True):
        a = oa.rotate(x, np.arange(5) + 100, f, inter)
        b = oa.rotate(y, np.arange(5) + 93, f, inter)
        assert np.allclose(np.sum(a * a, -1), np.sum(x * x, -1))
        assert np.array_equal(a[..., 32:], x[..., 32:])
        c = oa.rotate(x, np.arange(5) + 7, f, inter)
        d = oa.rotate(y, np.arange(5), f, inter)
        assert np.allclose(np.sum(a * b, -1), np.sum(c * d, -1))     # depends on 7 alone


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 6, 4, 8))
    o, a, _ = oa.attention(q, k[:, :2], v[:, :2], window=1)
    assert np.allclose(o, np.repeat(v[:, :2], 2, 1))                 # sees itself only
    o, a, _ = oa.attention(0 * q, k, v)
    assert np.allclose(o, np.cumsum(v, 0) / np.arange(1, 7)[:, None, None])
    o1, _, _ = oa.attention(q, k, v)
    o2, _, _ = oa.attention(q[-1:], k, v)
    assert np.allclose(o1[-1:], o2)


def test_paged_cache_holds_what_was_written():
    rng = np.random.default_rng(3)
    c = oa.PagedCache(rng.integers(0, 256, (7, 2, 16, 64)), rng.random((7, 2)), [[3, 0, 5], [1, 6, -1]])
    x = rng.standard_normal((41, 2, 64)) * np.linspace(0.1, 9, 41)[:, None, None]
    for t in range(41):
        c.append(0, t, x[t:t + 1])
    got, there = c.tokens(0, 41)
    assert there.all()
    # one rounding at the final scale, another for each growth (exact but for subnormal codes)
    assert np.all(np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * np.max(np.abs(x)) / 224)
    c.append(1, 30, x[:10])          # its third page is none: dropped
    assert c.tokens(1, 40)[1].sum() == 32
