"""Inputs, error bounds and runners shared by the tests of the attention operators."""
import numpy as np
import torch

from oracle import attention as oa

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inv_freq(rope, theta=1e4, stretch=1.0):
    if rope == 0:
        return None
    return (theta ** (-torch.arange(0, rope, 2, dtype=torch.float64) / rope) / stretch).float()


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def rope_bound(ref, x_ref, factor, dtype):
    """Error bound of a normed and rotated row, by element: half a step of the
    output type, and relative to the length R of the row's largest pair
    (bounded by sqrt(2) max|y|): the norm's sum of squares (19 additions in
    fp32, halved by the root), reciprocal root, two products, the rotation's
    three operations and sine and cosine: 32 half steps of fp32; where the
    result is bf16, the hardware's sine adds up to 2^-18."""
    R = np.sqrt(2.0) * np.max(np.abs(x_ref), -1, keepdims=True) * max(1.0, abs(factor))
    return HALF[dtype] * np.abs(ref) + R * (32 * 2.0 ** -24 + (2.0 ** -18 if dtype == BF else 0.0))


def attn_bound(o, a, reach, n, d, dtype):
    """Error bound of attention by element.  a = sum p |v| / sum p, n keys.
    Scores: d + 4 fp32 roundings relative to sum |q k|, in the exponent, for
    the weight and for the sum of weights; exp2 2^-22; sums of n terms.  bf16:
    weights rounded to bf16 before the product, the output rounded."""
    eps = 2.0 ** -24
    rel = 2 * ((d + 4) * eps * reach * 1.5 + 2.0 ** -22) + 2 * (n + 16) * eps
    if dtype == BF:
        rel += HALF[BF]
    return rel * a + HALF[dtype] * np.abs(o) + 1e-30


def within(x, ref, bound, what=""):
    x = f64(x) if torch.is_tensor(x) else x
    assert np.all(np.isfinite(x)), f"{what}: non-finite values"
    over = np.abs(x - ref) - bound
    assert np.all(over <= 0), f"{what}: off by {np.max(np.abs(x - ref)):.3g}, {np.max(over):.3g} over the bound"


def cache_case(N, Hk, d, P, max_pages, seed, spare=2, lens=None):
    """A pool of random codes (no NaN among those in use) and page tables of distinct pages."""
    g = gen(seed)
    num = N * max_pages + spare
    x = torch.randn(num, Hk, P, d, generator=g)
    scale = 2.0 ** torch.randint(-8, -5, (num, Hk), generator=g).float()
    codes = {}
    for name in "kv":
        y = (torch.randn(num, Hk, P, d, generator=g) / scale[:, :, None, None]).clamp(-448, 448)
        codes[name] = y.to(torch.float8_e4m3fn)
    table = torch.randperm(num, generator=g)[:N * max_pages].view(N, max_pages).to(torch.int32)
    vs = 2.0 ** torch.randint(-8, -5, (num, Hk), generator=g).float()
    del x
    return dict(k=codes["k"], v=codes["v"], ks=scale, vs=vs, table=table)


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def cache_oracles(c):
    return (oa.PagedCache(u8(c["k"]), f64(c["ks"]), c["table"].cpu().numpy()),
            oa.PagedCache(u8(c["v"]), f64(c["vs"]), c["table"].cpu().numpy()))
