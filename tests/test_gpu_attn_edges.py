"""GPU parity of the attention operators at the edges of their documented
ranges, against the definitions in 64 bits."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from attn_helpers import BF, F32, attn_bound, cache_case, cache_oracles, f64, gen, inv_freq, rope_bound, u8, within
from helpers import announce
from oracle import attention as oa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import gated_delta_rule_gdn_amd as gdn  # noqa: E402
import test_gpu_attn as ta  # noqa: E402


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window,lens,width", [(12, [37, 28, 44], 3), (1000, [1025, 1080, 1016], 80)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_decode_scales_of_pages_before_the_window(window, lens, width, bad, dtype):
    """Pages that lie wholly before the window have no part in the output, whatever their codes and scales,
    also where the window begins in the second half of a step of 32 tokens (pages of 16; caches that one
    workgroup takes whole, and joined ones)."""
    announce(f"decode before the window window={window} bad={bad} {dtype}")
    P, d = 16, 128
    c = cache_case(len(lens), 2, d, P, width, seed=41)
    for n, L in enumerate(lens):
        for page in c["table"][n, :(L - window) // P].long():
            for x in "kv":
                c[x].view(torch.uint8)[page] = 0x7f
                c[x + "s"][page] = bad
    q = torch.randn(len(lens), 6, d, generator=gen(7)).to(dtype)
    g = ta.to_dev(c)
    o = gdn.gdn_attn_decode(q.cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], torch.tensor(lens).cuda(), window=window)
    torch.cuda.synchronize()
    ta.check_decode(o, q, c, lens, window, None, dtype, P, d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [2 ** 63 - 32, 2 ** 63 - 1])
def test_windows_of_any_size(window, dtype):
    """A window beyond every token is none, bit for bit in decode."""
    announce(f"window {window} {dtype}")
    P, d, lens = 16, 128, [1, 37, 2000]
    c = cache_case(len(lens), 2, d, P, 125, seed=5)
    g = ta.to_dev(c)
    q = torch.randn(len(lens), 4, d, generator=gen(2)).to(dtype).cuda()
    run = lambda w: gdn.gdn_attn_decode(q, g["k"], g["v"], g["ks"], g["vs"], g["table"], torch.tensor(lens).cuda(), window=w)  # noqa: E731
    assert torch.equal(run(window), run(0))
    host, dv = ta.prefill_case(500, 4, 2, d, dtype, 9)
    cu = torch.tensor([0, 70, 500])
    for offsets in (None, cu.cuda()):
        o = gdn.gdn_attn_prefill(*dv, cu_seqlens=offsets, window=window)
        ta.check_prefill(o, host, [0, 500] if offsets is None else cu.tolist(), 0, None, dtype, d)


def spin(x, pos, f, inter):
    """x [rows, H, d] rotated by pos * f, each angle reduced in rational numbers."""
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    turn = np.array([[float(Fraction(int(p)) * Fraction(float(w)) / two_pi % 1) for w in f] for p in pos])
    c, s = np.cos(2 * np.pi * turn)[:, None], np.sin(2 * np.pi * turn)[:, None]
    y, half = f64(x).copy(), len(f)
    ia = slice(0, 2 * half, 2) if inter else slice(0, half)
    ib = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
    a, b = f64(x)[..., ia], f64(x)[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("grow", [1.0, 64.0, 1e4])
def test_norm_rope_angles_at_every_position(grow, inter, dtype):
    """The angle's error is 2^-25 of a turn at near and far positions alike, and for frequencies above 1 too
    (products up to 2^53 times 1, or 2^24 times 10^4): the bound has no term that grows with the position."""
    announce(f"norm_rope angles grow={grow} inter={inter} {dtype}")
    d, most = 64, 53 if grow == 1.0 else 40
    pos = [0, 1, -1, 4097, (1 << 24) - 1, 1 << 24, -(1 << 24), (1 << 24) + 1, 12345678, (1 << 31) + 5, -(1 << 33) - 7]
    pos += [(1 << e) - 3 * e for e in range(25, most + 1, 2)] + [(1 << most) - 1]
    f = inv_freq(d) * grow
    x = torch.randn(len(pos), 2, d, generator=gen(3)).to(dtype)
    q, _ = gdn.gdn_qk_norm_rope(x.cuda(), positions=torch.tensor(pos).cuda(), inv_freq=f.cuda(), interleaved=inter)
    torch.cuda.synchronize()
    ref = spin(x, pos, f.tolist(), inter)
    within(q, ref, rope_bound(ref, f64(x), 1.0, dtype), "angles")


def ties(score, v, window):
    """Attention where scores are equal or far apart: the mean of the values of the largest; and of |v|."""
    T = len(v)
    o, a = np.zeros((T,) + v.shape[1:]), np.zeros((T,) + v.shape[1:])
    for t in range(T):
        lo = max(0, t + 1 - window) if window else 0
        top = score[lo:t + 1] == score[lo:t + 1].max()
        o[t], a[t] = v[lo:t + 1][top].mean(0), np.abs(v[lo:t + 1][top]).mean(0)
    return o, a


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,window,d", [(1, 0, 128), (40, 0, 64), (300, 0, 128), (300, 50, 64), (600, 0, 128)])
@pytest.mark.parametrize("size", [8, 14, 20, 56])
def test_prefill_scores_of_any_finite_size(size, T, window, d, dtype):
    """Scores around +-2^(2 size): equal ones share the weight, the others are too far apart for any. The
    products are exact, so equal scores are equal in the kernels too, and the bound has no term for their error."""
    announce(f"prefill scores 2^{2 * size} T={T} window={window} d={d} {dtype}")
    g = gen(T + size)
    c = (1 + torch.randint(0, 8, (T,), generator=g) / 8) * (torch.randint(0, 2, (T,), generator=g) * 2 - 1)
    c[0] = -c[0].abs()
    q, k = torch.zeros(T, 2, d), torch.zeros(T, 1, d)
    q[..., 3] = 2.0 ** size
    k[:, 0, 3] = c * 2.0 ** size
    v = torch.randn(T, 1, d, generator=g).to(dtype)
    for scale in (0.125, -0.125):
        o = gdn.gdn_attn_prefill(q.to(dtype).cuda(), k.to(dtype).cuda(), v.cuda(), window=window, scale=scale)
        ro, ra = ties(np.sign(scale) * f64(c), f64(v), window)
        ro, ra = np.repeat(ro, 2, 1), np.repeat(ra, 2, 1)
        within(o, ro, attn_bound(ro, ra, 0.0, T, d, dtype), f"scale {scale}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [8, 160])
@pytest.mark.parametrize("size", [8, 14, 20, 56])
def test_decode_scores_of_any_finite_size(size, width, dtype):
    """The same over a cache that one workgroup takes whole and over a joined one."""
    announce(f"decode scores 2^{2 * size} width={width} {dtype}")
    P, d, Hk = 16, 128, 2
    lens = [1, 2, 33, width * P - 5, 0]
    c = cache_case(len(lens), Hk, d, P, width, seed=size)
    g = gen(size)
    code = (1 + torch.randint(0, 8, c["k"].shape[:3], generator=g) / 8) * (torch.randint(0, 2, c["k"].shape[:3], generator=g) * 2 - 1)
    code = -code.abs() if size == 56 else code
    k = torch.zeros(c["k"].shape)
    k[..., 5] = code
    c["k"], c["ks"] = k.to(torch.float8_e4m3fn), torch.full_like(c["ks"], 2.0 ** size)
    _, ov = cache_oracles(c)
    q = torch.zeros(len(lens), 4, d)
    q[..., 5] = 2.0 ** size
    e = ta.to_dev(c)
    for scale in (0.125, -0.125):
        o = gdn.gdn_attn_decode(q.to(dtype).cuda(), e["k"], e["v"], e["ks"], e["vs"], e["table"],
                                torch.tensor(lens).cuda(), scale=scale)
        for n, L in enumerate(lens):
            if L == 0:
                assert bool((o[n] == 0).all())
                continue
            v, _ = ov.tokens(n, L)
            at = [(int(c["table"][n, t // P]), t % P) for t in range(L)]
            for h in range(4):
                s = np.sign(scale) * np.array([float(code[p, h // 2, r]) for p, r in at])
                top = s == s.max()
                ro, ra = v[top, h // 2].mean(0), np.abs(v[top, h // 2]).mean(0)
                within(o[n, h], ro, attn_bound(ro, ra, 0.0, L, d, dtype), f"sequence {n} head {h} scale {scale}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,d,rope", [(16, 64, 32), (128, 128, 96), (64, 64, 64)])
def test_append_scaled_rotation_and_large_eps(P, d, rope, dtype):
    """rope_scale and eps reach the cached keys as they reach the queries."""
    announce(f"append rope_scale eps P={P} d={d} rope={rope} {dtype}")
    Hk, held, new = 2, 5, P + 9
    c = cache_case(1, Hk, d, P, 3, seed=P)
    ok, ov = cache_oracles(c)
    g = ta.to_dev(c)
    f, w = inv_freq(rope), 1 + 0.1 * torch.randn(d, generator=gen(2))
    x = torch.randn(2, new, Hk, d, generator=gen(6)).to(dtype)
    gdn.gdn_kv_append(x[0].cuda(), x[1].cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], torch.tensor([held]).cuda(),
                      inv_freq=f.cuda(), k_weight=w.cuda(), rope_scale=1.25, eps=3.0)
    torch.cuda.synchronize()
    ok.append(0, held, oa.norm_rope(x[0], w, held + np.arange(new), f.numpy(), False, 1.25, 3.0))
    ov.append(0, held, x[1])
    ta.check_cache(g, ok, ov, "scaled", k_bound=0.01)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,d", [(128, 128), (128, 64), (64, 128), (16, 64)])
def test_append_infinities_in_one_waves_rows(P, d, dtype):
    """Infinities and NaN among some rows of a page that several waves write, behind older tokens that are
    rounded again: they move no scale, saturate, and stay NaN."""
    announce(f"append infinities P={P} d={d} {dtype}")
    Hk, held = 2, P // 4 + 3
    c = cache_case(2, Hk, d, P, 2, seed=P + d)
    ok, ov = cache_oracles(c)
    g = ta.to_dev(c)
    new = P - held
    x = 30 * torch.randn(2, 2, new, Hk, d, generator=gen(8))     # larger than the page's older values: its scale grows
    x[:, 0, new // 2, :, 3], x[:, 0, new // 2, :, 9], x[:, 0, new // 2, :, 11] = math.inf, -math.inf, math.nan
    x[:, 1, -1, 0] = math.inf
    x = x.to(dtype)
    gdn.gdn_kv_append(x[0].flatten(0, 1).cuda(), x[1].flatten(0, 1).cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"],
                      torch.full((2,), held).cuda())
    torch.cuda.synchronize()
    for n in range(2):
        ok.append(n, held, x[0, n])
        ov.append(n, held, x[1, n])
    for name, want in (("k", ok), ("v", ov)):
        assert np.array_equal(f64(g[name + "s"]), want.scale), name
        got, ref = oa.E4M3[u8(g[name])], oa.E4M3[want.codes]
        assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)]), name
    assert bool((f64(g["vs"])[c["table"][:, 0].numpy()] > f64(c["vs"])[c["table"][:, 0].numpy()]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [10, 160])
def test_decode_query_that_is_not_finite(width, dtype):
    """A NaN or infinite query head spoils its own output only, in a group whose heads share every product,
    over a cache that one workgroup takes whole and over a joined one."""
    announce(f"decode NaN query width={width} {dtype}")
    P, d = 16, 128
    lens = [1, 100, width * P]
    c = cache_case(len(lens), 2, d, P, width, seed=3)
    g = ta.to_dev(c)
    q = torch.randn(len(lens), 10, d, generator=gen(5)).to(dtype)
    run = lambda x: gdn.gdn_attn_decode(x.cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], torch.tensor(lens).cuda())  # noqa: E731
    want = run(q)
    ta.check_decode(want, q, c, lens, 0, None, dtype, P, d)
    for n, h, bad in ((0, 0, math.nan), (1, 7, math.inf), (2, 4, math.nan), (2, 9, -math.inf)):
        w = q.clone()
        w[n, h, 17] = bad
        o = run(w)
        o[n, h] = want[n, h]
        assert torch.equal(o, want), (n, h, bad)


@pytest.mark.parametrize("T,Hq,Hk,d,window", [(2500, 2, 1, 128, 0), (2500, 2, 2, 64, 0), (2500, 2, 1, 128, 700), (2500, 12, 2, 64, 0)])
def test_prefill_long_fp32(T, Hq, Hk, d, window):
    """fp32 prompts of many key tiles."""
    announce(f"prefill fp32 T={T} Hq={Hq} Hk={Hk} d={d} window={window}")
    host, dv = ta.prefill_case(T, Hq, Hk, d, F32, T + d)
    o = gdn.gdn_attn_prefill(*dv, window=window)
    torch.cuda.synchronize()
    ta.check_prefill(o, host, [0, T], window, None, F32, d)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_of_a_model_gone_nan(dtype):
    """Values that are all NaN give NaN, in a time of the same order: every wave computes its rows again
    for them, but no row walks on through its keys once all of its columns are NaN."""
    announce(f"prefill all NaN {dtype}")
    T = 8192
    q, k, v = torch.randn(T, 8, 64, generator=gen(1)), torch.randn(T, 2, 64, generator=gen(2)), torch.randn(T, 2, 64, generator=gen(3))
    q, k, v = [t.to(dtype).cuda() for t in (q, k, v)]
    nan = torch.full_like(v, math.nan)
    o = torch.empty_like(q)

    def best(values):
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            gdn.gdn_attn_prefill(q, k, values, o=o)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    clean = best(v)
    slow = best(nan)
    assert bool(o.isnan().all())
    assert slow < 20 * clean, (slow, clean)
    late = v.clone()
    late[T - 100] = math.nan                 # the rows before it see none
    gdn.gdn_attn_prefill(q, k, late, o=o)
    assert bool(o[:T - 100].isfinite().all()) and bool(o[T - 100:].isnan().all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 600])
def test_prefill_large_scores_among_many_tiles(window, dtype):
    """As above where the query tiles fill the chip, among ordinary rows: huge scores in some heads only."""
    announce(f"prefill large scores, many tiles, window={window} {dtype}")
    T, Hq, d = 1133, 32, 128
    host, _ = ta.prefill_case(T, Hq, 8, d, dtype, 3)
    q, k, v = [t.clone().contiguous() for t in host]
    c = (1 + torch.randint(0, 8, (T,), generator=gen(4)) / 8) * (torch.randint(0, 2, (T,), generator=gen(5)) * 2 - 1)
    q[:, 8:12], k[:, 2] = 0, 0
    q[:, 8:12, 3] = 2.0 ** 20
    k[:, 2, 3] = c * 2.0 ** 20
    o = gdn.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), window=window, scale=0.125)
    ro, ra = ties(f64(c), f64(v[:, 2:3]), window)
    ro, ra = np.repeat(ro, 4, 1), np.repeat(ra, 4, 1)
    within(o[:, 8:12], ro, attn_bound(ro, ra, 0.0, T, d, dtype), "huge scores")
    rest = [h for h in range(Hq) if not 8 <= h < 12]
    kr = [h for h in range(8) if h != 2]
    ro, ra, reach = oa.attention(q[:, rest], k[:, kr], v[:, kr], window, 0.125)
    within(o[:, rest], ro, attn_bound(ro, ra, reach, T, d, dtype), "ordinary heads")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,T,Hq,Hk,window", [(300, 3, 4, 2, 0), (257, 1, 3, 3, 0), (64, 33, 8, 1, 5), (40, 129, 2, 2, 64)])
def test_prefill_many_equal_prompts(N, T, Hq, Hk, window, dtype):
    announce(f"prefill many equal N={N} T={T} Hq={Hq} Hk={Hk} window={window} {dtype}")
    host, dv = ta.prefill_case(N * T, Hq, Hk, 64, dtype, N + T)
    o = gdn.gdn_attn_prefill(*dv, N=N, window=window)
    torch.cuda.synchronize()
    ta.check_prefill(o, host, list(range(0, N * T + 1, T)), window, None, dtype, 64)


def test_default_stream_given_as_a_handle():
    """Stream 0, as a number: the default stream, for calls that allocate too."""
    announce("stream 0")
    c = cache_case(2, 2, 64, 16, 90, seed=6)
    g = ta.to_dev(c)
    q = torch.randn(2, 4, 64, generator=gen(1)).to(BF).cuda()
    lens = torch.tensor([1400, 3]).cuda()
    args = (q, g["k"], g["v"], g["ks"], g["vs"], g["table"], lens)
    want = gdn.gdn_attn_decode(*args)
    assert torch.equal(gdn.gdn_attn_decode(*args, stream=0), want)
    assert torch.equal(gdn.gdn_attn_decode(*args, stream=torch.cuda.current_stream()), want)
    x = torch.randn(5, 2, 64, generator=gen(2)).cuda()
    assert torch.equal(gdn.gdn_qk_norm_rope(x, stream=0)[0], x)
