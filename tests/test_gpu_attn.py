"""GPU parity of the attention operators (gdn_qk_norm_rope, gdn_kv_append,
gdn_attn_prefill, gdn_attn_decode) against the float64 oracle
(``oracle.attention``), through the C ABI.  Bounds are per element and derived
in attn_helpers."""
import math

import numpy as np
import pytest
import torch

from attn_helpers import (BF, F32, attn_bound, cache_case, cache_oracles, f64, gen, inv_freq, rope_bound, u8, within)
from helpers import announce
from oracle import attention as oa

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import gated_delta_rule_gdn_amd as gdn  # noqa: E402


def dev(x):
    return None if x is None else x.cuda()


# ----------------------------------------------------------------------------
# norms and rotation
# ----------------------------------------------------------------------------

def rope_case(rows, Hq, Hk, d, dtype, seed, pad=24, far=1 << 17):
    g = gen(seed)
    x = (1.5 * torch.randn(rows, (Hq + Hk) * d + pad, generator=g)).to(dtype)
    return dict(x=x, qw=1 + 0.1 * torch.randn(d, generator=g), kw=1 + 0.1 * torch.randn(d, generator=g),
                pos=torch.randint(far, (rows,), generator=g))


def split(x, Hq, Hk, d):
    return x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,d,rope", [
    (1, 16, 2, 128, 64), (33, 5, 1, 128, 128), (70, 4, 3, 64, 64), (257, 1, 1, 64, 32), (3, 8, 8, 128, 96),
    (65, 9, 2, 64, 16), (129, 2, 1, 128, 0)])
def test_norm_rope(rows, Hq, Hk, d, rope, inter, dtype):
    announce(f"norm_rope rows={rows} Hq={Hq} Hk={Hk} d={d} rope={rope} inter={inter} {dtype}")
    c = rope_case(rows, Hq, Hk, d, dtype, 100 + rows)
    f = inv_freq(rope)
    q_raw, k_raw = split(dev(c["x"]), Hq, Hk, d)
    q, k = gdn.gdn_qk_norm_rope(q_raw, k_raw, positions=dev(c["pos"]) if rope else None, inv_freq=dev(f),
                                q_weight=dev(c["qw"]), k_weight=dev(c["kw"]), interleaved=inter, rope_scale=1.25)
    torch.cuda.synchronize()
    for got, raw, w in ((q, q_raw, c["qw"]), (k, k_raw, c["kw"])):
        y = oa.rms_norm(raw.cpu(), w, 1e-6)
        ref = oa.rotate(y, c["pos"], None if f is None else f.numpy(), inter, 1.25)
        within(got, ref, rope_bound(ref, y, 1.25, dtype), "norm_rope")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_rope_one_operand_no_weights_in_place(dtype):
    """Queries alone and keys alone, without a norm, in place on a dense tensor; large eps with a norm."""
    announce(f"norm_rope single operands {dtype}")
    c = rope_case(40, 3, 0, 128, dtype, 7, pad=0)
    f = inv_freq(128)
    x = c["x"].view(40, 3, 128)
    ref = oa.rotate(x, c["pos"], f.numpy(), False)
    for as_q in (True, False):
        y = x.cuda()
        kw = dict(positions=dev(c["pos"]), inv_freq=dev(f))
        out = gdn.gdn_qk_norm_rope(y, q=y, **kw) if as_q else gdn.gdn_qk_norm_rope(None, y, k=y, **kw)
        assert out[0 if as_q else 1].data_ptr() == y.data_ptr() and out[1 if as_q else 0] is None
        within(y, ref, rope_bound(ref, f64(x), 1.0, dtype), "in place")
    q, _ = gdn.gdn_qk_norm_rope(dev(x), q_weight=dev(c["qw"]), eps=3.0)
    ref = oa.rms_norm(x, c["qw"], 3.0)
    within(q, ref, rope_bound(ref, ref, 1.0, dtype), "large eps")


def test_norm_rope_far_positions_keep_their_angle():
    """Positions up to 2^40: an angle formed in fp32 would be off by turns."""
    announce("norm_rope far positions")
    c = rope_case(64, 2, 1, 64, F32, 9)
    pos = torch.cat([torch.randint(1 << 40, (60,), generator=gen(1)), torch.tensor([0, 1, (1 << 31) + 5, 1 << 32])])
    f = inv_freq(64, theta=1e6, stretch=8.0)
    q_raw, k_raw = split(dev(c["x"]), 2, 1, 64)
    q, k = gdn.gdn_qk_norm_rope(q_raw, k_raw, positions=dev(pos), inv_freq=dev(f))
    for got, raw in ((q, q_raw), (k, k_raw)):
        # the angle's own rounding in 64 bits: pos * freq * 2^-53, on both sides
        ref = oa.rotate(raw.cpu(), pos, f.numpy(), False)
        bound = rope_bound(ref, f64(raw), 1.0, F32) + 2.0 ** 40 * 2.0 ** -51 * np.max(np.abs(f64(raw)), -1, keepdims=True)
        within(got, ref, bound, "far")


def test_norm_rope_zero_rows_and_zero_vectors():
    announce("norm_rope zeros")
    q, k = gdn.gdn_qk_norm_rope(torch.empty(0, 4, 64, dtype=BF, device="cuda"), torch.empty(0, 2, 64, dtype=BF, device="cuda"))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    w = torch.ones(64, device="cuda")
    q, _ = gdn.gdn_qk_norm_rope(torch.zeros(5, 4, 64, device="cuda"), q_weight=w)
    assert bool((q == 0).all())


# ----------------------------------------------------------------------------
# cache append
# ----------------------------------------------------------------------------

def to_dev(c):
    return {n: t.cuda() for n, t in c.items()}


def check_cache(c, ok, ov, what, k_bound=None):
    """Values' codes and both scales bit for bit; keys' codes too, but where rounding may fall either way."""
    assert np.array_equal(f64(c["vs"]), ov.scale), what
    assert np.array_equal(f64(c["ks"]), ok.scale), what
    v, vr = u8(c["v"]), ov.codes
    nan = np.isnan(oa.E4M3[vr])
    assert np.array_equal(v[~nan], vr[~nan]) and np.isnan(oa.E4M3[v[nan]]).all(), what
    k, kr = oa.E4M3[u8(c["k"])], oa.E4M3[ok.codes]
    if k_bound is None:
        assert np.array_equal(u8(c["k"]), ok.codes), what
    else:
        step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(kr), 2.0 ** -6))) * 2.0 ** -3, 2.0 ** -9)
        differ = k != kr
        assert np.mean(differ) < k_bound and np.all(np.abs(k - kr) <= step * 1.0001), what


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P,d,Hk", [(16, 64, 3), (32, 128, 2), (64, 128, 1), (128, 64, 2)])
@pytest.mark.parametrize("rotate", [False, True])
def test_append_packed(P, d, Hk, rotate, dtype):
    """Sequences with 0, 1 and many new tokens behind caches that end at every kind of place, twice in
    a row. Without rotation and norm every code is the oracle's; with them a key that lies within fp32
    rounding of the border of two codes may take either."""
    announce(f"append P={P} d={d} Hk={Hk} rotate={rotate} {dtype}")
    held = [0, 1, P - 1, P, P + 1, 2 * P - 1, 0, 5, 3]
    new = [1, P, 1, 0, 2 * P + 3, 2, 3 * P, 0, P - 3]
    width = 7
    c = cache_case(len(held), Hk, d, P, width, seed=P + d)
    ok, ov = cache_oracles(c)
    g = to_dev(c)
    f = inv_freq(d) if rotate else None
    w = 1 + 0.1 * torch.randn(d, generator=gen(2)) if rotate else None
    for call in range(2):
        cu = torch.tensor([0] + list(np.cumsum(new)))
        x = torch.randn(int(cu[-1]), 2 * Hk * d + 16, generator=gen(call + 31))
        x = (x * torch.exp(torch.randn(int(cu[-1]), 1, generator=gen(call)))).to(dtype)    # tokens of different size
        k_raw = x[:, :Hk * d].unflatten(1, (Hk, d))
        v_raw = x[:, Hk * d:2 * Hk * d].unflatten(1, (Hk, d))
        xd = x.cuda()
        lens = torch.tensor(held)
        gdn.gdn_kv_append(xd[:, :Hk * d].unflatten(1, (Hk, d)), xd[:, Hk * d:2 * Hk * d].unflatten(1, (Hk, d)),
                          g["k"], g["v"], g["ks"], g["vs"], g["table"], lens.cuda(), cu_seqlens=cu.cuda(),
                          inv_freq=dev(f), k_weight=dev(w))
        torch.cuda.synchronize()
        for n in range(len(held)):
            a, b = int(cu[n]), int(cu[n + 1])
            pos = held[n] + np.arange(b - a)
            k = oa.norm_rope(k_raw[a:b], w, pos, None if f is None else f.numpy())
            ok.append(n, held[n], k)
            ov.append(n, held[n], v_raw[a:b])
        check_cache(g, ok, ov, f"call {call}", k_bound=0.01 if rotate else None)
        held = [h + m for h, m in zip(held, new)]
        new = [2, 0, 1, P, 1, P + 1, 4, 1, 2]


def test_append_one_token_each_matches_packed_form():
    """The single-token form (no offsets) over many steps, pages being filled and rescaled on the way."""
    announce("append single tokens")
    N, Hk, d, P = 5, 2, 64, 16
    c = cache_case(N, Hk, d, P, 4, seed=3)
    ok, ov = cache_oracles(c)
    g, g2 = to_dev(c), to_dev(c)
    cu = torch.arange(N + 1).cuda()
    lens = torch.tensor([0, 3, 14, 15, 16])
    for step in range(20):
        x = (torch.randn(N, 2, Hk, d, generator=gen(step)) * 1.3 ** step).to(BF)
        k, v = x[:, 0].contiguous(), x[:, 1].contiguous()
        for t, off in ((g, None), (g2, cu)):
            gdn.gdn_kv_append(k.cuda(), v.cuda(), t["k"], t["v"], t["ks"], t["vs"], t["table"], lens.cuda(), cu_seqlens=off)
        for n in range(N):
            ok.append(n, int(lens[n]), k[n:n + 1])
            ov.append(n, int(lens[n]), v[n:n + 1])
        lens = lens + 1
    torch.cuda.synchronize()
    check_cache(g, ok, ov, "single")
    check_cache(g2, ok, ov, "packed")


def test_append_special_values_and_zero_rows():
    """Infinities saturate without moving the scale, NaN stays NaN, all-zero pages get the least scale, and
    values that meet a code or a border of the scale exactly."""
    announce("append special values")
    c = cache_case(3, 1, 64, 16, 2, seed=4)
    ok, ov = cache_oracles(c)
    g = to_dev(c)
    x = torch.randn(3, 1, 64, generator=gen(5))
    x[0, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    x[1] = 0
    x[2] *= 0.1
    x[2, 0, 0] = 448.0 * 2.0 ** -5
    k = x.clone()
    k[2, 0, 0] = 448.0 * 2.0 ** -5 * (1 + 2.0 ** -20)
    lens = torch.zeros(3, dtype=torch.int64)
    gdn.gdn_kv_append(k.cuda(), x.cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], lens.cuda())
    torch.cuda.synchronize()
    for n in range(3):
        ok.append(n, 0, k[n:n + 1])
        ov.append(n, 0, x[n:n + 1])
    assert np.array_equal(f64(g["vs"]), ov.scale) and np.array_equal(f64(g["ks"]), ok.scale)
    assert f64(g["vs"])[int(c["table"][1, 0]), 0] == 2.0 ** -100
    assert f64(g["vs"])[int(c["table"][2, 0]), 0] == 2.0 ** -5 and f64(g["ks"])[int(c["table"][2, 0]), 0] == 2.0 ** -4
    got, ref = oa.E4M3[u8(g["v"])], oa.E4M3[ov.codes]
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])


def test_append_bad_tables_and_lengths_write_only_what_they_name():
    """Entries that are no page, lengths beyond the table or negative, malformed offsets: the rest of the
    cache keeps its bytes, and well-formed sequences beside them are right."""
    announce("append bad pages")
    N, Hk, d, P = 4, 2, 128, 16
    c = cache_case(N, Hk, d, P, 3, seed=6, spare=5)
    num = c["k"].shape[0]
    c["table"][1] = torch.tensor([-1, num, 2 ** 31 - 1])
    ok, ov = cache_oracles(c)
    g = to_dev(c)
    x = torch.randn(4 * 20, Hk, d, generator=gen(8)).to(BF)
    lens = torch.tensor([0, 4, 3 * P - 2, 10 ** 12])     # sequence 2 runs out of table, 3 is beyond it
    gdn.gdn_kv_append(x.cuda(), x.cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], lens.cuda())
    torch.cuda.synchronize()
    for n in range(N):
        ok.append(n, int(lens[n]), x[20 * n:20 * n + 20])
        ov.append(n, int(lens[n]), x[20 * n:20 * n + 20])
    check_cache(g, ok, ov, "bad pages")
    # malformed offsets: sequence 0 is [0, 20), 1 reversed, 2 beyond the end
    c = cache_case(3, Hk, d, P, 3, seed=7)
    ok, ov = cache_oracles(c)
    g = to_dev(c)
    cu = torch.tensor([0, 20, 5, 10 ** 9])
    gdn.gdn_kv_append(x[:30].cuda(), x[:30].cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"],
                      torch.tensor([0, -7, 3]).cuda(), cu_seqlens=cu.cuda())
    torch.cuda.synchronize()
    ov.append(0, 0, x[:20])
    first = c["table"][0, :2].numpy()
    assert np.array_equal(u8(g["v"])[first], ov.codes[first])


# ----------------------------------------------------------------------------
# prompt attention
# ----------------------------------------------------------------------------

def prefill_case(T, Hq, Hk, d, dtype, seed):
    g = gen(seed)
    x = torch.randn(T, (Hq + 2 * Hk) * d + 8, generator=g).to(dtype)
    xd = x.cuda()
    parts, at = [], 0
    for H in (Hq, Hk, Hk):
        parts.append(slice(at, at + H * d))
        at += H * d
    cut = lambda t: [t[:, s].unflatten(1, (-1, d)) for s in parts]  # noqa: E731
    return cut(x), cut(xd)


def check_prefill(o, host, bounds, window, scale, dtype, d):
    q, k, v = host
    for a, b in zip(bounds, bounds[1:]):
        if a == b:
            continue
        ro, ra, reach = oa.attention(q[a:b], k[a:b], v[a:b], window, scale)
        within(o[a:b], ro, attn_bound(ro, ra, reach, b - a, d, dtype), f"rows {a}:{b}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 1, 20, 64, 200])
@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 128), (3, 3, 64), (7, 1, 128), (16, 1, 64)])
def test_prefill_packed(Hq, Hk, d, window, dtype):
    """Packed sequences of every length class, rows of a wider buffer."""
    announce(f"prefill Hq={Hq} Hk={Hk} d={d} window={window} {dtype}")
    lens = [1, 0, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 0, 300]
    bounds = [0] + list(np.cumsum(lens))
    host, dv = prefill_case(bounds[-1], Hq, Hk, d, dtype, 11 + Hq)
    o = gdn.gdn_attn_prefill(*dv, cu_seqlens=torch.tensor(bounds).cuda(), window=window)
    torch.cuda.synchronize()
    check_prefill(o, host, bounds, window, None, dtype, d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,T", [(1, 1), (3, 100), (2, 512), (1, 1000)])
def test_prefill_equal_lengths_and_scales(N, T, dtype):
    announce(f"prefill N={N} T={T} {dtype}")
    host, dv = prefill_case(N * T, 4, 2, 128, dtype, N + T)
    bounds = list(range(0, N * T + 1, T))
    for scale in (None, -0.05, 1.0):
        o = gdn.gdn_attn_prefill(*dv, N=N, scale=scale)
        check_prefill(o, host, bounds, 0, scale, dtype, 128)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_keeps_uncovered_rows_and_sequences_apart(dtype):
    """Rows that no range covers keep their output; NaN and infinities in one sequence, and in rows of no
    sequence, reach no other."""
    announce(f"prefill apart {dtype}")
    T = 300
    host, _ = prefill_case(T, 2, 1, 64, dtype, 5)
    q, k, v = [t.clone().contiguous() for t in host]
    for t, bad in ((q, math.nan), (k, math.inf), (v, math.nan)):
        t[100:170] = bad          # the second sequence
        t[260:] = bad             # behind the last one
    o = torch.full((T, 2, 64), 7.0, dtype=dtype, device="cuda")
    cu = torch.tensor([0, 100, 170, 260])
    gdn.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu_seqlens=cu.cuda(), o=o)
    torch.cuda.synchronize()
    assert bool((o[260:] == 7).all())
    check_prefill(o, (q, k, v), [0, 100], 0, None, dtype, 64)
    ro, ra, reach = oa.attention(q[170:260], k[170:260], v[170:260])
    within(o[170:260], ro, attn_bound(ro, ra, reach, 90, 64, dtype), "third sequence")


def test_prefill_large_scores_and_equal_scores():
    """Scores of some hundred (one key takes all), falling and rising maxima, and equal scores."""
    announce("prefill large scores")
    T, d = 400, 128
    g = gen(3)
    q = torch.randn(T, 2, d, generator=g).to(BF)
    k = (torch.randn(T, 1, d, generator=g) * torch.linspace(0.1, 12, T)[:, None, None]).to(BF)
    v = torch.randn(T, 1, d, generator=g).to(BF)
    for kk in (k, k.flip(0), torch.zeros_like(k)):
        o = gdn.gdn_attn_prefill(q.cuda(), kk.cuda(), v.cuda(), scale=0.3)
        check_prefill(o, (q, kk, v), [0, T], 0, 0.3, BF, d)


def test_prefill_malformed_offsets_stay_in_bounds():
    announce("prefill malformed offsets")
    host, dv = prefill_case(200, 2, 1, 128, BF, 8)
    cu = torch.tensor([0, 130, 40, 10 ** 12])
    o = gdn.gdn_attn_prefill(*dv, cu_seqlens=cu.cuda())
    torch.cuda.synchronize()
    check_prefill(o, host, [0, 40], 0, None, BF, 128)


# ----------------------------------------------------------------------------
# attention over the cache
# ----------------------------------------------------------------------------

def check_decode(o, q, c, lens, window, scale, dtype, P, d):
    ok, ov = cache_oracles(c)
    for n, L in enumerate(lens):
        k, there = ok.tokens(n, L)
        v, _ = ov.tokens(n, L)
        L = len(k)
        lo = max(0, L - window) if window else 0
        keep = np.arange(L)[there & (np.arange(L) >= lo)]
        kk, vv = k[keep], v[keep]
        if len(keep) == 0:
            assert bool((o[n] == 0).all()), n
            continue
        ro, ra, reach = oa.attention(f64(q[n:n + 1]), kk, vv, 0, scale)
        within(o[n:n + 1], ro, attn_bound(ro, ra, reach, len(keep), d, dtype), f"sequence {n} of {L}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 1, 50, 640])
@pytest.mark.parametrize("Hq,Hk,d,P", [(4, 2, 128, 16), (16, 1, 64, 32), (21, 3, 128, 64), (40, 2, 64, 128), (3, 3, 128, 32)])
def test_decode(Hq, Hk, d, P, window, dtype):
    """Lengths of every class: none, one, at and around steps, pages and splits, beyond the table."""
    announce(f"decode Hq={Hq} Hk={Hk} d={d} P={P} window={window} {dtype}")
    width = 1536 // P
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, P, P + 1, 511, 512, 513, 1000, 1536, 5000, -3]
    c = cache_case(len(lens), Hk, d, P, width, seed=Hq + P)
    q = torch.randn(len(lens), Hq, d, generator=gen(4)).to(dtype)
    g = to_dev(c)
    o = gdn.gdn_attn_decode(q.cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], torch.tensor(lens).cuda(),
                            window=window)
    torch.cuda.synchronize()
    check_decode(o, q, c, lens, window, None, dtype, P, d)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_one_long_sequence(dtype):
    """One sequence split over many workgroups, with a workspace of the caller's that held something else."""
    announce(f"decode long {dtype}")
    P, d = 64, 128
    c = cache_case(1, 2, d, P, 300, seed=1)
    q = torch.randn(1, 8, d, generator=gen(6)).to(dtype)
    g = to_dev(c)
    for L, scale in ((300 * P, None), (300 * P - 37, -0.2), (6000, 0.5)):
        need = gdn.gdn_attn_decode_workspace_size(dev(q), g["k"], g["table"])
        assert need > 0
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
        o = gdn.gdn_attn_decode(q.cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], torch.tensor([L]).cuda(),
                                scale=scale, workspace=ws)
        torch.cuda.synchronize()
        assert bool((ws[need:] == 255).all())
        check_decode(o, q, c, [L], 0, scale, dtype, P, d)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_ignores_what_lies_behind_the_last_token(dtype):
    """NaN codes, infinite and NaN scales behind the last token and in pages that are not used; entries that
    are no page hide their tokens."""
    announce(f"decode NaN behind {dtype}")
    N, Hk, d, P = 4, 1, 128, 16
    lens = [5, 16, 37, 90]
    c = cache_case(N, Hk, d, P, 6, seed=2, spare=3)
    used = np.zeros(c["k"].shape[:1] + (P,), bool)
    for n, L in enumerate(lens):
        for t in range(L):
            used[int(c["table"][n, t // P]), t % P] = True
    for name in "kv":
        raw = c[name].view(torch.uint8)
        raw[torch.from_numpy(~used)[:, None, :, None].expand_as(raw)] = 0x7f
    free = torch.from_numpy(~used.any(1))
    c["ks"][free], c["vs"][free] = math.inf, math.nan
    c["table"][3, 1], c["table"][3, 4] = -5, 2 ** 31 - 1
    c["table"][1, 1:] = c["k"].shape[0]
    q = torch.randn(N, 4, d, generator=gen(9)).to(dtype)
    g = to_dev(c)
    for window in (0, 12):
        o = gdn.gdn_attn_decode(q.cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], torch.tensor(lens).cuda(),
                                window=window)
        torch.cuda.synchronize()
        check_decode(o, q, c, lens, window, None, dtype, P, d)


# ----------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 24])
def test_prompt_then_decode_steps(window, dtype):
    """A layer as it is served: packed prompts through norm and rotation, prompt attention and the cache,
    then single tokens; every decode output against the oracle on the cache that was really written, and the
    last prompt row against the same row from the cache (whose codes are 8 bits)."""
    announce(f"prompt then decode window={window} {dtype}")
    Hq, Hk, d, P, rope = 8, 2, 128, 16, 64
    lens = [1, 40, 17, 64]
    N, steps = len(lens), 5
    f = inv_freq(rope)
    gq, gk = 1 + 0.1 * torch.randn(2, d, generator=gen(1))
    c = cache_case(N, Hk, d, P, 6, seed=12)
    g = to_dev(c)
    held = torch.zeros(N, dtype=torch.int64, device="cuda")

    def project(rows, seed):
        x = torch.randn(rows, (Hq + 2 * Hk) * d, generator=gen(seed)).to(dtype).cuda()
        return (x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)),
                x[:, (Hq + Hk) * d:].unflatten(1, (Hk, d)))

    cu = torch.tensor([0] + list(np.cumsum(lens)))
    pos = torch.cat([torch.arange(L) for L in lens])
    q_raw, k_raw, v = project(int(cu[-1]), 20)
    kw = dict(inv_freq=dev(f))
    q, k = gdn.gdn_qk_norm_rope(q_raw, k_raw, positions=dev(pos), q_weight=dev(gq), k_weight=dev(gk), **kw)
    o = gdn.gdn_attn_prefill(q, k, v, cu_seqlens=cu.cuda(), window=window)
    gdn.gdn_kv_append(k_raw, v, g["k"], g["v"], g["ks"], g["vs"], g["table"], held, cu_seqlens=cu.cuda(),
                      k_weight=dev(gk), **kw)
    held += torch.tensor(lens).cuda()
    check_prefill(o, (q.cpu(), k.cpu(), v.cpu()), cu.tolist(), window, None, dtype, d)
    last = gdn.gdn_attn_decode(q[cu[1:] - 1].contiguous(), g["k"], g["v"], g["ks"], g["vs"], g["table"], held,
                               window=window)
    ref = o[cu[1:] - 1]
    # codes are off by at most 2^-4 relative on every k and v: far from exact, but the same row
    assert float((last.double() - ref.double()).norm() / ref.double().norm()) < 0.1
    for step in range(steps):
        q_raw, k_raw, v = project(N, 30 + step)
        q, _ = gdn.gdn_qk_norm_rope(q_raw, positions=held, q_weight=dev(gq), **kw)
        gdn.gdn_kv_append(k_raw, v, g["k"], g["v"], g["ks"], g["vs"], g["table"], held, k_weight=dev(gk), **kw)
        held += 1
        o = gdn.gdn_attn_decode(q, g["k"], g["v"], g["ks"], g["vs"], g["table"], held, window=window)
        torch.cuda.synchronize()
        check_decode(o, q.cpu(), {n: t.cpu() for n, t in g.items()}, held.tolist(), window, None, dtype, P, d)


def test_captured_decode_step_replays():
    """A decode step (norm and rotation, append, attention over a split cache) captured into a graph and
    replayed with new inputs, eager work between the replays; every replay against the eager call."""
    announce("captured decode step")
    N, Hq, Hk, d, P, width = 3, 8, 2, 128, 32, 60
    c = cache_case(N, Hk, d, P, width, seed=13)
    g, e = to_dev(c), to_dev(c)
    f = dev(inv_freq(128))
    x = torch.zeros(N, (Hq + 2 * Hk) * d, dtype=BF, device="cuda")
    held = torch.tensor([0, 700, 1800], device="cuda")
    o = torch.zeros(N, Hq, d, dtype=BF, device="cuda")

    def step(t, out):
        q_raw = x[:, :Hq * d].unflatten(1, (Hq, d))
        k_raw, v = x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)), x[:, (Hq + Hk) * d:].unflatten(1, (Hk, d))
        q, _ = gdn.gdn_qk_norm_rope(q_raw, positions=held, inv_freq=f)
        gdn.gdn_kv_append(k_raw, v, t["k"], t["v"], t["ks"], t["vs"], t["table"], held, inv_freq=f)
        return gdn.gdn_attn_decode(q, t["k"], t["v"], t["ks"], t["vs"], t["table"], held + 1, o=out)

    assert gdn.gdn_attn_decode_workspace_size(o, g["k"], g["table"]) > 0
    step(to_dev(c), torch.empty_like(o))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(g, o)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=gen(i)).to(BF))
        graph.replay()
        torch.cuda.synchronize()
        want = step(e, torch.empty_like(o))
        torch.cuda.synchronize()
        assert torch.equal(o, want), i
        for n in ("k", "v"):
            assert torch.equal(g[n].view(torch.uint8), e[n].view(torch.uint8)), i
        assert torch.equal(g["ks"], e["ks"]) and torch.equal(g["vs"], e["vs"])
        held += 1


def test_streams_and_raw_handles():
    """Work on a stream other than the current one, given as a stream and as a handle; outputs and
    workspaces that the call allocates belong to that stream."""
    announce("streams")
    P, d = 64, 128
    c = cache_case(2, 2, d, P, 100, seed=14)
    g = to_dev(c)
    q = torch.randn(2, 8, d, generator=gen(1)).to(BF).cuda()
    lens = torch.tensor([6400, 3000]).cuda()
    want = gdn.gdn_attn_decode(q, g["k"], g["v"], g["ks"], g["vs"], g["table"], lens)
    host, dv = prefill_case(300, 4, 2, 128, BF, 2)
    want_p = gdn.gdn_attn_prefill(*dv)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for _ in range(8):
            o = gdn.gdn_attn_decode(q, g["k"], g["v"], g["ks"], g["vs"], g["table"], lens, stream=stream)
            p = gdn.gdn_attn_prefill(*dv, stream=stream)
            s.synchronize()
            assert torch.equal(o, want) and torch.equal(p, want_p)


def test_results_are_the_same_every_time():
    announce("bitwise repeatable")
    host, dv = prefill_case(700, 4, 2, 128, BF, 3)
    c = to_dev(cache_case(2, 2, 128, 32, 100, seed=15))
    q = torch.randn(2, 8, 128, generator=gen(1)).to(BF).cuda()
    lens = torch.tensor([3200, 1111]).cuda()
    p0 = gdn.gdn_attn_prefill(*dv)
    d0 = gdn.gdn_attn_decode(q, c["k"], c["v"], c["ks"], c["vs"], c["table"], lens)
    for _ in range(5):
        assert torch.equal(p0, gdn.gdn_attn_prefill(*dv))
        assert torch.equal(d0, gdn.gdn_attn_decode(q, c["k"], c["v"], c["ks"], c["vs"], c["table"], lens))


@pytest.mark.parametrize("N", [63, 64, 70, 300, 1100])
def test_many_sequences(N):
    """More sequences than lanes of a wave, and than are ranked: packed append, prompt attention and
    cached attention, sequences of no token among them."""
    announce(f"many sequences N={N}")
    Hq, Hk, d, P, dtype = 4, 2, 64, 16, BF
    g = gen(N)
    lens = torch.randint(0, 40, (N,), generator=g)
    lens[torch.rand(N, generator=g) < 0.2] = 0
    lens[N // 2] = 300
    bounds = [0] + torch.cumsum(lens, 0).tolist()
    cu = torch.tensor(bounds)
    host, dv = prefill_case(bounds[-1], Hq, Hk, d, dtype, N)
    for window in (0, 7, 5000):
        o = gdn.gdn_attn_prefill(*dv, cu_seqlens=cu.cuda(), window=window)
        torch.cuda.synchronize()
        check_prefill(o, host, bounds, window, None, dtype, d)
    width = 30
    num = N * 4 + 40
    table = torch.full((N, width), -1, dtype=torch.int32)
    order, at = torch.randperm(num, generator=g).to(torch.int32), 0
    held = torch.randint(0, 20, (N,), generator=g)
    for n in range(N):
        c = -(-int(held[n] + lens[n]) // P)
        table[n, :c] = order[at:at + c]
        at += c
    assert at <= num
    c = cache_case(1, Hk, d, P, 1, seed=N, spare=num - 1)
    c["table"] = table
    ok, ov = cache_oracles(c)
    e = to_dev(c)
    gdn.gdn_kv_append(dv[1], dv[2], e["k"], e["v"], e["ks"], e["vs"], e["table"], held.cuda(), cu_seqlens=cu.cuda())
    torch.cuda.synchronize()
    for n in range(N):
        ok.append(n, int(held[n]), host[1][bounds[n]:bounds[n + 1]])
        ov.append(n, int(held[n]), host[2][bounds[n]:bounds[n + 1]])
    check_cache(e, ok, ov, "many")
    for io in (BF, F32):
        q = torch.randn(N, Hq, d, generator=g).to(io)
        now = held + lens
        o = gdn.gdn_attn_decode(q.cuda(), e["k"], e["v"], e["ks"], e["vs"], e["table"], now.cuda())
        torch.cuda.synchronize()
        check_decode(o, q, {n: t.cpu() for n, t in e.items()}, now.tolist(), 0, None, io, P, d)


def test_caches_beyond_32_bit_offsets():
    """Pages that lie more than 2^32 bytes into the caches."""
    announce("cache beyond 4 GiB")
    Hk, d, P, N = 2, 128, 128, 2
    num = (1 << 32) // (Hk * P * d) + 64
    g = gen(1)
    k = torch.zeros(num, Hk, P, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.zeros_like(k.view(torch.uint8)).view(torch.float8_e4m3fn)
    ks, vs = torch.ones(2, num, Hk, device="cuda")
    table = torch.tensor([[num - 1, 5, num - 7], [num - 2, num - 30, 0]], dtype=torch.int32)
    lens = torch.tensor([300, 200])
    x = torch.randn(500, 2, Hk, d, generator=g).to(BF)
    cu = torch.tensor([0, 300, 500])
    gdn.gdn_kv_append(x[:, 0].contiguous().cuda(), x[:, 1].contiguous().cuda(), k, v, ks, vs, table.cuda(),
                      torch.zeros(2, dtype=torch.int64, device="cuda"), cu_seqlens=cu.cuda())
    q = torch.randn(N, 4, d, generator=g).to(BF)
    o = gdn.gdn_attn_decode(q.cuda(), k, v, ks, vs, table.cuda(), lens.cuda())
    torch.cuda.synchronize()
    used = table.flatten().long()
    small = dict(k=k.view(torch.uint8)[used.cuda()].cpu().view(torch.float8_e4m3fn),
                 v=v.view(torch.uint8)[used.cuda()].cpu().view(torch.float8_e4m3fn),
                 ks=ks[used.cuda()].cpu(), vs=vs[used.cuda()].cpu(),
                 table=torch.arange(6, dtype=torch.int32).view(2, 3))
    ok, ov = cache_oracles({**small, "k": torch.zeros_like(small["k"].view(torch.uint8)).view(torch.float8_e4m3fn),
                            "v": torch.zeros_like(small["v"].view(torch.uint8)).view(torch.float8_e4m3fn),
                            "ks": torch.ones(6, Hk), "vs": torch.ones(6, Hk)})
    for n in range(N):
        ok.append(n, 0, x[int(cu[n]):int(cu[n + 1]), 0])
        ov.append(n, 0, x[int(cu[n]):int(cu[n + 1]), 1])
    assert np.array_equal(u8(small["k"])[:5], ok.codes[:5]) and np.array_equal(u8(small["v"])[:5], ov.codes[:5])
    check_decode(o, q, small, lens.tolist(), 0, None, BF, P, d)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_beyond_32_bit_offsets(dtype):
    """Query, key and value rows more than 2^32 bytes into a wide buffer."""
    announce(f"rows beyond 4 GiB {dtype}")
    ld, d = 1 << 17, 64
    T = (1 << 32) // (ld * dtype.itemsize) + 700
    x = torch.empty(T, ld, dtype=dtype, device="cuda")
    x[T - 600:, :4 * d] = torch.randn(600, 4 * d, generator=gen(3)).to(dtype).cuda()
    x[:T - 600, :4 * d] = 1.0
    q, k, v = x[:, :2 * d].unflatten(1, (2, d)), x[:, 2 * d:3 * d].unflatten(1, (1, d)), x[:, 3 * d:4 * d].unflatten(1, (1, d))
    cu = torch.tensor([0, T - 600, T - 250, T])
    o = gdn.gdn_attn_prefill(q, k, v, cu_seqlens=cu.cuda(), window=500)
    torch.cuda.synchronize()
    for a, b in ((T - 600, T - 250), (T - 250, T)):
        ro, ra, reach = oa.attention(q[a:b].cpu(), k[a:b].cpu(), v[a:b].cpu(), 500)
        within(o[a:b], ro, attn_bound(ro, ra, reach, b - a, d, dtype), "far rows")
    pos = torch.arange(T).cuda()
    f = inv_freq(d)
    qn, kn = gdn.gdn_qk_norm_rope(q, k, positions=pos, inv_freq=dev(f))
    y = f64(q[T - 9:])
    ref = oa.rotate(y, np.arange(T - 9, T), f.numpy(), False)
    within(qn[T - 9:], ref, rope_bound(ref, y, 1.0, dtype), "far norm_rope")


def test_calls_on_two_streams_at_once():
    """Split decodes and appends of two caches on two streams, many in flight: each as if alone."""
    announce("two streams at once")
    P, d = 32, 128
    cases = []
    for i in range(2):
        c = to_dev(cache_case(3, 2, d, P, 120, seed=20 + i))
        q = torch.randn(3, 8, d, generator=gen(i)).to(BF).cuda()
        lens = torch.tensor([3000 - i, 17, 2048 + i]).cuda()
        x = torch.randn(3, 2, d, generator=gen(5 + i)).to(BF).cuda()
        cases.append((c, q, lens, x))

    def run(c, q, lens, x):
        gdn.gdn_kv_append(x, x, c["k"], c["v"], c["ks"], c["vs"], c["table"], lens)
        return gdn.gdn_attn_decode(q, c["k"], c["v"], c["ks"], c["vs"], c["table"], lens + 1)

    want = [run(*t) for t in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_two_captured_graphs_with_a_workspace_each():
    """Two graphs of split decodes, replayed in turn and after eager work; outputs as the eager calls'."""
    announce("two graphs")
    P, d = 32, 128
    c = to_dev(cache_case(2, 2, d, P, 100, seed=30))
    graphs = []
    for i in range(2):
        q = torch.randn(2, 8, d, generator=gen(i)).to(BF).cuda()
        lens = torch.tensor([3000, 500 + 100 * i]).cuda()
        o = torch.empty_like(q)
        call = lambda q=q, lens=lens, o=o, **kw: gdn.gdn_attn_decode(  # noqa: E731
            q, c["k"], c["v"], c["ks"], c["vs"], c["table"], lens, o=o, **kw)
        call()
        torch.cuda.synchronize()
        want = o.clone()
        ws = torch.empty(gdn.gdn_attn_decode_workspace_size(q, c["k"], c["table"]), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(workspace=ws)
        graphs.append((g, o, want, call))
    for r in range(3):
        for g, o, want, call in graphs:
            o.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, o, want, call in graphs:
            assert torch.equal(o, want), r
            call()


def test_nothing_to_do():
    """No sequences, no tokens."""
    e = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    assert gdn.gdn_attn_prefill(e, e, e).shape == (0, 2, 64)
    c = to_dev(cache_case(1, 2, 64, 16, 2, seed=1))
    none = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    n0 = torch.empty(0, dtype=torch.int64, device="cuda")
    before = u8(c["k"])
    gdn.gdn_kv_append(e, e, c["k"], c["v"], c["ks"], c["vs"], none, n0)
    gdn.gdn_kv_append(e, e, c["k"], c["v"], c["ks"], c["vs"], c["table"], torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert gdn.gdn_attn_decode(e, c["k"], c["v"], c["ks"], c["vs"], none, n0).shape == (0, 2, 64)
    torch.cuda.synchronize()
    assert np.array_equal(u8(c["k"]), before)


def test_binding_refusals():
    x = torch.zeros(4, 2, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="dense rows"):
        gdn.gdn_qk_norm_rope(x.transpose(0, 1))
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        gdn.gdn_attn_prefill(x, x, x.float())
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        gdn.gdn_attn_prefill(x.half(), x.half(), x.half())
    with pytest.raises(ValueError, match="device tensor"):
        gdn.gdn_attn_prefill(x, x.cpu(), x)
    with pytest.raises(ValueError, match="shape"):
        gdn.gdn_attn_prefill(x, x, x[:3])
    with pytest.raises(ValueError, match="positions"):
        gdn.gdn_qk_norm_rope(x, inv_freq=torch.ones(32, device="cuda"))
    with pytest.raises(gdn.GdnError) as e:
        gdn.gdn_attn_prefill(torch.zeros(4, 2, 96, dtype=BF, device="cuda"), *[torch.zeros(4, 1, 96, dtype=BF, device="cuda")] * 2)
    assert e.value.status == gdn.GDN_ERR_UNSUPPORTED
    cache = torch.zeros(3, 2, 16, 64, dtype=torch.uint8, device="cuda")
    sc = torch.ones(3, 2, device="cuda")
    t, n = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        gdn.gdn_attn_decode(x, cache, cache, sc, sc, t, n)
    f8 = cache.view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="int64"):
        gdn.gdn_attn_decode(x, f8, f8.clone(), sc, sc, t, n.int())
    with pytest.raises(ValueError, match="N \\+ 1"):
        gdn.gdn_kv_append(x, x, f8, f8.clone(), sc, sc.clone(), t, n, cu_seqlens=n[:3])


@pytest.mark.parametrize("window", [0, 256, 300, 700])
@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 128), (3, 3, 64), (7, 1, 128)])
def test_prefill_few_long_prompts(Hq, Hk, d, window):
    """Few query tiles with many keys each (two waves share a tile's keys)."""
    announce(f"prefill few Hq={Hq} Hk={Hk} d={d} window={window}")
    lens = [0, 1, 64, 65, 129, 770, 63, 0, 1500]
    bounds = [0] + list(np.cumsum(lens))
    host, dv = prefill_case(bounds[-1], Hq, Hk, d, BF, 31 + Hq)
    o = gdn.gdn_attn_prefill(*dv, cu_seqlens=torch.tensor(bounds).cuda(), window=window)
    torch.cuda.synchronize()
    check_prefill(o, host, bounds, window, None, BF, d)


@pytest.mark.parametrize("T", [1, 63, 64, 65, 127, 128, 129, 256, 257, 320, 385, 449])
def test_prefill_one_prompt_of_every_tile_edge(T):
    announce(f"prefill one prompt T={T}")
    for d in (64, 128):
        host, dv = prefill_case(T, 2, 1, d, BF, T)
        for window in (0, 256, 257):
            o = gdn.gdn_attn_prefill(*dv, window=window)
            torch.cuda.synchronize()
            check_prefill(o, host, [0, T], window, None, BF, d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 40, 256])
@pytest.mark.parametrize("T,d", [(200, 128), (400, 64), (400, 128)])
def test_prefill_values_that_a_query_does_not_see(T, d, window, dtype):
    """Infinite and NaN values and keys reach the queries that see their token and no other, not those of
    the same tile either."""
    announce(f"prefill unseen T={T} d={d} window={window} {dtype}")
    host, _ = prefill_case(T, 2, 1, d, dtype, T + window)
    q, k, v = [t.clone().contiguous() for t in host]
    for j in (0, 5, 70, 100, 133, T - 2, T - 1):
        sees = torch.arange(T) >= j
        if window:
            sees &= torch.arange(T) < j + window
        clean = v.clone()
        clean[j, 0, 7] = 0
        ro, ra, reach = oa.attention(q, k, clean, window, 0.05)
        bound = attn_bound(ro, ra, reach, T, d, dtype)
        for bad in (math.nan, math.inf, -math.inf):
            w = clean.clone()
            w[j, 0, 7] = bad
            o = gdn.gdn_attn_prefill(q.cuda(), k.cuda(), w.cuda(), window=window, scale=0.05).cpu()
            hit = o[sees][:, :, 7]
            assert bool(hit.isnan().all()) if math.isnan(bad) else bool((hit == bad).all()), (j, bad)
            o[:, :, 7] = torch.where(sees[:, None], torch.as_tensor(ro[:, :, 7]).to(o.dtype), o[:, :, 7])
            within(o, ro, bound, f"value {bad} at {j}")
        kk = k.clone()
        kk[j, 0, 3] = math.nan
        o = gdn.gdn_attn_prefill(q.cuda(), kk.cuda(), clean.cuda(), window=window, scale=0.05).cpu()
        assert bool(o[sees].isnan().all()), j
        o[sees] = torch.as_tensor(ro).to(o.dtype)[sees]
        within(o, ro, bound, f"key at {j}")


@pytest.mark.parametrize("N,T,Hq,Hk", [(2, 300, 8, 4), (8, 257, 2, 1), (1, 600, 16, 8), (4, 300, 12, 2), (1, 2048, 16, 2)])
def test_prefill_few_equal_prompts(N, T, Hq, Hk):
    """The same in every order that tiles of equal prompts are dealt in."""
    announce(f"prefill few equal N={N} T={T} Hq={Hq} Hk={Hk}")
    for d in (64, 128):
        host, dv = prefill_case(N * T, Hq, Hk, d, BF, N + T + d)
        o = gdn.gdn_attn_prefill(*dv, N=N)
        torch.cuda.synchronize()
        check_prefill(o, host, list(range(0, N * T + 1, T)), 0, None, BF, d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("P,d,rope", [(16, 64, 32), (32, 128, 64), (128, 128, 96), (64, 64, 16)])
def test_append_part_of_the_head_turned(P, d, rope, inter, dtype):
    """Partly rotated and interleaved keys, with norm, at positions on both sides of 2^24 (where the
    angles' arithmetic changes), some behind older tokens of their page."""
    announce(f"append P={P} d={d} rope={rope} inter={inter} {dtype}")
    Hk, new = 2, 10
    width = (1 << 24) // P + 2
    f, w = inv_freq(rope), 1 + 0.1 * torch.randn(d, generator=gen(2))
    for at in (0, (1 << 24) - 5, (1 << 24) + P):
        c = cache_case(1, Hk, d, P, 3, seed=P + d)
        first = at // P
        few = c["table"]
        c["table"] = torch.full((1, width + 2), -1, dtype=torch.int32)
        c["table"][:, first:first + 2] = few[:, :2]
        ok, ov = cache_oracles(c)
        g = to_dev(c)
        x = torch.randn(2, new, Hk, d, generator=gen(at % 97)).to(dtype)
        lens = torch.tensor([at])
        gdn.gdn_kv_append(x[0].cuda(), x[1].cuda(), g["k"], g["v"], g["ks"], g["vs"], g["table"], lens.cuda(),
                          inv_freq=f.cuda(), k_weight=w.cuda(), interleaved=inter)
        torch.cuda.synchronize()
        ok.append(0, at, oa.norm_rope(x[0], w, at + np.arange(new), f.numpy(), inter))
        ov.append(0, at, x[1])
        check_cache(g, ok, ov, f"at {at}", k_bound=0.01)


def test_binding_refuses_what_is_no_flag_and_no_stream():
    x = torch.zeros(4, 2, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="true or false"):
        gdn.gdn_qk_norm_rope(x, interleaved=torch.zeros(2))
    with pytest.raises(ValueError, match="stream"):
        gdn.gdn_qk_norm_rope(x, q=x.clone(), stream=1 << 80)
    gdn.gdn_qk_norm_rope(x)
    torch.cuda.synchronize()


@pytest.mark.parametrize("window", [0, 300])
def test_prefill_many_prompts_of_one_head(window):
    """Packed prompts that more than a wave's lanes rank, few tiles in all."""
    announce(f"prefill many prompts of one head, window={window}")
    lens = torch.randint(0, 600, (70,), generator=gen(5)).tolist()
    bounds = [0] + list(np.cumsum(lens))
    host, dv = prefill_case(bounds[-1], 1, 1, 128, BF, 17)
    o = gdn.gdn_attn_prefill(*dv, cu_seqlens=torch.tensor(bounds).cuda(), window=window)
    torch.cuda.synchronize()
    check_prefill(o, host, bounds, window, None, BF, 128)


@pytest.mark.parametrize("window", [0, 64, 65, 300])
@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 128), (3, 3, 64), (16, 1, 128)])
def test_prefill_fp32_few_and_many_tiles(Hq, Hk, d, window):
    """fp32: few query tiles (more waves to a tile's keys) and many of them."""
    announce(f"prefill fp32 Hq={Hq} Hk={Hk} d={d} window={window}")
    lens = [0, 1, 64, 65, 129, 330, 63, 0, 400]
    bounds = [0] + list(np.cumsum(lens))
    host, dv = prefill_case(bounds[-1], Hq, Hk, d, F32, 41 + Hq)
    for N in (len(lens), 1):                 # the same rows as one prompt of 1052 tokens
        o = gdn.gdn_attn_prefill(*dv, cu_seqlens=torch.tensor(bounds if N > 1 else [0, bounds[-1]]).cuda(), window=window)
        torch.cuda.synchronize()
        check_prefill(o, host, bounds if N > 1 else [0, bounds[-1]], window, None, F32, d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [130, 400])
def test_prefill_query_that_is_not_finite(T, dtype):
    """A NaN or infinite query spoils its own row only."""
    announce(f"prefill NaN query T={T} {dtype}")
    host, _ = prefill_case(T, 2, 1, 128, dtype, T)
    q, k, v = [t.clone().contiguous() for t in host]
    ro, ra, reach = oa.attention(q, k, v)
    bound = attn_bound(ro, ra, reach, T, 128, dtype)
    for j, bad in ((0, math.nan), (77, math.inf), (T - 1, math.nan)):
        w = q.clone()
        w[j, 1, 9] = bad
        o = gdn.gdn_attn_prefill(w.cuda(), k.cuda(), v.cuda()).cpu()
        o[j, 1] = torch.as_tensor(ro[j, 1]).to(o.dtype)
        within(o, ro, bound, f"query {bad} at {j}")
