"""GPU parity of a hybrid's training and residual operators (gdn_attn_prefill_save,
gdn_attn_backward, gdn_qk_norm_rope_backward, gdn_add_norm, gdn_add_norm_backward)
against the float64 oracle (``oracle.hybrid``), through the C ABI.  Bounds are per
element and derived in hybrid_helpers."""
import math

import numpy as np
import pytest
import torch

from attn_helpers import BF, F32, HALF, attn_bound, f64, gen, inv_freq, within
from helpers import announce
from hybrid_helpers import EPS, attn_grads, attn_inputs, check_attn, norm_grad_bound, rope_grads, views
from oracle import attention as oa
from oracle import hybrid as oh

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import gated_delta_rule_gdn_amd as gdn  # noqa: E402


def dev(x):
    return None if x is None else x.cuda()


def case(T, Hq, Hk, d, dtype, seed):
    host = attn_inputs(T, Hq, Hk, d, dtype, seed)
    width = (Hq + 2 * Hk) * d + 8
    x = torch.empty(T, width, dtype=dtype, device="cuda")
    on = views(x, Hq, Hk, d)
    for a, b in zip(on, host):
        a.copy_(b)
    return host, (*on, host[3].cuda())


def both(dv, **kw):
    q, k, v, d_o = dv
    grad = kw.pop("grad_dtype", None)
    o, stats = gdn.gdn_attn_prefill_save(q, k, v, **kw)
    return o, stats, gdn.gdn_attn_backward(q, k, v, o, d_o, stats, grad_dtype=grad, **kw)


# ----------------------------------------------------------------------------
# attention and its gradients
# ----------------------------------------------------------------------------

def stats_of(stats, o):
    """[T, Hq, 2] and (bf16) the bytes [T, Hq, d] behind it."""
    T, H, d = o.shape
    return stats[:2 * T * H].view(T, H, 2), stats[2 * T * H:].view(torch.uint8).view(T, H, -1)


def to_16_bits(o, stats):
    """o before its rounding to bf16, with the bytes that stats holds of it."""
    low = stats_of(stats, o)[1].to(torch.int32)
    bits = o.contiguous().view(torch.int16).to(torch.int32) << 16
    return (bits + 256 * low - 0x7f80).view(torch.float32)


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("N,L,Hq,Hk,d,window", [(1, 700, 4, 2, 128, 0), (1, 700, 4, 1, 64, 100), (3, 90, 40, 40, 128, 0),
                                                (5, 130, 90, 45, 64, 33), (2, 1, 1, 1, 64, 0)])
def test_statistics_and_low_bytes(N, L, Hq, Hk, d, window, far):
    """Equal scores: weights of 1 and a sum that is their number, so outputs are means of values, in fp32 up to
    their rounding.  `far`: an infinite value at each sequence's end sends queries that do not see it another way."""
    announce(f"statistics N={N} L={L} Hq={Hq} d={d} window={window} far={far}")
    host = [t.clone().contiguous() for t in attn_inputs(N * L, Hq, Hk, d, BF, L + d)]
    host[0].zero_()
    if far:
        host[2][L - 1::L] = math.inf
    q, k, v, _ = (dev(t) for t in host)
    o, stats = gdn.gdn_attn_prefill_save(q, k, v, N=N, window=window)
    torch.cuda.synchronize()
    got = f64(to_16_bits(o, stats).cpu())
    st = f64(stats_of(stats, o)[0].cpu())
    t = np.arange(L)
    n = np.minimum(t + 1, window or L)
    for i in range(N):
        rows = slice(i * L, (i + 1) * L)
        # 2^m l is the number of keys; one or both rounded once, 2^(0 - m) exact for the m that scores of 0 leave
        total = np.exp2(st[rows, :, 0]) * st[rows, :, 1]
        assert np.all(np.abs(total - n[:, None]) <= 2.0 ** -20 * n[:, None])
        vh = f64(host[2][rows]).repeat(Hq // Hk, axis=1)
        sums = np.stack([vh[j + 1 - n[j]:j + 1].sum(0) for j in t])
        mean, reach = sums / n[:, None, None], np.cumsum(np.abs(vh), 0) / n[:, None, None]
        seen = t < L - 1 if far else t < L
        # sums of n terms in fp32 and a byte's half step (a whole one at its end)
        bound = (n[:, None, None] + 16) * EPS * reach + 2.0 ** -15 * np.abs(mean) + 1e-30
        assert np.all(np.abs(got[rows][seen] - mean[seen]) <= bound[seen])
        if far:
            assert not np.any(np.isfinite(got[rows][-1]))     # spoiled, as what it sees


LENS = [1, 0, 2, 31, 32, 33, 64, 127, 128, 129, 300, 5]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 1, 20, 64, 129])
@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 128), (16, 1, 64), (3, 3, 128), (6, 2, 64), (7, 1, 128)])
def test_attention_packed(Hq, Hk, d, window, dtype):
    announce(f"attn backward packed Hq={Hq} Hk={Hk} d={d} window={window} {dtype}")
    bounds = np.concatenate([[0], np.cumsum(LENS)]).tolist()
    host, on = case(bounds[-1], Hq, Hk, d, dtype, Hq + window)
    kw = dict(cu_seqlens=torch.tensor(bounds).cuda(), window=window)
    o, stats, got = both(on, **kw)
    plain = gdn.gdn_attn_prefill(*on[:3], **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, plain)
    check_attn(got, host, bounds, window, None, dtype, what="packed")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,L,scale", [(1, 1, None), (1, 200, -0.11), (3, 100, 0.3), (8, 65, None), (2, 257, 1e-3)])
def test_attention_equal_lengths_and_scales(N, L, scale, dtype):
    announce(f"attn backward equal N={N} L={L} scale={scale} {dtype}")
    host, on = case(N * L, 4, 2, 128, dtype, N + L)
    _, _, got = both(on, N=N, scale=scale)
    torch.cuda.synchronize()
    check_attn(got, host, list(range(0, N * L + 1, L)), 0, scale, dtype, what="equal")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hk,d,window", [(1500, 8, 1, 64, 0), (1100, 2, 2, 128, 0), (1300, 4, 1, 128, 500)])
def test_attention_one_long_sequence(T, Hq, Hk, d, window, dtype):
    """Key tiles that several workgroups share."""
    announce(f"attn backward long T={T} {dtype}")
    host, on = case(T, Hq, Hk, d, dtype, T)
    _, _, got = both(on, window=window)
    torch.cuda.synchronize()
    check_attn(got, host, [0, T], window, None, dtype, what="long")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,d,window", [(3, 3, 128, 0), (4, 2, 64, 0), (2, 1, 128, 150), (6, 2, 64, 190)])
def test_attention_few_tiles_of_many_keys(Hq, Hk, d, window, dtype):
    announce(f"attn backward few tiles Hq={Hq} d={d} window={window} {dtype}")
    bounds = [0, 300, 429, 430, 687, 687, 1010]
    host, on = case(bounds[-1], Hq, Hk, d, dtype, window + d)
    _, _, got = both(on, cu_seqlens=torch.tensor(bounds).cuda(), window=window)
    torch.cuda.synchronize()
    check_attn(got, host, bounds, window, None, dtype, what="few tiles")


def test_attention_many_sequences():
    """More sequences than are ranked by cost, and many equal ones."""
    announce("attn backward many sequences")
    lens = [1 + 7 * i % 13 for i in range(1100)]
    bounds = np.concatenate([[0], np.cumsum(lens)]).tolist()
    for dtype in (BF, F32):
        host, on = case(bounds[-1], 2, 1, 64, dtype, 3)
        _, _, got = both(on, cu_seqlens=torch.tensor(bounds).cuda())
        torch.cuda.synchronize()
        check_attn(got, host, bounds, 0, None, dtype, what="many")


@pytest.mark.parametrize("grad", [BF, F32])
@pytest.mark.parametrize("Hq,Hk,d,window", [(32, 4, 128, 0), (32, 8, 128, 50), (48, 6, 64, 0), (50, 10, 64, 50)])
def test_attention_of_many_heads(Hq, Hk, d, window, grad):
    """So many query tiles that each takes 128 queries."""
    announce(f"attn backward many heads Hq={Hq} Hk={Hk} d={d} window={window} {grad}")
    bounds = np.concatenate([[0], np.cumsum([1 + 37 * i % 97 for i in range(20)] + [161, 0, 257])]).tolist()
    host, on = case(bounds[-1], Hq, Hk, d, BF, Hq + d)
    _, _, got = both(on, cu_seqlens=torch.tensor(bounds).cuda(), window=window, grad_dtype=grad)
    torch.cuda.synchronize()
    check_attn(got, host, bounds, window, None, BF, grad, "many heads")


@pytest.mark.parametrize("d", [64, 128])
def test_attention_gradients_in_fp32_into_column_blocks(d):
    """bf16 inputs, gradients in fp32, all three into one buffer; other columns and rows of no sequence stay."""
    announce(f"attn backward column blocks d={d}")
    T, Hq, Hk = 150, 4, 2
    host, on = case(T, Hq, Hk, d, BF, 5)
    for grad in (BF, F32):
        x = torch.full((T, (Hq + 2 * Hk) * d + 16), 7.0, dtype=grad, device="cuda")
        dq, dk, dv = views(x, Hq, Hk, d)
        cu = torch.tensor([0, 60, 140]).cuda()
        q, k, v, d_o = on
        o, stats = gdn.gdn_attn_prefill_save(q, k, v, cu_seqlens=cu)
        gdn.gdn_attn_backward(q, k, v, o, d_o, stats, cu_seqlens=cu, dq=dq, dk=dk, dv=dv)
        torch.cuda.synchronize()
        check_attn((dq, dk, dv), host, [0, 60, 140], 0, None, BF, grad, "blocks")
        assert bool((x[:, -16:] == 7).all()) and bool((x[140:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_sequences_are_apart(dtype):
    """Rows that no range covers keep their gradients; NaN and infinities in one sequence, and in rows of no
    sequence, reach no other."""
    announce(f"attn backward apart {dtype}")
    T = 400
    host = [t.clone().contiguous() for t in attn_inputs(T, 2, 1, 64, dtype, 5)]
    for t, bad in zip(host, (math.nan, math.inf, math.nan, -math.inf)):
        t[100:170] = bad          # the second sequence
        t[360:] = bad             # behind the last one
    cu = torch.tensor([0, 100, 170, 360]).cuda()
    on = [t.cuda() for t in host]
    o, stats = torch.full((T, 2, 64), 7.0, dtype=dtype, device="cuda"), torch.full((T * 2 * (2 + 16 * (dtype == BF)),), 7.0, device="cuda")
    gdn.gdn_attn_prefill_save(*on[:3], cu_seqlens=cu, o=o, stats=stats)
    grads = [torch.full((T, h, 64), 7.0, dtype=dtype, device="cuda") for h in (2, 1, 1)]
    ws = torch.full((gdn.gdn_attn_backward_workspace_size(on[0], on[1], N=3),), 255, dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_backward(*on[:3], o, on[3], stats, cu_seqlens=cu, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
    torch.cuda.synchronize()
    assert all(bool((t[360:] == 7).all()) for t in (o, stats_of(stats, o)[0], *grads))
    if dtype == BF:
        kept = stats_of(torch.full_like(stats, 7.0), o)[1]
        assert torch.equal(stats_of(stats, o)[1][360:], kept[360:])
    check_attn(grads, host, [0, 100], 0, None, dtype, what="first")
    check_attn([t[170:360] for t in grads], [t[170:360] for t in host], [0, 190], 0, None, dtype, what="third")


def test_attention_malformed_offsets_stay_in_bounds():
    """Ranges that overlap, run backwards and pass the end: the queries of one range alone have its gradients."""
    announce("attn backward malformed offsets")
    for dtype in (BF, F32):
        host, on = case(200, 2, 1, 128, dtype, 8)
        _, _, got = both(on, cu_seqlens=torch.tensor([0, 130, 40, 10 ** 12]).cuda())
        torch.cuda.synchronize()
        ref, bound = attn_grads(*[t[:40] for t in host], 0, None, dtype)[0]
        within(got[0][:40], ref, bound, "dq")


def test_attention_large_and_equal_scores():
    """Scores of some hundred (one key takes all), rising and falling, and all equal."""
    announce("attn backward large scores")
    T, d = 300, 128
    for dtype in (BF, F32):
        g = gen(3)
        q = torch.randn(T, 2, d, generator=g).to(dtype)
        k = (torch.randn(T, 1, d, generator=g) * torch.linspace(0.1, 4, T)[:, None, None]).to(dtype)
        v, d_o = torch.randn(T, 1, d, generator=g).to(dtype), torch.randn(T, 2, d, generator=g).to(dtype)
        for kk in (k, k.flip(0), torch.zeros_like(k)):
            _, _, got = both([t.cuda() for t in (q, kk, v, d_o)], scale=0.3)
            torch.cuda.synchronize()
            check_attn(got, (q, kk, v, d_o), [0, T], 0, 0.3, dtype, what="large")


def test_attention_same_bits_again():
    announce("attn backward same bits")
    for dtype in (BF, F32):
        _, on = case(900, 8, 1, 128, dtype, 11)
        a, b = both(on)[2], both(on)[2]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# ----------------------------------------------------------------------------
# norm and rotation
# ----------------------------------------------------------------------------

def split(x, Hq, Hk, d):
    return x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))


@pytest.mark.parametrize("io,grad", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rows,Hq,Hk,d,rope", [
    (1, 16, 2, 128, 64), (33, 5, 1, 128, 128), (70, 4, 3, 64, 64), (2000, 1, 1, 64, 32), (3, 8, 8, 128, 96),
    (65, 9, 2, 64, 16), (129, 2, 1, 128, 0)])
def test_norm_rope(rows, Hq, Hk, d, rope, inter, io, grad):
    announce(f"norm_rope backward rows={rows} Hq={Hq} Hk={Hk} d={d} rope={rope} inter={inter} {io} {grad}")
    g = gen(rows + rope)
    x = (1.5 * torch.randn(rows, (Hq + Hk) * d + 24, generator=g)).to(io)
    up = [torch.randn(rows, h, d, generator=g).to(grad) for h in (Hq, Hk)]
    w = [1 + 0.1 * torch.randn(d, generator=g) for _ in range(2)]
    pos, f = torch.randint(1 << 17, (rows,), generator=g), inv_freq(rope)
    raw = split(x, Hq, Hk, d)
    out = torch.full((rows, (Hq + Hk) * d + 8), 7.0, dtype=grad, device="cuda")
    to = split(out, Hq, Hk, d)
    r = gdn.gdn_qk_norm_rope_backward(dev(up[0]), dev(up[1]), *split(dev(x), Hq, Hk, d), positions=dev(pos) if rope else None,
                                      inv_freq=dev(f), q_weight=dev(w[0]), k_weight=dev(w[1]), interleaved=inter,
                                      rope_scale=1.25, dq_raw=to[0], dk_raw=to[1])
    torch.cuda.synchronize()
    assert bool((out[:, -8:] == 7).all())
    for i in range(2):
        (dx, bx), (dw, bw) = rope_grads(raw[i], w[i], pos, f, up[i], inter, 1.25, 1e-6, grad)
        within(r[i], dx, bx, "dx")
        within(r[2 + i], dw, bw, "d_weight")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_rope_one_operand_without_a_norm_in_place(dtype):
    announce(f"norm_rope backward single operands {dtype}")
    g = gen(7)
    up, pos, f = torch.randn(40, 3, 128, generator=g).to(dtype), torch.randint(1 << 17, (40,), generator=g), inv_freq(128)
    (ref, bound), _ = rope_grads(up, None, pos, f, up, False, 1.0, 0.0, dtype)
    for as_q in (True, False):
        y = up.cuda()
        kw = dict(positions=dev(pos), inv_freq=dev(f))
        r = (gdn.gdn_qk_norm_rope_backward(y, None, dq_raw=y, **kw) if as_q else
             gdn.gdn_qk_norm_rope_backward(None, y, dk_raw=y, **kw))
        torch.cuda.synchronize()
        assert r[0 if as_q else 1].data_ptr() == y.data_ptr() and [t is None for t in r].count(True) == 3
        within(y, ref, bound, "in place")


# ----------------------------------------------------------------------------
# the residual stream
# ----------------------------------------------------------------------------

WIDTHS = [8, 72, 512, 520, 1024, 1032, 1536, 1544, 2048, 2056, 4096, 5000, 8192, 16384]


def step_of(z):
    """Half a step of e4m3 at |z|."""
    return np.maximum(np.abs(z) * 2.0 ** -4, 2.0 ** -10)


@pytest.mark.parametrize("io,rt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("C", WIDTHS)
def test_add_norm(C, io, rt):
    announce(f"add_norm C={C} {io} {rt}")
    g = gen(C)
    for rows in (1, 2, 5, 33):
        x = torch.randn(rows, C + 16, generator=g).to(io)[:, :C]
        res, w = (3 * torch.randn(rows, C, generator=g)).to(rt), 1 + 0.1 * torch.randn(C, generator=g)
        on = torch.zeros(rows, C + 16, dtype=io, device="cuda")[:, :C]
        on.copy_(x)
        for use_res, use_w in ((True, True), (False, True), (True, False)):
            ry, rr = oh.add_norm(x, res if use_res else None, w if use_w else None, 1e-6)
            kw = dict(res=dev(res) if use_res else None, weight=dev(w) if use_w else None)
            y, scale, r = gdn.gdn_add_norm(on, **kw)
            assert scale is None and (r is not None) == use_res
            within(y, ry, (96 * EPS + HALF[io]) * np.abs(ry) + 1e-30, "y")
            if use_res:
                within(r, rr, (EPS + HALF[rt]) * np.abs(rr) + 1e-30, "r")
            for group in (0, 32, 64, 128):
                if group and C % group:
                    continue
                y, scale, r = gdn.gdn_add_norm(on, group=group, **kw)
                z = ry.reshape(rows, -1, group or C)
                top = np.abs(z).max(-1) / 448
                within(scale, top, 100 * EPS * top, "scale")
                z = (z / top[..., None]).reshape(rows, C)
                within(y.float(), z, step_of(z) * (1 + 2.0 ** -10) + 256 * EPS * np.abs(z), "codes")
                if use_res:
                    within(r, rr, (EPS + HALF[rt]) * np.abs(rr) + 1e-30, "r")


def test_add_norm_in_place_and_values_that_are_not_finite():
    announce("add_norm in place")
    g = gen(2)
    x, res, w = torch.randn(9, 256, generator=g).to(BF), torch.randn(9, 256, generator=g).to(BF), torch.ones(256)
    want = gdn.gdn_add_norm(x.cuda(), res.cuda(), w.cuda())
    a, b = x.cuda(), res.cuda()
    y, _, r = gdn.gdn_add_norm(a, b, w.cuda(), res_out=b, y=a)
    assert torch.equal(y, want[0]) and torch.equal(r, want[2]) and y.data_ptr() == a.data_ptr()
    c = x.cuda()
    y, _, r = gdn.gdn_add_norm(c, res.cuda(), w.cuda(), res_out=c)
    assert torch.equal(y, want[0]) and torch.equal(r, want[2])
    # rows that are not finite spoil themselves alone; a row of zeros is zero, at the least scale
    x[3, 7], x[5, 0] = math.nan, math.inf
    x[6], res[6] = 0, 0
    good = [0, 1, 2, 4, 7, 8]
    for group in (None, 0, 64):
        y, s, r = gdn.gdn_add_norm(x.cuda(), res.cuda(), w.cuda(), group=group)
        torch.cuda.synchronize()
        if group is None:
            assert torch.equal(y[good], want[0][good])
        else:
            assert bool((s[6] == np.float32(2.0 ** -100) / np.float32(448)).all())
            assert bool(torch.isfinite(y[good].float()).all()) and bool(torch.isfinite(s[good]).all())
        assert bool((y[6].float() == 0).all()) and bool(torch.isnan(y[3].float()).any())
    big = w.clone()
    big[5] = math.inf             # an infinite value: the largest code, and no part in the scale
    y, s, _ = gdn.gdn_add_norm(x[:3].cuda(), None, big.cuda(), group=0)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(s).all()) and y[:, 5].float().abs().tolist() == [448.0] * 3


@pytest.mark.parametrize("io,rt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("C", WIDTHS)
def test_add_norm_backward(C, io, rt):
    announce(f"add_norm backward C={C} {io} {rt}")
    g = gen(C + 1)
    for rows in (1, 3, 4, 5, 700 if C < 1100 else 37):
        dy = torch.randn(rows, C, generator=g).to(io)
        r, up = (3 * torch.randn(rows, C, generator=g)).to(rt), torch.randn(rows, C, generator=g).to(rt)
        w = 1 + 0.1 * torch.randn(C, generator=g)
        for use_up, use_w in ((True, True), (False, True), (True, False)):
            ref, refw = oh.add_norm_backward(dy, r, w if use_w else None, up if use_up else None, 1e-6)
            bx, bw = norm_grad_bound(r, w if use_w else np.ones(C), 1e-6, dy, np.zeros(C), K=160)
            if use_up:
                bx = bx + 2 * EPS * (np.abs(f64(up)) + np.abs(ref))
            dx, d_res, dw = gdn.gdn_add_norm_backward(dev(dy), dev(r), dev(w) if use_w else None,
                                                      d_res_out=dev(up) if use_up else None)
            torch.cuda.synchronize()
            within(dx, ref, bx + HALF[io] * np.abs(ref), "dx")
            within(d_res, ref, bx + HALF[rt] * np.abs(ref), "d_res")
            assert (dx is d_res) == (io == rt) and (dw is None) == (not use_w)
            if use_w:
                within(dw, refw, bw, "d_weight")


def test_add_norm_backward_in_place_and_many_rows():
    announce("add_norm backward in place, many rows")
    g = gen(9)
    rows, C = 9001, 264
    dy, r, up = [torch.randn(rows, C, generator=g) for _ in range(3)]
    w = 1 + 0.1 * torch.randn(C, generator=g)
    dy = dy.to(BF)
    ref, refw = oh.add_norm_backward(dy, r, w, up, 1e-6)
    bx, bw = norm_grad_bound(r, w, 1e-6, dy, np.zeros(C))
    bx = bx + 2 * EPS * (np.abs(f64(up)) + np.abs(ref))
    a, b = dy.cuda(), up.cuda()
    dx, d_res, dw = gdn.gdn_add_norm_backward(a, r.cuda(), w.cuda(), d_res_out=b, dx=a, d_res=b)
    torch.cuda.synchronize()
    assert dx.data_ptr() == a.data_ptr() and d_res.data_ptr() == b.data_ptr()
    within(dx, ref, bx + HALF[BF] * np.abs(ref), "dx")
    within(d_res, ref, bx + HALF[F32] * np.abs(ref), "d_res")
    within(dw, refw, bw, "d_weight")


def test_no_rows_give_zero_weight_gradients():
    announce("no rows")
    z = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    _, _, dw = gdn.gdn_add_norm_backward(z, z, w)
    h = torch.zeros(0, 2, 64, device="cuda")
    r = gdn.gdn_qk_norm_rope_backward(h, h, h, h, q_weight=w, k_weight=w)
    torch.cuda.synchronize()
    for t in (dw, r[2], r[3]):
        assert bool((t == 0).all())
    y, _, _ = gdn.gdn_add_norm(z, z, w)
    assert y.shape == (0, 64)
    o, stats = gdn.gdn_attn_prefill_save(h, h, h)
    assert all(t.shape == h.shape for t in gdn.gdn_attn_backward(h, h, h, o, h, stats))
