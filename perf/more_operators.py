"""What a hybrid's training needs next to the delta rule's own forward and
backward: the attention layers' gradients, and the residual stream between
all layers, as cases that can be measured.

  attn_train     causal attention over packed prompts with its backward pass,
                 which forms the probabilities again
  norm_rope_grad the gradient of the norm and rotation of query and key heads
  add_norm       the residual's addition and the RMS norm behind it, the output
                 in the inputs' type or in 8 bits with scales
  add_norm_grad  its gradient

`run` computes a case in elementary torch operations, or with `own` set
through this repository's entry points; `exact` computes it in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
LARGEST_FLOPS = 14 * 128 * 16 * 16384 * 16385 / 2   # the largest listed case: train_long
LARGEST_ROWS = 32768 * 4096                         # elements of the largest residual stream


def listed():
    return [
        # three short prompts in fp32 at the small fp32 shape's heads: latency
        dict(name="train_small_fp32", op="attn_train", N=3, tokens=257, Hq=4, Hk=2, d=64, window=0, dtype="fp32",
             packed=True),
        # the B8 T4096 training shape's tokens and heads, every query head with a key head of its own
        dict(name="train_B8_T4096", op="attn_train", N=8, tokens=32768, Hq=16, Hk=16, d=128, window=0, dtype="bf16",
             packed=False),
        # a hybrid's 2K sliding window over 16 packed documents of mixed lengths, grouped heads
        dict(name="train_window_mix", op="attn_train", N=16, tokens=32768, Hq=16, Hk=2, d=128, window=2048,
             dtype="bf16", packed=True),
        # one long document, grouped heads
        dict(name="train_long", op="attn_train", N=1, tokens=16384, Hq=16, Hk=2, d=128, window=0, dtype="bf16",
             packed=False),
        # many short documents packed together, heads of 64, odd lengths
        dict(name="train_short_d64", op="attn_train", N=29, tokens=8191, Hq=6, Hk=3, d=64, window=0, dtype="bf16",
             packed=True),
        # the gradient of a training batch's queries and keys, all of the head rotated
        dict(name="norm_rope_grad_train", op="norm_rope_grad", rows=32768, Hq=16, Hk=2, d=128, rope=128, inter=False,
             dtype="bf16", far=1 << 15, stretch=1.0),
        # fp32, interleaved pairs, half of the head, far positions with stretched frequencies
        dict(name="norm_rope_grad_far_fp32", op="norm_rope_grad", rows=1023, Hq=6, Hk=3, d=64, rope=32, inter=True,
             dtype="fp32", far=1 << 20, stretch=8.0),
        # one decode step of one sequence: launch latency is all there is
        dict(name="add_norm_one", op="add_norm", rows=1, C=2048, dtype="bf16", res="bf16", group=-1),
        # a training batch's rows at the width of 16 heads of 128, the residual stream in fp32
        dict(name="add_norm_train", op="add_norm", rows=32768, C=2048, dtype="bf16", res="fp32", group=-1),
        # a prefill's rows for an 8-bit projection, a scale for each 128 channels
        dict(name="add_norm_e4m3", op="add_norm", rows=8192, C=4096, dtype="bf16", res="bf16", group=128),
        # the gradient of a training batch, the residual stream in fp32
        dict(name="add_norm_grad_train", op="add_norm_grad", rows=32768, C=2048, dtype="bf16", res="fp32"),
        # fp32, few rows of an odd width
        dict(name="add_norm_grad_odd_fp32", op="add_norm_grad", rows=777, C=1032, dtype="fp32", res="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_train", "attn_train", "norm_rope_grad", "add_norm", "add_norm_grad"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    Hk = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if op == "attn_train":
        N = _log(rng, 1, 32)
        tokens = _log(rng, 16 * N, max(16 * N + 1, 4096 if dtype == "fp32" else 16384))
        window = rng.choice([0, 0, _log(rng, 16, 4096)])
        packed = rng.random() < 0.7
        if not packed:
            tokens -= tokens % N
        Hq = Hk * group
        while Hq > Hk and 7.0 * d * Hq * tokens * min(tokens, window or tokens) > LARGEST_FLOPS:
            Hq -= Hk
        return dict(op=op, N=N, tokens=tokens, Hq=Hq, Hk=Hk, d=d, window=window, dtype=dtype, packed=packed)
    if op == "norm_rope_grad":
        return dict(op=op, rows=_log(rng, 1, 32768), Hq=Hk * group, Hk=Hk, d=d,
                    rope=rng.choice([r for r in (0, 32, 64, 96, 128) if r <= d]), inter=rng.random() < 0.3,
                    dtype=dtype, far=_log(rng, 1 << 10, 1 << 20), stretch=rng.choice([1.0, 4.0, 32.0]))
    res = rng.choice([dtype, "fp32"])
    rows = _log(rng, 1, 32768)
    C = 8 * _log(rng, 8, min(1024, LARGEST_ROWS // (8 * rows)))
    if op == "add_norm_grad":
        return dict(op=op, rows=rows, C=C, dtype=dtype, res=res)
    g = rng.choice([-1, -1, 0, 32, 64, 128])     # -1: no 8-bit output, 0: one scale for a row
    if g > 0:
        C = max(g, C // g * g)
    return dict(op=op, rows=rows, C=C, dtype=dtype, res=res, group=g)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(n, total, seed, least):
    """n lengths of at least `least` that sum to total: log-normal shares, as documents come."""
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(0.8 * torch.randn(n, generator=g, dtype=torch.float64))
    lens = torch.floor(w / w.sum() * (total - n * least)).to(torch.int64) + least
    lens[int(torch.randint(n, (1,), generator=g))] += total - int(lens.sum())
    return lens


def _inv_freq(rope, stretch):
    i = torch.arange(0, rope, 2, dtype=torch.float64)
    return (1e6 ** (-i / rope) / stretch).to(torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "attn_train":
        N, T, Hq, Hk, d = case["N"], case["tokens"], case["Hq"], case["Hk"], case["d"]
        lens = _lengths(N, T, seed, 1) if case["packed"] else torch.full((N,), T // N)
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(lens, 0)])
        # q and k normed and rotated, v a column block of the projection's rows
        s.update(q=randn(T, Hq, d).to(dt), k=randn(T, Hk, d).to(dt),
                 v=randn(T, 2 * Hk * d).to(dt)[:, Hk * d:].unflatten(1, (Hk, d)), d_o=randn(T, Hq, d).to(dt),
                 cu_seqlens=cu.cuda() if case["packed"] else None, bounds=cu.tolist())
        return s
    if case["op"] == "norm_rope_grad":
        rows, Hq, Hk, d = case["rows"], case["Hq"], case["Hk"], case["d"]
        qkv = (1.5 * randn(rows, (Hq + 2 * Hk) * d)).to(dt)     # the projection's rows: q | k | v
        s.update(q_raw=qkv[:, :Hq * d].unflatten(1, (Hq, d)),
                 k_raw=qkv[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)),
                 positions=torch.randint(case["far"], (rows,), generator=gen, device="cuda"),
                 inv_freq=_inv_freq(case["rope"], case["stretch"]).cuda() if case["rope"] else None,
                 rope_scale=1.0 + 0.1 * math.log(case["stretch"]), q_weight=1.0 + 0.1 * randn(d),
                 k_weight=1.0 + 0.1 * randn(d), dq=randn(rows, Hq, d).to(dt), dk=randn(rows, Hk, d).to(dt))
        return s
    rows, C, rt = case["rows"], case["C"], DTYPES[case["res"]]
    s.update(weight=1.0 + 0.1 * randn(C))
    if case["op"] == "add_norm":
        s.update(x=randn(rows, C).to(dt), res=(3.0 * randn(rows, C)).to(rt))
    else:
        s.update(r=(3.0 * randn(rows, C)).to(rt), dy=randn(rows, C).to(dt), d_res_out=randn(rows, C).to(rt))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"attn_train": _attn_train, "norm_rope_grad": _norm_rope_grad, "add_norm": _add_norm,
            "add_norm_grad": _add_norm_grad}[s["case"]["op"]](s)


def _attn_train(s):
    c, q, k, v, d_o = s["case"], s["q"], s["k"], s["v"], s["d_o"]
    if own:
        import gated_delta_rule_gdn_amd as gdn
        kw = dict(cu_seqlens=s["cu_seqlens"], N=c["N"], window=c["window"])
        o, stats = gdn.gdn_attn_prefill_save(q, k, v, **kw)
        dq, dk, dv = gdn.gdn_attn_backward(q, k, v, o, d_o, stats, **kw)
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}
    H, G, d = c["Hk"], c["Hq"] // c["Hk"], c["d"]
    o, dq = torch.empty_like(q), torch.empty_like(q)
    dk, dv = torch.empty_like(k), torch.empty(v.shape, dtype=v.dtype, device=v.device)
    for a, b in zip(s["bounds"], s["bounds"][1:]):
        kh, vh = (x[a:b].float().transpose(0, 1).contiguous() for x in (k, v))       # [H, L, d]
        kt, vt = kh.transpose(1, 2).contiguous(), vh.transpose(1, 2).contiguous()    # [H, d, L]
        gk, gv = torch.zeros_like(kh), torch.zeros_like(vh)
        step = max(1, (1 << 28) // (c["Hq"] * (b - a)))                      # query rows at a time
        for lo in range(a, b, step):
            hi = min(b, lo + step)
            first = max(a, lo + 1 - c["window"]) if c["window"] else a       # the first key that any row sees
            n, at = hi - lo, slice(first - a, hi - a)

            def rows(x):                                                     # [H, G n, d]
                return x[lo:hi].float().view(n, H, G, d).permute(1, 2, 0, 3).reshape(H, G * n, d)

            def back(x, to):
                to[lo:hi] = x.view(H, G, n, d).permute(2, 0, 1, 3).reshape(n, H * G, d).to(to.dtype)

            qs, gs = rows(q), rows(d_o)
            p = (qs @ kt[:, :, at].contiguous()).view(H, G, n, hi - first) * d ** -0.5
            t = torch.arange(lo, hi, device=q.device)[:, None]
            u = torch.arange(first, hi, device=q.device)
            p.masked_fill_((u > t) | (u <= t - c["window"]) if c["window"] else u > t, -math.inf)
            p = torch.exp(p - p.amax(-1, keepdim=True))
            p = (p / p.sum(-1, keepdim=True)).view(H, G * n, hi - first)
            r = p @ vh[:, at].contiguous()
            back(r, o)
            gv[:, at] += p.transpose(1, 2).contiguous() @ gs
            p = p * (gs @ vt[:, :, at].contiguous() - (gs * r).sum(-1, keepdim=True)) * d ** -0.5
            back(p @ kh[:, at].contiguous(), dq)
            gk[:, at] += p.transpose(1, 2).contiguous() @ qs
        dk[a:b], dv[a:b] = (x.transpose(0, 1).to(k.dtype) for x in (gk, gv))
    return {"o": o, "dq": dq, "dk": dk, "dv": dv}


def _turned_back(g, positions, inv_freq, inter, factor):
    """g [rows, H, d], its first 2 len(inv_freq) channels turned back by the angles of its position."""
    if inv_freq is None:
        return g
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()     # 64 bits: far positions
    c = (angle.cos() * factor).float()[:, None]
    sn = (angle.sin() * factor).float()[:, None]
    r, rest = g[..., :2 * half], g[..., 2 * half:]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        out = torch.stack((a * c + b * sn, b * c - a * sn), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        out = torch.cat((a * c + b * sn, b * c - a * sn), -1)
    return torch.cat((out, rest), -1)


def _norm_grad(x, weight, g):
    """Gradients of x / sqrt(mean(x^2) + eps) * weight (fp32)."""
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * inv
    w = (g * n).flatten(0, -2).sum(0)
    g = g * weight
    return inv * (g - n * (n * g).mean(-1, keepdim=True)), w


def _norm_rope_grad(s):
    inter, f = s["case"]["inter"], s["rope_scale"]
    if own:
        import gated_delta_rule_gdn_amd as gdn
        dq, dk, qw, kw = gdn.gdn_qk_norm_rope_backward(
            s["dq"], s["dk"], s["q_raw"], s["k_raw"], positions=s["positions"] if s["inv_freq"] is not None else None,
            inv_freq=s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"], interleaved=inter, rope_scale=f,
            eps=EPS)
        return {"dq_raw": dq, "dk_raw": dk, "dq_weight": qw, "dk_weight": kw}
    out = {}
    for n in "qk":
        g = _turned_back(s["d" + n].float(), s["positions"], s["inv_freq"], inter, f)
        x, w = _norm_grad(s[n + "_raw"].float(), s[n + "_weight"], g)
        out["d%s_raw" % n], out["d%s_weight" % n] = x.to(s["d" + n].dtype), w
    return out


def _add_norm(s):
    c = s["case"]
    if own:
        import gated_delta_rule_gdn_amd as gdn
        y, scale, r = gdn.gdn_add_norm(s["x"], s["res"], s["weight"], eps=EPS,
                                       group=None if c["group"] < 0 else c["group"])
        return {"y": y, "r": r} if scale is None else {"y": y, "scale": scale, "r": r}
    r = s["x"].float() + s["res"].float()
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"]
    if c["group"] < 0:
        return {"y": y.to(s["x"].dtype), "r": r.to(s["res"].dtype)}
    y = y.unflatten(1, (-1, c["group"] or c["C"]))
    scale = y.abs().amax(-1) / E4M3_MAX
    return {"y": (y / scale[..., None]).flatten(1).to(torch.float8_e4m3fn), "scale": scale, "r": r.to(s["res"].dtype)}


def _add_norm_grad(s):
    if own:
        import gated_delta_rule_gdn_amd as gdn
        dx, d_res, w = gdn.gdn_add_norm_backward(s["dy"], s["r"], s["weight"], d_res_out=s["d_res_out"], eps=EPS)
        return {"dx": dx, "d_res": d_res, "d_weight": w}
    x, w = _norm_grad(s["r"].float(), s["weight"], s["dy"].float())
    x = x + s["d_res_out"].float()
    return {"dx": x.to(s["dy"].dtype), "d_res": x.to(s["r"].dtype), "d_weight": w}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _pairs(lens, window):
    """(query, key) pairs of causal sequences."""
    n = 0
    for L in lens:
        w = min(L, window) if window else L
        n += w * (w + 1) // 2 + (L - w) * w
    return n


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "attn_train":
        lens = [case["tokens"] / case["N"]] * case["N"]
        if case["packed"]:
            lens = _lengths(case["N"], case["tokens"], 0, 1).tolist()
        n = _pairs([int(L) for L in lens], case["window"])
        # 2 products of the forward, 5 of the backward
        return {"bytes": case["tokens"] * 4 * (case["Hq"] + case["Hk"]) * case["d"] * b,
                "flops": 14 * case["d"] * case["Hq"] * n}
    if case["op"] == "norm_rope_grad":
        n = case["rows"] * (case["Hq"] + case["Hk"]) * case["d"]
        return {"bytes": 3 * n * b + 8 * case["rows"], "flops": 18 * n}
    n, rb = case["rows"] * case["C"], BYTES[case["res"]]
    if case["op"] == "add_norm":
        out = b if case["group"] < 0 else 1 + 4 / (case["group"] or case["C"])
        return {"bytes": n * (b + 2 * rb + out) + 4 * case["C"], "flops": 5 * n}
    # one gradient serves x and the residual where their types are one
    return {"bytes": n * (b + 3 * rb + (b if b != rb else 0)) + 8 * case["C"], "flops": 12 * n}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _attn64(s, case):
    """Head by head: the softmax's Jacobian applied to d_o v^T."""
    G, c = case["Hq"] // case["Hk"], 1.0 / math.sqrt(case["d"])
    out = {n: torch.zeros(s[m].shape, dtype=torch.float64, device="cuda")
           for n, m in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    for a, b in zip(s["bounds"], s["bounds"][1:]):
        for h in range(case["Hq"]):
            k, v = s["k"][a:b, h // G].double(), s["v"][a:b, h // G].double()
            for lo in range(a, b, 4096):
                hi = min(b, lo + 4096)
                q, g = s["q"][lo:hi, h].double(), s["d_o"][lo:hi, h].double()
                gap = torch.arange(lo, hi, device="cuda")[:, None] - torch.arange(a, hi, device="cuda")
                seen = (gap >= 0) & (gap < case["window"]) if case["window"] else gap >= 0
                p = torch.softmax(torch.where(seen, c * torch.mm(q, k[:hi - a].T), -math.inf), -1)
                e = torch.mm(g, v[:hi - a].T)
                e = c * (p * e - p * torch.linalg.vecdot(p, e)[:, None])
                out["o"][lo:hi, h] = torch.mm(p, v[:hi - a])
                out["dq"][lo:hi, h] = torch.mm(e, k[:hi - a])
                out["dk"][a:hi, h // G] += torch.mm(e.T, q)
                out["dv"][a:hi, h // G] += torch.mm(p.T, g)
    return out


def _norm64(x, w, g):
    """x, g in 64 bits: the gradient of x / rms(x) * w is (w g - x (x . w g) / (n rms^2)) / rms."""
    ms = x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS
    wg = w.double() * g
    dx = (wg - x * ((x * wg).sum(-1, keepdim=True) / (x.shape[-1] * ms))) / ms.sqrt()
    return dx, (g * x / ms.sqrt()).reshape(-1, x.shape[-1]).sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn_train":
        return _attn64(s, case)
    if case["op"] == "norm_rope_grad":
        out = {}
        for n in "qk":
            g = s["d" + n].double()
            if s["inv_freq"] is not None:
                h = s["inv_freq"].numel()
                angle = -torch.outer(s["positions"].double(), s["inv_freq"].double())[:, None, :]
                spin = torch.polar(torch.full_like(angle, s["rope_scale"]), angle)
                at = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["inter"] else (slice(0, h), slice(h, 2 * h))
                z = torch.complex(g[..., at[0]].contiguous(), g[..., at[1]].contiguous()) * spin
                g[..., at[0]], g[..., at[1]] = z.real, z.imag
            out["d%s_raw" % n], out["d%s_weight" % n] = _norm64(s[n + "_raw"].double(), s[n + "_weight"], g)
        return out
    if case["op"] == "add_norm":
        r = s["x"].double() + s["res"].double()
        y = r / torch.sqrt(r.square().sum(-1, keepdim=True) / case["C"] + EPS) * s["weight"].double()
        if case["group"] < 0:
            return {"y": y, "r": r}
        y = y.view(case["rows"], -1, case["group"] or case["C"])
        scale = y.abs().max(-1).values / E4M3_MAX
        return {"y": (y / scale[..., None]).view(case["rows"], -1), "scale": scale, "r": r}
    dx, w = _norm64(s["r"].double(), s["weight"], s["dy"].double())
    dx = dx + s["d_res_out"].double()
    return {"dx": dx, "d_res": dx, "d_weight": w}
