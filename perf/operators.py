"""The operators of the softmax-attention layers that stand between gated
delta-rule layers in a hybrid model, as cases that can be measured.

  norm_rope   norms of q and k per head with the rotary position in the same pass
  append      keys (normed, rotated) and values into a paged cache of 8-bit
              floats, one power-of-two scale for each page and head
  prefill     causal attention over packed prompts, grouped heads, full or in a
              sliding window
  decode      attention of one new token per sequence over that cache

`run` computes a case in elementary torch operations, or with `own` set
through this repository's entry points; `exact` computes it in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}
LARGEST_FLOPS = 4 * 128 * 16 * 32768 * 32769 / 2   # the largest listed case: long_prompt
MOST_CACHED = 1 << 20                                # tokens in a drawn batch's cache


def listed():
    return [
        # one decode step of one sequence: launch latency is all there is; rotation of half the head
        dict(name="norm_rope_one", op="norm_rope", rows=1, Hq=16, Hk=2, d=128, rope=64, inter=False, dtype="bf16",
             far=1 << 17, stretch=1.0),
        # a prefill's queries and keys, as many tokens as the B8 T4096 training shape, all of the head rotated
        dict(name="norm_rope_prefill", op="norm_rope", rows=32768, Hq=16, Hk=2, d=128, rope=128, inter=False,
             dtype="bf16", far=1 << 15, stretch=1.0),
        # fp32, interleaved pairs, positions far beyond the trained length with stretched frequencies
        dict(name="norm_rope_far_fp32", op="norm_rope", rows=1023, Hq=6, Hk=3, d=64, rope=64, inter=True,
             dtype="fp32", far=1 << 20, stretch=8.0),
        # one decode step of a serving batch: one token for each of 256 sequences, most pages partly filled
        dict(name="append_step", op="append", N=256, new=256, Hk=4, d=128, page=32, held=2048, rope=128, inter=False,
             dtype="bf16"),
        # a packed prefill of 16 prompts of mixed lengths written to fresh pages
        dict(name="append_prefill", op="append", N=16, new=32768, Hk=4, d=128, page=64, held=0, rope=64, inter=False,
             dtype="bf16"),
        # three short prompts in fp32 at the small fp32 shape's heads
        dict(name="prefill_small_fp32", op="prefill", N=3, tokens=257, Hq=4, Hk=2, d=64, window=0, dtype="fp32",
             packed=True),
        # the B8 T4096 training shape's tokens and heads, every query head with a key head of its own
        dict(name="prefill_B8_T4096", op="prefill", N=8, tokens=32768, Hq=16, Hk=16, d=128, window=0, dtype="bf16",
             packed=False),
        # a hybrid's 2K sliding window over 16 packed prompts of mixed lengths
        dict(name="prefill_window_mix", op="prefill", N=16, tokens=32768, Hq=16, Hk=2, d=128, window=2048,
             dtype="bf16", packed=True),
        # one long prompt, grouped heads
        dict(name="long_prompt", op="prefill", N=1, tokens=32768, Hq=16, Hk=2, d=128, window=0, dtype="bf16",
             packed=False),
        # a few short sequences in fp32, some of them empty or of one token: latency
        dict(name="decode_few_fp32", op="decode", N=5, longest=77, Hq=6, Hk=2, d=64, page=16, window=0, dtype="fp32"),
        # a serving batch of mixed lengths
        dict(name="decode_batch", op="decode", N=256, longest=8192, Hq=32, Hk=4, d=128, page=32, window=0,
             dtype="bf16"),
        # one sequence with a long cache: the work of one row split over the chip
        dict(name="decode_long", op="decode", N=1, longest=131072, Hq=32, Hk=4, d=128, page=64, window=0,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "prefill", "decode"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    inter = rng.random() < 0.3
    rope = rng.choice([r for r in (0, 32, 64, 96, 128) if r <= d])
    Hk = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm_rope":
        return dict(op=op, rows=_log(rng, 1, 32768), Hq=Hk * group, Hk=Hk, d=d, rope=rope, inter=inter, dtype=dtype,
                    far=_log(rng, 1 << 10, 1 << 20), stretch=rng.choice([1.0, 4.0, 32.0]))
    if op == "append":
        N = _log(rng, 1, 256)
        new = N if rng.random() < 0.5 else _log(rng, N, 32768)
        return dict(op=op, N=N, new=new, Hk=Hk, d=d, page=page, held=rng.choice([0, _log(rng, 1, 2048)]), rope=rope,
                    inter=inter, dtype=dtype)
    if op == "prefill":
        N = _log(rng, 1, 32)
        tokens = max(N, _log(rng, 1, 4096 if dtype == "fp32" else 32768))
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        packed = rng.random() < 0.7
        if not packed:
            tokens -= tokens % N
        Hq = Hk * group
        while Hq > Hk and 2.0 * d * Hq * tokens * min(tokens, window or tokens) > LARGEST_FLOPS:
            Hq -= Hk
        return dict(op=op, N=N, tokens=tokens, Hq=Hq, Hk=Hk, d=d, window=window, dtype=dtype, packed=packed)
    N = _log(rng, 1, 256)
    longest = _log(rng, 1, min(131072, MOST_CACHED // N))
    return dict(op=op, N=N, longest=longest, Hq=Hk * group, Hk=Hk, d=d, page=page,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(n, total, seed, least):
    """n lengths of at least `least` that sum to total: log-normal shares, as prompts come."""
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(0.8 * torch.randn(n, generator=g, dtype=torch.float64))
    lens = torch.floor(w / w.sum() * (total - n * least)).to(torch.int64) + least
    lens[int(torch.randint(n, (1,), generator=g))] += total - int(lens.sum())
    return lens


def _offsets(lens):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(lens, 0)])


def _held(case, seed):
    """Tokens that each sequence has in its cache."""
    g = torch.Generator().manual_seed(seed + 1)
    if case["op"] == "append":
        return torch.randint(case["held"] // 2, case["held"] + 1, (case["N"],), generator=g)
    u = torch.rand(case["N"], generator=g, dtype=torch.float64)
    lens = torch.floor((u ** 2) * (case["longest"] + 1)).to(torch.int64).clamp(max=case["longest"])
    lens[0] = case["longest"]
    return lens


def _inv_freq(rope, stretch):
    i = torch.arange(0, rope, 2, dtype=torch.float64)
    return (1e6 ** (-i / rope) / stretch).to(torch.float32)


def _cache(gen, held, pages_of, case):
    """A pool of pages in random order and the sequences' page tables. Every page holds values
    of about unit size at a scale of 2^-6 or 2^-7, as normed keys are."""
    N, Hk, P, d = case["N"], case["Hk"], case["page"], case["d"]
    counts = [(int(t) + P - 1) // P for t in pages_of]
    width = max(max(counts), 1)
    # the pool has room for the longest sequences that the case can hold, and is the same for every seed
    num = N * (case["held"] // P + 2) + case["new"] // P if case["op"] == "append" else sum(counts) + 3
    order = torch.randperm(num, generator=torch.Generator().manual_seed(N + num)).to(torch.int32)
    table = torch.full((N, width), -1, dtype=torch.int32)
    at = 0
    for n, c in enumerate(counts):
        table[n, :c] = order[at:at + c]
        at += c
    def pool():
        scale = torch.where(torch.rand(num, Hk, generator=gen, device="cuda") < 0.5, 2.0 ** -6, 2.0 ** -7)
        x = torch.randn(num, Hk, P, d, generator=gen, device="cuda")
        x = (x / scale[:, :, None, None]).clamp_(-E4M3_MAX, E4M3_MAX)
        return x.to(torch.float8_e4m3fn), scale
    kc, ks = pool()
    vc, vs = pool()
    return dict(k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, page_table=table.cuda(),
                seq_lens=held.cuda())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, d, Hk = DTYPES[case["dtype"]], case["d"], case["Hk"]
    s = dict(case=case)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def weight():
        return 1.0 + 0.1 * randn(d)

    if case["op"] == "norm_rope":
        Hq, rows = case["Hq"], case["rows"]
        qkv = (1.5 * randn(rows, (Hq + 2 * Hk) * d)).to(dt)     # the projection's rows: q | k | v
        s.update(q_raw=qkv[:, :Hq * d].unflatten(1, (Hq, d)),
                 k_raw=qkv[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)),
                 positions=torch.randint(case["far"], (rows,), generator=gen, device="cuda"),
                 inv_freq=_inv_freq(case["rope"], case["stretch"]).cuda() if case["rope"] else None,
                 rope_scale=1.0 + 0.1 * math.log(case["stretch"]), q_weight=weight(), k_weight=weight(),
                 q=torch.empty(rows, Hq, d, dtype=dt, device="cuda"),
                 k=torch.empty(rows, Hk, d, dtype=dt, device="cuda"))
        return s
    if case["op"] == "append":
        N, new = case["N"], case["new"]
        lens = torch.ones(N, dtype=torch.int64) if new == N else _lengths(N, new, seed, 1)
        held = _held(case, seed)
        kv = (1.5 * randn(new, 2 * Hk * d)).to(dt)
        s.update(_cache(gen, held, held + lens, case))
        s.update(k_raw=kv[:, :Hk * d].unflatten(1, (Hk, d)), v_raw=kv[:, Hk * d:].unflatten(1, (Hk, d)),
                 cu_seqlens=None if new == N else _offsets(lens).cuda(), k_weight=weight(),
                 inv_freq=_inv_freq(case["rope"], 1.0).cuda() if case["rope"] else None)
        # where each new token goes, for the plain form's gathers
        seq = torch.repeat_interleave(torch.arange(N), lens)
        pos = torch.arange(new) - _offsets(lens)[seq] + held[seq]
        s.update(seq=seq.cuda(), pos=pos.cuda())
        return s
    if case["op"] == "prefill":
        N, T, Hq = case["N"], case["tokens"], case["Hq"]
        lens = _lengths(N, T, seed, 1) if case["packed"] else torch.full((N,), T // N)
        cu = _offsets(lens)
        s.update(q=randn(T, Hq, d).to(dt), k=randn(T, Hk, d).to(dt),
                 v=randn(T, 2 * Hk * d).to(dt)[:, Hk * d:].unflatten(1, (Hk, d)),
                 cu_seqlens=cu.cuda() if case["packed"] else None, bounds=cu.tolist(),
                 o=torch.empty(T, Hq, d, dtype=dt, device="cuda"))
        return s
    held = _held(case, seed)
    s.update(_cache(gen, held, held, case))
    s.update(q=randn(case["N"], case["Hq"], d).to(dt),
             o=torch.empty(case["N"], case["Hq"], d, dtype=dt, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"norm_rope": _norm_rope, "append": _append, "prefill": _prefill, "decode": _decode}[s["case"]["op"]](s)


def _normed(x, weight, eps=1e-6):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _rotated(x, positions, inv_freq, inter, factor=1.0):
    """x [rows, H, d] with its first 2 len(inv_freq) channels rotated by the angles of its position."""
    if inv_freq is None:
        return x
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()     # 64 bits: far positions
    c = (angle.cos() * factor).float()[:, None]
    sn = (angle.sin() * factor).float()[:, None]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        out = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        out = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((out, rest), -1)


def _norm_rope(s):
    inter, f = s["case"]["inter"], s["rope_scale"]
    if own:
        import gated_delta_rule_gdn_amd as gdn
        q, k = gdn.gdn_qk_norm_rope(s["q_raw"], s["k_raw"], positions=s["positions"], inv_freq=s["inv_freq"],
                                    q_weight=s["q_weight"], k_weight=s["k_weight"], interleaved=inter, rope_scale=f,
                                    q=s["q"], k=s["k"])
        return {"q": q, "k": k}
    dt = s["q"].dtype
    return {"q": _rotated(_normed(s["q_raw"], s["q_weight"]), s["positions"], s["inv_freq"], inter, f).to(dt),
            "k": _rotated(_normed(s["k_raw"], s["k_weight"]), s["positions"], s["inv_freq"], inter, f).to(dt)}


def _write(x, cache, scale, s):
    """New tokens x [rows, H, d] (fp32) into the pages of their sequences. A page's scale is the least
    power of two that brings what it holds within the type; tokens that the page already held are
    rounded again where it grows."""
    P = cache.shape[2]
    table, lens, seq, pos = s["page_table"].long(), s["seq_lens"], s["seq"], s["pos"]
    page = table[seq, pos // P]
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax)
    need = torch.ldexp(torch.ones_like(amax), torch.where(m > 0.875, e - 8, e - 9).clamp(min=-100))
    kept_of = torch.zeros(cache.shape[0], dtype=torch.int64, device=x.device)
    first = pos == lens[seq]                           # a sequence's first new token: its page may hold older ones
    kept_of[page[first]] = pos[first] % P
    touched = torch.zeros(cache.shape[0], dtype=torch.bool, device=x.device)
    touched[page] = True
    at = touched.nonzero().flatten()
    kept, need, old_scale = kept_of[at][:, None], need[at], scale[at]
    new = torch.where(kept > 0, torch.maximum(old_scale, need), need)
    old = cache.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    again = (old * (old_scale / new)[:, :, None, None]).to(torch.float8_e4m3fn)
    held = torch.arange(P, device=x.device) < kept
    bits = torch.where(held[:, None, :, None], again.view(torch.uint8), cache.view(torch.uint8)[at])
    cache.view(torch.uint8)[at] = bits
    scale[at] = new
    cache.view(torch.uint8)[page, :, pos % P] = (x / scale[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _append(s):
    inter = s["case"]["inter"]
    if own:
        import gated_delta_rule_gdn_amd as gdn
        gdn.gdn_kv_append(s["k_raw"], s["v_raw"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                          s["page_table"], s["seq_lens"], cu_seqlens=s["cu_seqlens"], inv_freq=s["inv_freq"],
                          k_weight=s["k_weight"], interleaved=inter)
    else:
        k = _rotated(_normed(s["k_raw"], s["k_weight"]), s["pos"], s["inv_freq"], inter)
        _write(k, s["k_cache"], s["k_scale"], s)
        _write(s["v_raw"].float(), s["v_cache"], s["v_scale"], s)
    return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _prefill(s):
    c, q, k, v, o = s["case"], s["q"], s["k"], s["v"], s["o"]
    if own:
        import gated_delta_rule_gdn_amd as gdn
        return gdn.gdn_attn_prefill(q, k, v, cu_seqlens=s["cu_seqlens"], N=c["N"], window=c["window"], o=o)
    H, G, d = c["Hk"], c["Hq"] // c["Hk"], c["d"]
    for a, b in zip(s["bounds"], s["bounds"][1:]):
        kt = k[a:b].float().permute(1, 2, 0).contiguous()                    # [H, d, L]
        vt = v[a:b].float().permute(1, 0, 2).contiguous()                    # [H, L, d]
        step = max(1, (1 << 29) // (c["Hq"] * (b - a)))                      # query rows at a time
        for lo in range(a, b, step):
            hi = min(b, lo + step)
            first = max(a, lo + 1 - c["window"]) if c["window"] else a       # the first key that any row sees
            qs = q[lo:hi].float().view(hi - lo, H, G, d).permute(1, 2, 0, 3).reshape(H, G * (hi - lo), d)
            p = (qs @ kt[:, :, first - a:hi - a].contiguous()).view(H, G, hi - lo, hi - first) * d ** -0.5
            t = torch.arange(lo, hi, device=q.device)[:, None]
            u = torch.arange(first, hi, device=q.device)
            p.masked_fill_((u > t) | (u <= t - c["window"]) if c["window"] else u > t, -math.inf)
            p = torch.exp(p - p.amax(-1, keepdim=True))
            r = (p.view(H, G * (hi - lo), hi - first) @ vt[:, first - a:hi - a].contiguous()).view(H, G, hi - lo, d)
            o[lo:hi] = (r / p.sum(-1, keepdim=True)).permute(2, 0, 1, 3).reshape(hi - lo, H * G, d).to(o.dtype)
    return o


def _decode(s):
    c, q = s["case"], s["q"]
    if own:
        import gated_delta_rule_gdn_amd as gdn
        return gdn.gdn_attn_decode(q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"],
                                   s["seq_lens"], window=c["window"], o=s["o"])
    N, H, G, d, P = c["N"], c["Hk"], c["Hq"] // c["Hk"], c["d"], c["page"]
    table = s["page_table"].long().clamp(min=0)

    def rows(cache, scale):     # [N, H, tokens, d]
        x = cache.view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(N * H, -1, d)

    k, v = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
    p = (q.float().view(N * H, G, d) @ k.transpose(1, 2).contiguous()).view(N, H, G, -1) * d ** -0.5
    u = torch.arange(p.shape[-1], device=q.device)
    lens = s["seq_lens"][:, None, None, None]
    out = u >= lens
    if c["window"]:
        out = out | (u < lens - c["window"])
    p = p.masked_fill(out, -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-1e30))             # an empty cache: all weights 0
    r = (p.view(N * H, G, -1) @ v).view(N, H, G, d) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return r.view(N, H * G, d).to(q.dtype)


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
    b, d, Hk = BYTES[case["dtype"]], case["d"], case["Hk"]
    if case["op"] == "norm_rope":
        n = case["rows"] * (case["Hq"] + Hk) * d
        return {"bytes": 2 * n * b + 8 * case["rows"], "flops": 10 * n}
    if case["op"] == "append":
        # rows read, codes and the pages' scales written; older codes of a page are read only where its scale grows
        n = case["new"] * Hk * d
        pages = case["new"] / case["page"] + case["N"]
        return {"bytes": 2 * n * b + 2 * n + pages * (4 + 16 * Hk), "flops": 14 * n}
    if case["op"] == "prefill":
        lens = [case["tokens"] / case["N"]] * case["N"]
        if case["packed"]:
            lens = _lengths(case["N"], case["tokens"], 0, 1).tolist()
        n = _pairs([int(L) for L in lens], case["window"])
        return {"bytes": case["tokens"] * (2 * case["Hq"] + 2 * Hk) * d * b, "flops": 4 * d * case["Hq"] * n}
    lens = _held(case, 0)
    if case["window"]:
        lens = lens.clamp(max=case["window"])
    n = int(lens.sum())
    return {"bytes": 2 * n * Hk * d + 2 * case["N"] * case["Hq"] * d * b + n / case["page"] * (4 + 8 * Hk),
            "flops": 4 * d * case["Hq"] * n}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _turn64(x, pos, inv_freq, inter, factor):
    """x [rows, H, d] as complex pairs times factor e^(i pos inv_freq)."""
    if inv_freq is None:
        return x
    h = inv_freq.numel()
    angle = torch.outer(pos.double(), inv_freq.double())[:, None, :]
    spin = torch.polar(torch.full_like(angle, factor), angle)
    y = x.clone()
    if inter:
        z = torch.complex(x[..., 0:2 * h:2].contiguous(), x[..., 1:2 * h:2].contiguous()) * spin
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * spin
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
    return y


def _rms64(x, w):
    x = x.double()
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()


def _append64(x, cache, scale, s, P):
    """Values in units of their page's scale (not rounded to 8 bits), page by page of each sequence."""
    vals, out = cache.double(), scale.double()
    cu = [0] + torch.bincount(s["seq"], minlength=s["case"]["N"]).cumsum(0).tolist()
    table, lens = s["page_table"].tolist(), s["seq_lens"].tolist()
    peak = x.abs().amax(-1).cpu()
    was = scale.double().cpu()
    for n in range(len(lens)):
        t = cu[n]
        while t < cu[n + 1]:
            pos = lens[n] + t - cu[n]
            pg, row = table[n][pos // P], pos % P
            m = min(P - row, cu[n + 1] - t)
            top = peak[t:t + m].amax(0) / E4M3_MAX
            sc = torch.tensor([2.0 ** max(-100, math.ceil(math.log2(v))) if v > 0 else 2.0 ** -100 for v in top.tolist()],
                              dtype=torch.float64)
            if row:
                sc = torch.maximum(sc, was[pg])
                vals[pg, :, :row] *= (was[pg] / sc).to(vals.device)[:, None, None]
            sc = sc.to(vals.device)
            vals[pg, :, row:row + m] = (x[t:t + m] / sc[:, None]).transpose(0, 1)
            out[pg] = sc
            t += m
    return vals, out


def exact(case, seed):
    s = prepare(case, seed)
    inter = case.get("inter")
    if case["op"] == "norm_rope":
        return {n: _turn64(_rms64(s[n + "_raw"], s[n + "_weight"]), s["positions"], s["inv_freq"], inter, s["rope_scale"])
                for n in ("q", "k")}
    if case["op"] == "append":
        k = _turn64(_rms64(s["k_raw"], s["k_weight"]), s["pos"], s["inv_freq"], inter, 1.0)
        kv, ks = _append64(k, s["k_cache"], s["k_scale"], s, case["page"])
        vv, vs = _append64(s["v_raw"].double(), s["v_cache"], s["v_scale"], s, case["page"])
        return {"k": kv, "v": vv, "k_scale": ks, "v_scale": vs}
    d, G = case["d"], case["Hq"] // case["Hk"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "prefill":
        for a, b in zip(s["bounds"], s["bounds"][1:]):
            for h in range(case["Hq"]):
                k, v = s["k"][a:b, h // G].double(), s["v"][a:b, h // G].double()
                for lo in range(a, b, 4096):
                    hi = min(b, lo + 4096)
                    x = s["q"][lo:hi, h].double() @ k[:hi - a].T / math.sqrt(d)
                    gap = torch.arange(lo, hi, device="cuda")[:, None] - torch.arange(a, hi, device="cuda")
                    seen = (gap >= 0) & (gap < case["window"]) if case["window"] else gap >= 0
                    out[lo:hi, h] = torch.softmax(torch.where(seen, x, -math.inf), -1) @ v[:hi - a]
        return out
    P = case["page"]
    for n, L in enumerate(s["seq_lens"].tolist()):
        if L == 0:
            continue
        pages = s["page_table"][n, :(L + P - 1) // P].tolist()
        lo = max(0, L - case["window"]) if case["window"] else 0
        k, v = ((torch.cat([s[c + "_cache"][p].double() * s[c + "_scale"][p].double()[:, None, None] for p in pages], 1)
                 if len(pages) < 256 else
                 (s[c + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
                  * s[c + "_scale"][pages].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2))[:, lo:L]
                for c in "kv")
        x = s["q"][n].double().view(case["Hk"], G, d) @ k.transpose(1, 2).contiguous() / math.sqrt(d)
        out[n] = (torch.softmax(x, -1) @ v).reshape(case["Hq"], d)
    return out
