"""GPU tests of a hybrid's training and residual operators at the edges of their
documented ranges, as they are used (together, captured, on streams, in place), and of
what they refuse."""
import math

import numpy as np
import pytest
import torch

from attn_helpers import BF, F32, HALF, f64, gen, inv_freq, within
from helpers import TOL_BF16, TOL_FP32, announce, relerr
from hybrid_helpers import EPS, attn_grads, attn_inputs, check_attn, norm_grad_bound, rope_grads, views
from oracle import attention as oa
from oracle import hybrid as oh

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import gated_delta_rule_gdn_amd as gdn  # noqa: E402
import test_gpu_hybrid as th  # noqa: E402


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("window", [0, 9])
def test_attention_of_many_tiles(window, packed, dtype):
    """So many key tiles that each has a workgroup of its own: 1000 sequences, equal and of mixed lengths."""
    announce(f"attn backward many tiles window={window} packed={packed} {dtype}")
    N, Hk = 1000, 5
    lens = [(7 * i) % 41 for i in range(N)] if packed else [20] * N
    lens[3] = 20 + 130 * packed
    bounds = np.concatenate([[0], np.cumsum(lens)]).tolist()
    host, on = th.case(bounds[-1], 5, Hk, 64, dtype, 21)
    kw = dict(cu_seqlens=torch.tensor(bounds).cuda()) if packed else dict(N=N)
    _, _, got = th.both(on, window=window, **kw)
    torch.cuda.synchronize()
    some = [0, 1, 2, 3, 4, 499, 500, 997, 998, 999]
    for i in some:
        a, b = bounds[i], bounds[i + 1]
        check_attn([t[a:b] for t in got], [t[a:b] for t in host], [0, b - a], window, None, dtype, what=f"sequence {i}")
    assert all(bool(torch.isfinite(t).all()) for t in got)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_one_sequence_of_every_tile_edge(dtype):
    announce(f"attn backward tile edges {dtype}")
    for L in [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 95, 96, 97, 127, 128, 129, 191, 192, 193, 255, 256, 257]:
        host, on = th.case(L, 2, 1, 64, dtype, L)
        for window in (0, 33):
            _, _, got = th.both(on, window=window)
            torch.cuda.synchronize()
            check_attn(got, host, [0, L], window, None, dtype, what=f"L {L}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [2 ** 63 - 32, 2 ** 63 - 1])
def test_attention_windows_of_any_size(window, dtype):
    announce(f"attn backward window {window} {dtype}")
    _, on = th.case(500, 4, 2, 128, dtype, 9)
    for kw in (dict(), dict(cu_seqlens=torch.tensor([0, 70, 500]).cuda())):
        a, b = th.both(on, window=window, **kw)[2], th.both(on, **kw)[2]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_attention_ranges_that_overlap_stay_within_the_workspace():
    """Offsets that name all rows again and again have more tiles than there are rows: nothing behind the
    workspace or the outputs is written."""
    announce("attn backward overlapping ranges")
    T, Hq, Hk, d = 300, 2, 1, 64
    for dtype in (BF, F32):
        _, on = th.case(T, Hq, Hk, d, dtype, 4)
        for N in (40, 900):
            cu = torch.tensor([0, 10 ** 12] * (N // 2) + [T]).cuda()
            n = len(cu) - 1
            o, stats = gdn.gdn_attn_prefill_save(*on[:3], cu_seqlens=cu)
            need = gdn.gdn_attn_backward_workspace_size(on[0], on[1], N=n)
            ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
            outs = [torch.full((T + 8, h, d), 7.0, dtype=dtype, device="cuda") for h in (Hq, Hk, Hk)]
            gdn.gdn_attn_backward(*on[:3], o, on[3], stats, cu_seqlens=cu, dq=outs[0][:T], dk=outs[1][:T],
                                  dv=outs[2][:T], workspace=ws)
            torch.cuda.synchronize()
            assert bool((ws[need:] == 171).all()) and all(bool((t[T:] == 7).all()) for t in outs)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_far_values_touch_no_far_token(dtype):
    """A value that is not finite changes no gradient further than the window and 256 tokens from it."""
    announce(f"attn backward far values {dtype}")
    T, window, at = 1400, 100, 700
    host = [t.clone().contiguous() for t in attn_inputs(T, 2, 1, 64, dtype, 6)]
    clean = [t.cuda() for t in host]
    want = th.both(clean, window=window)[2]
    for i, bad in ((0, math.nan), (1, math.inf), (2, math.nan), (3, -math.inf)):
        on = [t.clone() for t in clean]
        on[i][at] = bad
        got = th.both(on, window=window)[2]
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[:at - window - 256], y[:at - window - 256])
            assert torch.equal(x[at + window + 256:], y[at + window + 256:])


def test_attention_workspace_is_the_callers():
    """A workspace of exactly the size, full of other bytes, gives the same bits; a shorter one is refused."""
    announce("attn backward workspace")
    for dtype in (BF, F32):
        _, on = th.case(700, 4, 1, 128, dtype, 3)
        o, stats, want = th.both(on)
        need = gdn.gdn_attn_backward_workspace_size(on[0], on[1])
        for fill in (0, 255):
            ws = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
            got = gdn.gdn_attn_backward(*on[:3], o, on[3], stats, workspace=ws[:need])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((ws[need:] == fill).all())
        with pytest.raises(gdn.GdnError):
            gdn.gdn_attn_backward(*on[:3], o, on[3], stats, workspace=ws[:need - 1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_beyond_32_bit_offsets(dtype):
    """Inputs and gradients more than 2^32 bytes into wide buffers."""
    announce(f"hybrid rows beyond 4 GiB {dtype}")
    ld, d = 1 << 17, 64
    T = (1 << 32) // (ld * dtype.itemsize) + 700
    x = torch.empty(T, ld, dtype=dtype, device="cuda")
    y = torch.zeros(T, ld, dtype=dtype, device="cuda")
    x[T - 600:, :4 * d] = torch.randn(600, 4 * d, generator=gen(3)).to(dtype).cuda()
    x[:T - 600, :4 * d] = 1.0

    def blocks(z):
        return z[:, :2 * d].unflatten(1, (2, d)), z[:, 2 * d:3 * d].unflatten(1, (1, d)), z[:, 3 * d:4 * d].unflatten(1, (1, d))

    q, k, v = blocks(x)
    dq, dk, dv = blocks(y)
    d_o = torch.randn(T, 2, d, generator=gen(4)).to(dtype).cuda()
    kw = dict(cu_seqlens=torch.tensor([0, T - 600, T - 250, T]).cuda(), window=300)
    o, stats = gdn.gdn_attn_prefill_save(q, k, v, **kw)
    gdn.gdn_attn_backward(q, k, v, o, d_o, stats, dq=dq, dk=dk, dv=dv, **kw)
    torch.cuda.synchronize()
    for a, b in ((T - 600, T - 250), (T - 250, T)):
        check_attn([t[a:b] for t in (dq, dk, dv)], [t[a:b].cpu() for t in (q, k, v, d_o)], [0, b - a], 300, None, dtype)
    assert bool((y[:, 4 * d:] == 0).all())
    pos, f, w = torch.arange(T).cuda(), inv_freq(d), 1 + 0.1 * torch.randn(d, generator=gen(5))
    up = torch.randn(T, 2, d, generator=gen(6)).to(dtype).cuda()
    gdn.gdn_qk_norm_rope_backward(up, None, q, positions=pos, inv_freq=f.cuda(), q_weight=w.cuda(), dq_raw=dq)
    torch.cuda.synchronize()
    (ref, bound), _ = rope_grads(q[T - 9:].cpu(), w, pos[T - 9:].cpu(), f, up[T - 9:].cpu(), False, 1.0, 1e-6, dtype)
    within(dq[T - 9:], ref, bound, "far norm_rope")
    # the same for the residual stream: rows of a wide buffer, and more than 2^31 elements in all
    C = 4096
    cols, wide = y[:, 8:8 + C], 1 + 0.1 * torch.randn(C, generator=gen(7))
    cols.copy_(torch.randn(T, C, generator=gen(8)).to(dtype))
    out, _, r = gdn.gdn_add_norm(cols, torch.ones(T, C, device="cuda").to(dtype), wide.cuda())
    torch.cuda.synchronize()
    ry, rr = oh.add_norm(cols[T - 5:].cpu(), np.ones((5, C)), wide, 1e-6)
    within(out[T - 5:], ry, (96 * EPS + HALF[dtype]) * np.abs(ry) + 1e-30, "far rows")
    within(r[T - 5:], rr, (EPS + HALF[dtype]) * np.abs(rr) + 1e-30, "far sums")


def test_residual_beyond_2_to_31_elements():
    announce("residual beyond 2^31 elements")
    rows, C = (1 << 31) // 4096 + 70, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    r = torch.randn(rows, C, generator=g, device="cuda", dtype=BF)
    dy = torch.randn(rows, C, generator=g, device="cuda", dtype=BF)
    w = torch.ones(C, device="cuda")
    y, s, out = gdn.gdn_add_norm(r, r, w, group=128)
    dx, _, _ = gdn.gdn_add_norm_backward(dy, r, w, d_res_out=r)
    torch.cuda.synchronize()
    at = slice(rows - 3, rows)
    ry, rr = oh.add_norm(r[at].cpu(), r[at].cpu(), None, 1e-6)
    z = ry.reshape(3, -1, 128)
    top = np.abs(z).max(-1) / 448
    within(s[at], top, 100 * EPS * top, "scale")
    z = (z / top[..., None]).reshape(3, C)
    within(y[at].float(), z, th.step_of(z) * (1 + 2.0 ** -10) + 256 * EPS * np.abs(z), "codes")
    within(out[at], rr, (EPS + HALF[BF]) * np.abs(rr) + 1e-30, "r")
    ref, _ = oh.add_norm_backward(dy[at].cpu(), r[at].cpu(), None, r[at].cpu(), 1e-6)
    bx, _ = norm_grad_bound(r[at].cpu(), np.ones(C), 1e-6, dy[at].cpu(), np.zeros(C))
    within(dx[at], ref, bx + 2 * EPS * (np.abs(f64(r[at])) + np.abs(ref)) + HALF[BF] * np.abs(ref), "dx")


# ----------------------------------------------------------------------------
# together, as a layer's training step uses them
# ----------------------------------------------------------------------------

class Layer:
    """A hybrid's attention layer between two additions to its residual stream."""

    def __init__(self, T, C, Hq, Hk, d, dtype, seed, lens):
        g = gen(seed)
        self.sizes, self.dtype, self.window = (Hq, Hk, d), dtype, 50
        self.bounds = np.concatenate([[0], np.cumsum(lens)]).tolist()
        p = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.host = dict(x=p(T, C), res=2 * p(T, C), w=1 + 0.1 * p(C), w2=1 + 0.1 * p(C), qw=1 + 0.1 * p(d), kw=1 + 0.1 * p(d),
                         proj=p((Hq + 2 * Hk) * d, C) / C ** 0.5, out=p(C, Hq * d) / (Hq * d) ** 0.5,
                         dy=p(T, C), dr=p(T, C))
        for n in ("x", "proj", "out", "dy"):
            self.host[n] = self.host[n].to(dtype)
        self.freq = inv_freq(d)
        self.pos = torch.cat([torch.arange(n) for n in lens])
        self.dev = {n: t.cuda() for n, t in self.host.items()}
        self.cu, self.fd, self.pd = torch.tensor(self.bounds).cuda(), self.freq.cuda(), self.pos.cuda()

    def step(self, io=None):
        """(y, r2) and all gradients, with the residual stream in fp32."""
        t, (Hq, Hk, d) = {**self.dev, **(io or {})}, self.sizes
        kw = dict(cu_seqlens=self.cu, window=self.window)
        h, _, r = gdn.gdn_add_norm(t["x"], t["res"], t["w"])
        qkv = h @ t["proj"].T
        q_raw, k_raw, v = views(qkv, Hq, Hk, d)
        rope = dict(positions=self.pd, inv_freq=self.fd, q_weight=t["qw"], k_weight=t["kw"])
        q, k = gdn.gdn_qk_norm_rope(q_raw, k_raw, **rope)
        o, stats = gdn.gdn_attn_prefill_save(q, k, v, **kw)
        a = o.flatten(1) @ t["out"].T
        y, _, r2 = gdn.gdn_add_norm(a, r, t["w2"])
        da, dr, dw2 = gdn.gdn_add_norm_backward(t["dy"], r2, t["w2"], d_res_out=t["dr"])
        do = (da @ t["out"]).unflatten(1, (Hq, d))
        dqkv = torch.empty_like(qkv)
        dq_raw, dk_raw, dv = views(dqkv, Hq, Hk, d)
        dq, dk, _ = gdn.gdn_attn_backward(q, k, v, o, do, stats, dv=dv, **kw)
        _, _, dqw, dkw = gdn.gdn_qk_norm_rope_backward(dq, dk, q_raw, k_raw, dq_raw=dq_raw, dk_raw=dk_raw, **rope)
        dh = dqkv @ t["proj"]
        dx, dres, dw = gdn.gdn_add_norm_backward(dh, r, t["w"], d_res_out=dr)
        return dict(y=y, r2=r2, dx=dx, dres=dres, dw=dw, dw2=dw2, dqw=dqw, dkw=dkw, dproj=dqkv.T @ h,
                    dout=da.T @ o.flatten(1))

    def reference(self):
        """The same by torch's own differentiation, on the host in 64 bits."""
        Hq, Hk, d = self.sizes
        p = {n: self.host[n].double().requires_grad_(n not in ("dy", "dr")) for n in self.host}

        def norm(x, w):
            return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

        def turned(x):
            angle = self.pos.double()[:, None] * self.freq.double()
            c, s = angle.cos()[:, None], angle.sin()[:, None]
            a, b = x[..., :d // 2], x[..., d // 2:]
            return torch.cat((a * c - b * s, b * c + a * s), -1)

        r = p["x"] + p["res"]
        qkv = norm(r, p["w"]) @ p["proj"].T
        q_raw, k_raw, v = views(qkv, Hq, Hk, d)
        q, k = turned(norm(q_raw, p["qw"])), turned(norm(k_raw, p["kw"]))
        k, v = k.repeat_interleave(Hq // Hk, 1), v.repeat_interleave(Hq // Hk, 1)
        o = []
        for a, b in zip(self.bounds, self.bounds[1:]):
            gap = torch.arange(b - a)[:, None] - torch.arange(b - a)
            s = torch.einsum("thc,shc->hts", q[a:b], k[a:b]) * d ** -0.5
            s = s.masked_fill((gap < 0) | (gap >= self.window), -math.inf)
            o.append(torch.einsum("hts,shc->thc", torch.softmax(s, -1), v[a:b]))
        r2 = r + torch.cat(o).flatten(1) @ p["out"].T
        y = norm(r2, p["w2"])
        ((y * p["dy"]).sum() + (r2 * p["dr"]).sum()).backward()
        g = {n: p[n].grad for n in p}
        return dict(y=y.detach(), r2=r2.detach(), dx=g["x"], dres=g["res"], dw=g["w"], dw2=g["w2"], dqw=g["qw"], dkw=g["kw"],
                    dproj=g["proj"], dout=g["out"])


@pytest.mark.parametrize("dtype,d", [(F32, 64), (F32, 128), (BF, 64), (BF, 128)])
def test_a_layers_training_step(dtype, d):
    """All of the operators in one step against differentiation of the whole layer in 64 bits, at the
    tolerances of the precision."""
    announce(f"layer step {dtype} d={d}")
    lens = [150, 1, 77, 0, 130]
    layer = Layer(sum(lens), 256, 4, 2, d, dtype, 31, lens)
    got = layer.step()
    torch.cuda.synchronize()
    ref = layer.reference()
    for n in ref:
        e = relerr(got[n], ref[n])
        assert e <= (TOL_FP32 if dtype == F32 else TOL_BF16), (n, e)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_captured_training_step_replays(dtype):
    """The step captured into a graph and replayed with new inputs, eager work between the replays."""
    announce(f"captured layer step {dtype}")
    lens = [200, 3, 300]
    layer = Layer(sum(lens), 256, 4, 2, 128, dtype, 8, lens)
    layer.step()
    torch.cuda.synchronize()
    io = {n: layer.dev[n].clone() for n in ("x", "dy", "dr")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.step(io)
    for i in range(4):
        for n in io:
            io[n].copy_(torch.randn(io[n].shape, generator=gen(50 + i)).to(io[n].dtype))
        graph.replay()
        torch.cuda.synchronize()
        want = layer.step({n: t.clone() for n, t in io.items()})
        torch.cuda.synchronize()
        for n in want:
            if n in ("dproj", "dout"):
                continue                    # library products, not what is tested
            assert torch.equal(got[n], want[n]), (i, n)


def test_two_captured_graphs_with_a_workspace_each():
    announce("two graphs of backward passes")
    graphs = []
    for i, dtype in enumerate((BF, F32)):
        _, on = th.case(600 + 40 * i, 4, 1, 128, dtype, i)
        o, stats, want = th.both(on)
        ws = torch.empty(gdn.gdn_attn_backward_workspace_size(on[0], on[1]), dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(t) for t in want]
        torch.cuda.synchronize()
        call = lambda on=on, o=o, stats=stats, outs=outs, **kw: gdn.gdn_attn_backward(  # noqa: E731
            *on[:3], o, on[3], stats, dq=outs[0], dk=outs[1], dv=outs[2], **kw)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(workspace=ws)
        graphs.append((g, outs, want, call))
    for r in range(3):
        for g, outs, want, call in graphs:
            for t in outs:
                t.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, outs, want, call in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), r
            call()


def test_streams_and_raw_handles():
    """Work on a stream other than the current one, given as a stream and as a handle; what the calls
    allocate belongs to that stream."""
    announce("hybrid streams")
    layers = [Layer(500, 256, 4, 2, 128, dtype, 3, [300, 200]) for dtype in (BF, F32)]
    s = torch.cuda.Stream()
    for layer in layers:
        t, (Hq, Hk, d) = layer.dev, layer.sizes
        h, _, r = gdn.gdn_add_norm(t["x"], t["res"], t["w"])
        q, k, v = [x.contiguous() for x in views(h @ t["proj"].T, Hq, Hk, d)]

        def run(**kw):
            o, stats = gdn.gdn_attn_prefill_save(q, k, v, cu_seqlens=layer.cu, **kw)
            g = gdn.gdn_attn_backward(q, k, v, o, q, stats, cu_seqlens=layer.cu, **kw)
            n = gdn.gdn_qk_norm_rope_backward(g[0], g[1], q, k, positions=layer.pd, inv_freq=layer.fd, q_weight=t["qw"],
                                              k_weight=t["kw"], **kw)
            e = gdn.gdn_add_norm(t["x"], t["res"], t["w"], group=64, **kw)
            b = gdn.gdn_add_norm_backward(t["dy"], r, t["w"], d_res_out=t["dr"], **kw)
            return [o, stats, *g, *n, *e, *b]

        want = run()
        torch.cuda.synchronize()
        for stream in (s, s.cuda_stream):
            for _ in range(6):
                got = run(stream=stream)
                s.synchronize()
                assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_calls_on_two_streams_at_once():
    announce("hybrid two streams at once")
    layers = [Layer(700 + 100 * i, 256, 4, 2, 128, BF, i, [400, 300 + 100 * i]) for i in range(2)]
    skip = ("dproj", "dout")
    want = [layer.step() for layer in layers]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layers[i].step())
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(g[n], want[i][n]) for n in g if n not in skip)


def test_results_are_the_same_every_time():
    announce("hybrid bitwise repeatable")
    for dtype in (BF, F32):
        layer = Layer(900, 512, 8, 2, 64, dtype, 2, [640, 260])
        a = layer.step()
        for _ in range(4):
            b = layer.step()
            torch.cuda.synchronize()
            assert all(torch.equal(a[n], b[n]) for n in a if n not in ("dproj", "dout"))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_against_differences(dtype):
    """Directional derivatives of the forward calls themselves: L(x + h u) - L(x - h u) over 2 h, in 64-bit
    sums of their outputs, against the gradient calls. In fp32 L is off by its outputs' roundings (2^-24 of
    sum |o g| each, and as much again within), which the step divides; in bf16 by 2^-8 of them."""
    announce(f"differences {dtype}")
    T, Hq, Hk, d = 70, 4, 2, 64
    host = attn_inputs(T, Hq, Hk, d, F32, 12)
    q, k, v, g = [t.contiguous().to(dtype).cuda() for t in host]
    o, stats = gdn.gdn_attn_prefill_save(q, k, v)
    grads = gdn.gdn_attn_backward(q, k, v, o, g, stats, grad_dtype=F32)
    size = float((o.double() * g.double()).abs().sum())
    for i, x in enumerate((q, k, v)):
        u = torch.randn(x.shape, generator=gen(60 + i)).cuda()
        h = 2.0 ** -6 if dtype == F32 else 2.0 ** -2
        ends = []
        for sign in (1, -1):
            y = (x.float() + sign * h * u).to(dtype)
            args = [q, k, v]
            args[i] = y
            ends.append((y.double(), float((gdn.gdn_attn_prefill(*args).double() * g.double()).sum())))
        moved = ends[0][0] - ends[1][0]     # as the inputs' type took it
        got = float((grads[i].double() * moved).sum())
        want = ends[0][1] - ends[1][1]
        # third-order term of the difference: of the order of h^2 of the first, times the scores' change (below 8)
        slack = 64 * HALF[dtype] * size / math.sqrt(T * Hq * d) + 8 * h * h * float((grads[i].double() * moved).abs().sum()) / math.sqrt(x.numel())
        assert abs(got - want) <= slack, (i, got, want, slack)


# ----------------------------------------------------------------------------
# refusals
# ----------------------------------------------------------------------------

def test_binding_refusals():
    announce("hybrid refusals")
    _, (q, k, v, g) = th.case(20, 4, 2, 64, BF, 1)
    q, k, v = [t.contiguous() for t in (q, k, v)]
    o, stats = gdn.gdn_attn_prefill_save(q, k, v)
    x, w = torch.zeros(6, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")

    def refused(call, what):
        with pytest.raises(ValueError, match=what):
            call()

    back = lambda **kw: gdn.gdn_attn_backward(*[kw.pop(n, t) for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("g", g), ("s", stats))], **kw)  # noqa: E731,E501
    refused(lambda: gdn.gdn_attn_prefill_save(q, k, v, stats=stats[:-1]), "stats has shape")
    refused(lambda: gdn.gdn_attn_prefill_save(q, k, v, stats=stats.to(BF)), "stats must be torch.float32")
    refused(lambda: back(o=o.float()), "o must be")
    refused(lambda: back(g=g[:19]), "d_o has shape")
    refused(lambda: back(s=stats.view(20, -1)), "stats has shape")
    refused(lambda: back(dq=torch.empty_like(q).transpose(1, 2).contiguous().transpose(1, 2)), "dq must have dense rows")
    refused(lambda: back(dq=torch.empty_like(q), dk=torch.empty(k.shape, device="cuda")), "dk must be")
    refused(lambda: back(grad_dtype=torch.float16), "float32 or bfloat16")
    refused(lambda: back(cu_seqlens=torch.tensor([0, 20], dtype=torch.int32).cuda()), "cu_seqlens must be")
    refused(lambda: back(window=1.5), "window must be")
    refused(lambda: gdn.gdn_qk_norm_rope_backward(q, None, q, k), "without dk")
    refused(lambda: gdn.gdn_qk_norm_rope_backward(q, None, q.float()[:, :2]), "q_raw has shape")
    refused(lambda: gdn.gdn_qk_norm_rope_backward(q, None, inv_freq=inv_freq(64).cuda()), "rotation needs positions")
    refused(lambda: gdn.gdn_qk_norm_rope_backward(q[:, :, :32], None), "contiguous")
    refused(lambda: gdn.gdn_add_norm(x, x.float()[:5]), "res has shape")
    refused(lambda: gdn.gdn_add_norm(x, weight=w.to(BF)), "weight must be")
    refused(lambda: gdn.gdn_add_norm(x.t()), "dense rows")
    refused(lambda: gdn.gdn_add_norm(x.half()), "float32 or bfloat16")
    refused(lambda: gdn.gdn_add_norm(x, group=48), "group must be")
    refused(lambda: gdn.gdn_add_norm(x, group=-3), "group must be")
    refused(lambda: gdn.gdn_add_norm(x, y_scale=w), "without group")
    refused(lambda: gdn.gdn_add_norm(x, group=0, y=torch.empty_like(x)), "y must be torch.float8_e4m3fn")
    refused(lambda: gdn.gdn_add_norm_backward(x, x[:, :32]), "r has shape")
    refused(lambda: gdn.gdn_add_norm_backward(x, x, d_res_out=x.float()), "d_res_out must be")
    refused(lambda: gdn.gdn_add_norm_backward(x[:, ::2], x[:, ::2]), "contiguous")
    for call, status in ((lambda: back(scale=1e-30), gdn.GDN_ERR_UNSUPPORTED), (lambda: back(scale=0.0), gdn.GDN_ERR_INVALID_ARG),
                         (lambda: gdn.gdn_add_norm(x[:, :60].contiguous()), gdn.GDN_ERR_INVALID_ARG),
                         (lambda: gdn.gdn_add_norm(x, group=16), gdn.GDN_ERR_UNSUPPORTED),
                         (lambda: gdn.gdn_add_norm(x, x, y=x, res_out=x), gdn.GDN_ERR_INVALID_ARG),
                         (lambda: gdn.gdn_add_norm(x.float(), x), gdn.GDN_ERR_UNSUPPORTED)):
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert e.value.status == status


def test_no_memory_for_outputs():
    """Outputs and workspaces that the calls allocate: torch's error, and the next call works."""
    announce("hybrid out of memory")
    x = torch.randn(1 << 14, 1024, device="cuda")
    w = torch.ones(1024, device="cuda")
    want = gdn.gdn_add_norm(x[:8], x[:8], w)[0].clone()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 20)) / total)
    kept = []
    try:
        for size in (1 << 30, 1 << 26, 1 << 23, 1 << 21):     # what the allocator holds
            with pytest.raises(torch.OutOfMemoryError):
                while True:
                    kept.append(torch.empty(size, dtype=torch.uint8, device="cuda"))
        for call in (lambda: gdn.gdn_add_norm(x, x, w), lambda: gdn.gdn_add_norm_backward(x, x, w),
                     lambda: gdn.gdn_qk_norm_rope_backward(x.view(-1, 8, 128), None, x.view(-1, 8, 128)),
                     lambda: gdn.gdn_attn_prefill_save(*[x.view(-1, 8, 128)] * 3)):
            with pytest.raises(torch.OutOfMemoryError):
                call()
    finally:
        kept.clear()
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(gdn.gdn_add_norm(x[:8], x[:8], w)[0], want)
