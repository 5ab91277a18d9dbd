"""GPU tests of the residual's operators over the magnitudes that include/gdn_hybrid.h
allows: rows whose squares add up past fp32, rows next to nothing, and gradients that are not finite."""
import numpy as np
import pytest
import torch

from attn_helpers import BF, F32, HALF, gen, within
from helpers import announce
from hybrid_helpers import EPS, norm_grad_bound
from oracle import hybrid as oh

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import gated_delta_rule_gdn_amd as gdn  # noqa: E402
import test_gpu_hybrid as th  # noqa: E402

TYPES = [(BF, BF), (BF, F32), (F32, F32)]
WIDTHS = [256, 512, 1024, 1536, 2048, 4096, 8192, 16384]      # every number of waves and chunks of a row
LARGE = 2.0 ** 60 * (1 - 2.0 ** -7)                           # the largest that both types hold below 2^60


def rows_of(C, seed):
    """Rows of one magnitude each, from the largest down, ordinary ones between them; the first has no other value."""
    g = gen(seed)
    x = 2 * torch.rand(9, C, generator=g) - 1
    x = torch.sign(x) * (0.5 + x.abs() / 2)
    x[0] = 1
    size = torch.tensor([LARGE, 1.0, LARGE, 2.0 ** 58, 2.0 ** 57, 3.0, 2.0 ** 56, 2.0 ** 40, LARGE])
    return size[:, None] * x


@pytest.mark.parametrize("io,rt", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_add_norm_of_large_rows(C, io, rt):
    """Bounds as for ordinary rows: a power of two on a row changes no rounding."""
    announce(f"add_norm large C={C} {io} {rt}")
    x = rows_of(C, C)
    res, x = (0.25 * x).to(rt), (0.75 * x).to(io)
    w = 1 + 0.1 * torch.randn(C, generator=gen(C + 1))
    ry, rr = oh.add_norm(x, res, w, 1e-6)
    y, _, r = gdn.gdn_add_norm(x.cuda(), res.cuda(), w.cuda())
    torch.cuda.synchronize()
    within(y, ry, (96 * EPS + HALF[io]) * np.abs(ry), "y")
    within(r, rr, (EPS + HALF[rt]) * np.abs(rr), "r")
    for group in (0, 128):
        y, scale, r = gdn.gdn_add_norm(x.cuda(), res.cuda(), w.cuda(), group=group)
        z = ry.reshape(len(x), -1, group or C)
        top = np.abs(z).max(-1) / 448
        within(scale, top, 100 * EPS * top, "scale")
        z = (z / top[..., None]).reshape(len(x), C)
        within(y.float(), z, th.step_of(z) * (1 + 2.0 ** -10) + 256 * EPS * np.abs(z), "codes")
        within(r, rr, (EPS + HALF[rt]) * np.abs(rr), "r")


@pytest.mark.parametrize("io,rt", TYPES)
@pytest.mark.parametrize("C", WIDTHS)
def test_add_norm_backward_of_large_rows(C, io, rt):
    """Large rows with ordinary gradients, and with gradients as large that follow the row, so that
    their products add up past fp32 too."""
    announce(f"add_norm backward large C={C} {io} {rt}")
    r = rows_of(C, C).to(rt)
    w = 1 + 0.1 * (2 * torch.rand(C, generator=gen(C + 1)) - 1)
    for dy in (torch.randn(r.shape, generator=gen(C + 2)), 0.75 * r.float()):
        dy = dy.to(io)
        ref, refw = oh.add_norm_backward(dy, r, w, None, 1e-6)
        bx, bw = norm_grad_bound(r, w, 1e-6, dy, np.zeros(C), K=160)
        dx, d_res, dw = gdn.gdn_add_norm_backward(dy.cuda(), r.cuda(), w.cuda())
        torch.cuda.synchronize()
        within(dx, ref, bx + HALF[io] * np.abs(ref), "dx")
        within(d_res, ref, bx + HALF[rt] * np.abs(ref), "d_res")
        within(dw, refw, bw, "d_weight")


@pytest.mark.parametrize("C", [512, 2048, 16384])
def test_add_norm_of_small_rows_without_eps(C):
    """eps 0 and means of squares at the smallest that a norm takes, 2^-126."""
    announce(f"add_norm small C={C}")
    x = torch.sign(torch.randn(4, C, generator=gen(C))) * 2.0 ** -63
    x[1] *= 1.5
    x[2] *= 2.0 ** 20
    w = torch.ones(C)
    ry, _ = oh.add_norm(x, None, w, 0.0)
    y, _, _ = gdn.gdn_add_norm(x.cuda(), None, w.cuda(), eps=0.0)
    dy = torch.randn(4, C, generator=gen(1))
    ref, refw = oh.add_norm_backward(dy, x, w, None, 0.0)
    bx, bw = norm_grad_bound(x, w, 0.0, dy, np.zeros(C), K=160)
    dx, _, dw = gdn.gdn_add_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=0.0)
    torch.cuda.synchronize()
    within(y, ry, (96 * EPS + HALF[F32]) * np.abs(ry), "y")
    within(dx, ref, bx + HALF[F32] * np.abs(ref), "dx")
    within(dw, refw, bw, "d_weight")


@pytest.mark.parametrize("C", [64, 2048])
def test_rows_of_zeros_with_an_eps_below_normal_numbers(C):
    announce(f"add_norm zeros C={C}")
    eps = 1e-40
    x, w, dy = torch.zeros(3, C), torch.ones(C), torch.randn(3, C, generator=gen(C))
    x[1] = 2.0 ** -66
    ry, _ = oh.add_norm(x, None, w, eps)
    ref, refw = oh.add_norm_backward(dy, x, w, None, eps)
    # eps has 16 bits there: off by 2^-17 of itself, the root of the sum by half of that
    part = eps / (np.mean(np.float64(x.numpy()) ** 2, 1, keepdims=True) + eps) * 2.0 ** -18
    bx, bw = norm_grad_bound(x, w, eps, dy, np.zeros(C), K=160)
    y, _, _ = gdn.gdn_add_norm(x.cuda(), None, w.cuda(), eps=eps)
    dx, _, dw = gdn.gdn_add_norm_backward(dy.cuda(), x.cuda(), w.cuda(), eps=eps)
    torch.cuda.synchronize()
    within(y, ry, (96 * EPS + HALF[F32] + part) * np.abs(ry), "y")
    n = np.abs(ry)
    size = (np.abs(dy.numpy()) + 2 * n * np.mean(n * np.abs(dy.numpy()), -1, keepdims=True)) * np.abs(1 / np.sqrt(eps))
    within(dx, ref, bx + HALF[F32] * np.abs(ref) + 3 * part * size, "dx")
    within(dw, refw, bw + (3 * part * n * np.abs(dy.numpy())).sum(0), "d_weight")


@pytest.mark.parametrize("io,rt", TYPES)
@pytest.mark.parametrize("C", [512, 2048])
def test_gradients_that_are_not_finite_stay_in_their_rows_and_channels(C, io, rt):
    announce(f"add_norm backward not finite C={C} {io} {rt}")
    g = gen(C)
    r, dy, w = (3 * torch.randn(6, C, generator=g)).to(rt).cuda(), torch.randn(6, C, generator=g).to(io).cuda(), torch.ones(C).cuda()
    want = gdn.gdn_add_norm_backward(dy, r, w)
    dy[2, 5], dy[4, 7] = float("nan"), float("inf")
    dx, d_res, dw = gdn.gdn_add_norm_backward(dy, r, w)
    torch.cuda.synchronize()
    rows, channels = [0, 1, 3, 5], [c for c in range(C) if c not in (5, 7)]
    assert torch.equal(dx[rows], want[0][rows]) and torch.equal(d_res[rows], want[1][rows])
    assert torch.equal(dw[channels], want[2][channels]) and not bool(torch.isfinite(dw[[5, 7]]).any())


@pytest.mark.parametrize("heads", [2, 16384])
def test_no_rows_of_many_heads_give_zero_weight_gradients(heads):
    announce(f"no rows, {heads} heads")
    h, w = torch.zeros(0, heads, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    r = gdn.gdn_qk_norm_rope_backward(h, None, h, q_weight=w, dq_weight=torch.full((64,), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert bool((r[2] == 0).all())
