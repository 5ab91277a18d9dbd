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
