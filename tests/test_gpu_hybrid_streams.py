"""GPU: refusals of a hybrid's operators when a stream is given are those of the same calls without one."""
import pytest
import torch

from attn_helpers import BF, inv_freq
from helpers import announce

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import gated_delta_rule_gdn_amd as gdn  # noqa: E402
import test_gpu_hybrid as th  # noqa: E402


def calls():
    _, (q, k, v, g) = th.case(20, 4, 2, 64, BF, 1)
    q, k, v = [t.contiguous() for t in (q, k, v)]
    o, stats = gdn.gdn_attn_prefill_save(q, k, v)
    x = torch.zeros(6, 64, dtype=BF, device="cuda")
    save = lambda *a, **kw: lambda **s: gdn.gdn_attn_prefill_save(*a, **kw, **s)  # noqa: E731
    back = lambda *a, **kw: lambda **s: gdn.gdn_attn_backward(*a, **kw, **s)  # noqa: E731
    rope = lambda *a, **kw: lambda **s: gdn.gdn_qk_norm_rope_backward(*a, **kw, **s)  # noqa: E731
    norm = lambda *a, **kw: lambda **s: gdn.gdn_add_norm(*a, **kw, **s)  # noqa: E731
    nback = lambda *a, **kw: lambda **s: gdn.gdn_add_norm_backward(*a, **kw, **s)  # noqa: E731
    return {
        "q of 2 dimensions": save(q[0], k, v), "q of another type": save(q.half(), k, v), "k of 1 dimension": save(q, k[0, 0], v),
        "q is a list": save([1], k, v), "k is None": save(q, None, v), "save, window": save(q, k, v, window=1.5),
        "back, q of 2 dimensions": back(q[0], k, v, o, g, stats), "back, k of 1 dimension": back(q, k[0, 0], v, o, g, stats),
        "back, offsets in a list": back(q, k, v, o, g, stats, cu_seqlens=[0, 20]),
        "back, offsets a number": back(q, k, v, o, g, stats, cu_seqlens=20), "back, N": back(q, k, v, o, g, stats, N="x"),
        "back, window": back(q, k, v, o, g, stats, window=1.5), "back, k is None": back(q, None, v, o, g, stats),
        "back, dq of another type": back(q, k, v, o, g, stats, dq=torch.empty_like(q).half()),
        "rope, 1 dimension": rope(q[0, 0], None), "rope, dk is a number": rope(q, 3), "rope, type": rope(q.half(), None),
        "rope, weight is a number": rope(q, None, q, q_weight=1.0), "rope, no positions": rope(q, None, inv_freq=inv_freq(64).cuda()),
        "norm, 1 dimension": norm(x[0], group=0), "norm, negative group": norm(x, group=-3), "norm, a group of 1.5": norm(x, group=1.5),
        "norm, a group of text": norm(x, group="x"), "norm, res is a number": norm(x, 1.0), "norm, x is a list": norm([1], group=0),
        "norm back, 1 dimension": nback(x[0], x[0]), "norm back, r is None": nback(x, None), "norm back, r is a number": nback(x, 2),
        "norm back, weight is a number": nback(x, x, 1.0), "norm back, types": nback(x.half(), x),
    }


@pytest.mark.parametrize("case", [
    "q of 2 dimensions", "q of another type", "k of 1 dimension", "q is a list", "k is None", "save, window",
    "back, q of 2 dimensions", "back, k of 1 dimension", "back, offsets in a list", "back, offsets a number", "back, N",
    "back, window", "back, k is None", "back, dq of another type", "rope, 1 dimension", "rope, dk is a number", "rope, type",
    "rope, weight is a number", "rope, no positions", "norm, 1 dimension", "norm, negative group", "norm, a group of 1.5",
    "norm, a group of text", "norm, res is a number", "norm, x is a list", "norm back, 1 dimension", "norm back, r is None",
    "norm back, r is a number", "norm back, weight is a number", "norm back, types"])
def test_refusals_are_value_errors_with_and_without_a_stream(case):
    announce(f"refusal: {case}")
    call, s = calls()[case], torch.cuda.Stream()
    texts = []
    for kw in ({}, {"stream": s}, {"stream": s.cuda_stream}):
        with pytest.raises(ValueError) as e:
            call(**kw)
        texts.append(str(e.value))
    assert texts[0] == texts[1] == texts[2]


def test_what_a_call_with_a_stream_allocates_belongs_to_it():
    """The current stream is as it was behind such a call, and the outputs' memory is that stream's: freed, it is given
    out there again, and not here."""
    announce("allocations on a given stream")
    x, w = torch.randn(4000, 1024, device="cuda"), torch.ones(1024, device="cuda")
    want = gdn.gdn_add_norm(x, x, w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    here, s = torch.cuda.current_stream(), torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        y, _, r = gdn.gdn_add_norm(x, x, w, stream=stream)
        s.synchronize()
        assert torch.cuda.current_stream() == here
        assert torch.equal(y, want[0]) and torch.equal(r, want[2])
        at = {y.data_ptr(), r.data_ptr()}
        del y, r
        mine = [torch.empty_like(x) for _ in range(2)]
        assert not at & {t.data_ptr() for t in mine}
        with torch.cuda.stream(s):
            theirs = [torch.empty_like(x) for _ in range(2)]
        assert at & {t.data_ptr() for t in theirs}
        del mine, theirs


def test_default_stream_given_as_a_handle():
    """Stream 0, as a number, from within another stream."""
    announce("hybrid stream 0")
    x, w = torch.randn(40, 256, device="cuda"), torch.ones(256, device="cuda")
    want = gdn.gdn_add_norm(x, x, w)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = gdn.gdn_add_norm(x, x, w, stream=0)
    torch.cuda.default_stream().synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_every_argument_goes_with_a_stream_where_it_goes_without():
    """None left at its default, and outputs and workspaces given."""
    announce("hybrid, all arguments with a stream")
    (_, (q, k, v, g)), s = th.case(40, 4, 2, 64, BF, 3), torch.cuda.Stream()
    cu, pos, freq = torch.tensor([0, 15, 40]).cuda(), torch.arange(7, 47).cuda(), inv_freq(32).cuda()
    w = [1 + 0.1 * torch.randn(64, device="cuda") for _ in range(2)]
    x, res, wide = torch.randn(40, 128, device="cuda").to(BF), torch.randn(40, 128, device="cuda"), torch.rand(128, device="cuda")
    empty = lambda t, dtype=None: torch.empty(t.shape, dtype=dtype or t.dtype, device="cuda")  # noqa: E731
    bytes_ = lambda n: torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")  # noqa: E731
    F = torch.float32

    def run(**kw):
        o, stats = gdn.gdn_attn_prefill_save(q, k, v, cu, 2, 9, 0.2, empty(q), torch.empty(40 * 4 * 18, device="cuda"), **kw)
        grads = gdn.gdn_attn_backward(q, k, v, o, g, stats, cu, 2, 9, 0.2, empty(q, F), empty(k, F), empty(v, F), F,
                                      bytes_(gdn.gdn_attn_backward_workspace_size(q, k, 2, 9)), **kw)
        rope = gdn.gdn_qk_norm_rope_backward(grads[0], grads[1], q, k, pos, freq, w[0], w[1], True, 1.5, 1e-3, empty(q, F),
                                             empty(k, F), empty(w[0]), empty(w[1]),
                                             bytes_(gdn.gdn_qk_norm_rope_backward_workspace_size(grads[0], grads[1])), **kw)
        codes = gdn.gdn_add_norm(x, res, wide, 1e-3, 64, empty(res), empty(x, torch.float8_e4m3fn),
                                 torch.empty(40, 2, device="cuda"), **kw)
        back = gdn.gdn_add_norm_backward(x, codes[2], wide, res, 1e-3, empty(x), empty(res), empty(wide),
                                         bytes_(gdn.gdn_add_norm_backward_workspace_size(x)), **kw)
        return [o, stats, *grads, *rope, *codes, *back]

    want = run()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = run(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(got, want))
