"""What the check of gradients against differences can see: mistakes planted in the oracle's gradients."""
import numpy as np
import pytest
import torch

from attn_helpers import BF, F32
from hybrid_differences import check_attention_differences
from hybrid_helpers import attn_inputs
from oracle import hybrid as oh


def oracle(host, window, dtype):
    """The oracle's gradients, rounded as the operators round theirs."""
    return [torch.from_numpy(x).to(dtype).double().numpy() for x in oh.attention_backward(*host, window)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("Hq,Hk,d", [(4, 2, 64), (3, 1, 128)])
def test_the_formula_passes_and_mistakes_of_a_fifth_do_not(Hq, Hk, d, window, dtype):
    host = [t.contiguous() for t in attn_inputs(70, Hq, Hk, d, dtype, 12)]
    right = oracle(host, window, dtype)
    check_attention_differences(right, host, window, None, dtype, F32)
    for i in range(3):
        for wrong in (0.8, 1.2):
            got = [x.copy() for x in right]
            got[i][:, -1] *= wrong
            with pytest.raises(AssertionError):
                check_attention_differences(got, host, window, None, dtype, F32)
    got = [x.copy() for x in right]
    got[1][:, 0] = oh.attention_backward(host[0][:, :1], host[1][:, :1], host[2][:, :1], host[3][:, :1], window)[1][:, 0]
    with pytest.raises(AssertionError):     # one query head of a group instead of all
        check_attention_differences(got, host, window, None, dtype, F32)
    assert np.isfinite(got[1]).all()
