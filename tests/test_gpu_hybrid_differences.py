"""GPU: the attention's gradients against differences of the forward formula in 64 bits."""
import pytest
import torch

from attn_helpers import BF, F32
from helpers import announce
from hybrid_differences import check_attention_differences

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import test_gpu_hybrid as th  # noqa: E402


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hk,d,window,scale", [(70, 4, 2, 64, 0, None), (70, 4, 2, 64, 20, None), (150, 3, 1, 128, 0, 0.1),
                                                    (150, 2, 2, 128, 33, -0.1)])
def test_gradients_along_themselves(T, Hq, Hk, d, window, scale, dtype):
    announce(f"differences in 64 bits T={T} Hq={Hq} Hk={Hk} d={d} window={window} scale={scale} {dtype}")
    host, on = th.case(T, Hq, Hk, d, dtype, 12)
    got = th.both(on, window=window, scale=scale, grad_dtype=F32)[2]
    torch.cuda.synchronize()
    check_attention_differences([t.cpu() for t in got], host, window, scale, dtype, F32)
