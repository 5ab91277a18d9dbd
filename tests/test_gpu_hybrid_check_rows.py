"""The rows' operators under the debug library libgdn_check.so in every form of a row: one
wave and four, each number of chunks, codes, sums that are formed again, and joins."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import test_gpu_hybrid as th  # noqa: E402
import test_gpu_hybrid_ranges as tr  # noqa: E402
from test_gpu_hybrid_check import check_library  # noqa: E402,F401

BF, F32 = torch.bfloat16, torch.float32
CASES = {f"residual {C}": lambda C=C: th.test_add_norm(C, BF, F32) for C in (72, 512, 1024, 1032, 1536, 1544, 2048, 4096, 16384)}
CASES.update({f"residual backward {C}": lambda C=C: th.test_add_norm_backward(C, BF, BF)
              for C in (72, 512, 520, 1024, 1536, 1544, 2048, 4096, 16384)})
CASES.update({f"large rows {C}": lambda C=C: (tr.test_add_norm_of_large_rows(C, F32, F32),
                                              tr.test_add_norm_backward_of_large_rows(C, F32, F32)) for C in (1024, 2048)})
CASES.update({f"a small eps {C}": lambda C=C: tr.test_rows_of_zeros_with_an_eps_below_normal_numbers(C) for C in (64, 2048)})
CASES["many rows"] = th.test_add_norm_backward_in_place_and_many_rows
CASES["no rows"] = th.test_no_rows_give_zero_weight_gradients


@pytest.mark.parametrize("case", list(CASES))
def test_parity_under_lds_checks(check_library, case):  # noqa: F811
    CASES[case]()
