"""A hybrid's training and residual operators under the debug library libgdn_check.so
(LDS filled with NaN at kernel start, LDS accesses compared with the kernel's layout,
GDN_ERR_CHECK on a violation): cases of test_gpu_hybrid with that library in place of
libgdn.so."""
import ctypes
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import gated_delta_rule_gdn_amd.attn as attn  # noqa: E402
import gated_delta_rule_gdn_amd.gdn as binding  # noqa: E402
import gated_delta_rule_gdn_amd.hybrid as hybrid  # noqa: E402
import test_gpu_hybrid as th  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
CASES = {
    "attention bf16": lambda: th.test_attention_packed(4, 2, 128, 0, BF),
    "attention bf16, window": lambda: th.test_attention_packed(6, 2, 64, 20, BF),
    "attention fp32": lambda: th.test_attention_packed(4, 2, 128, 64, F32),
    "attention fp32, d 64": lambda: th.test_attention_packed(16, 1, 64, 0, F32),
    "attention, equal lengths": lambda: th.test_attention_equal_lengths_and_scales(3, 100, 0.3, BF),
    "attention, one long sequence": lambda: th.test_attention_one_long_sequence(1300, 4, 1, 128, 500, BF),
    "attention, one long sequence, d 64": lambda: th.test_attention_one_long_sequence(1500, 8, 1, 64, 0, BF),
    "attention, one long sequence, fp32": lambda: th.test_attention_one_long_sequence(1300, 4, 1, 128, 500, F32),
    "attention, few tiles, fp32": lambda: th.test_attention_few_tiles_of_many_keys(3, 3, 128, 0, F32),
    "attention, few tiles, fp32, d 64": lambda: th.test_attention_few_tiles_of_many_keys(6, 2, 64, 190, F32),
    "attention, many heads": lambda: th.test_attention_of_many_heads(32, 8, 128, 50, F32),
    "attention, many heads, d 64": lambda: th.test_attention_of_many_heads(48, 6, 64, 0, BF),
    "attention, fp32 gradients": lambda: th.test_attention_gradients_in_fp32_into_column_blocks(128),
    "attention, malformed offsets": th.test_attention_malformed_offsets_stay_in_bounds,
    "norm and rotation": lambda: th.test_norm_rope(33, 5, 1, 128, 128, False, BF, BF),
    "norm and rotation, many rows": lambda: th.test_norm_rope(2000, 1, 1, 64, 32, True, BF, F32),
    "residual, a wave to a row": lambda: th.test_add_norm(2048, BF, F32),
    "residual, a workgroup to a row": lambda: th.test_add_norm(5000, BF, BF),
    "residual backward, a wave to a row": lambda: th.test_add_norm_backward(1032, BF, F32),
    "residual backward, a workgroup to a row": lambda: th.test_add_norm_backward(8192, F32, F32),
}


@pytest.fixture(scope="module")
def check_library():
    path = os.path.join(os.path.dirname(binding.LIB_PATH), "libgdn_check.so")
    assert os.path.exists(path), f"{path} is missing: run the build"
    lib = ctypes.CDLL(path)
    attn._use(lib)
    hybrid._use(lib)
    yield
    attn._use(binding.lib)
    hybrid._use(binding.lib)


@pytest.mark.parametrize("case", list(CASES))
def test_parity_under_lds_checks(check_library, case):
    CASES[case]()
