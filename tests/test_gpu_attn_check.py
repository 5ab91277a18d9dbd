"""The attention operators under the debug library libgdn_check.so (LDS filled
with NaN at kernel start, LDS accesses compared with the kernel's layout,
GDN_ERR_CHECK on a violation): cases of test_gpu_attn with that library in
place of libgdn.so."""
import ctypes
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU hosts, skipped there
    pytest.skip("needs a GPU", allow_module_level=True)

import gated_delta_rule_gdn_amd.attn as attn  # noqa: E402
import gated_delta_rule_gdn_amd.gdn as binding  # noqa: E402
import test_gpu_attn as ta  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
CASES = {
    "norm and rotation": lambda: ta.test_norm_rope(33, 5, 1, 128, 128, False, BF),
    "append, pages of 16": lambda: ta.test_append_packed(16, 64, 3, True, BF),
    "append, pages of 128": lambda: ta.test_append_packed(128, 64, 2, False, F32),
    "append, bad pages": ta.test_append_bad_tables_and_lengths_write_only_what_they_name,
    "prefill bf16": lambda: ta.test_prefill_packed(4, 2, 128, 0, BF),
    "prefill bf16, window": lambda: ta.test_prefill_packed(16, 1, 64, 20, BF),
    "prefill fp32": lambda: ta.test_prefill_packed(4, 2, 128, 64, F32),
    "prefill, equal lengths": lambda: ta.test_prefill_equal_lengths_and_scales(3, 100, BF),
    "prefill, few long prompts": lambda: ta.test_prefill_few_long_prompts(4, 2, 128, 300),
    "prefill, few long prompts, d 64": lambda: ta.test_prefill_few_long_prompts(3, 3, 64, 0),
    "prefill fp32, few and many tiles": lambda: ta.test_prefill_fp32_few_and_many_tiles(3, 3, 64, 65),
    "prefill, unseen values": lambda: ta.test_prefill_values_that_a_query_does_not_see(400, 128, 40, BF),
    "prefill, malformed offsets": ta.test_prefill_malformed_offsets_stay_in_bounds,
    "decode bf16": lambda: ta.test_decode(21, 3, 128, 64, 0, BF),
    "decode fp32, window": lambda: ta.test_decode(4, 2, 128, 16, 50, F32),
    "decode, one long sequence": lambda: ta.test_decode_one_long_sequence(BF),
    "decode, NaN behind the last token": lambda: ta.test_decode_ignores_what_lies_behind_the_last_token(BF),
    "prompt, then decode steps": lambda: ta.test_prompt_then_decode_steps(24, BF),
}


@pytest.fixture(scope="module")
def check_library():
    path = os.path.join(os.path.dirname(binding.LIB_PATH), "libgdn_check.so")
    assert os.path.exists(path), f"{path} is missing: run the build"
    attn._use(ctypes.CDLL(path))
    yield
    attn._use(binding.lib)


@pytest.mark.parametrize("case", list(CASES))
def test_parity_under_lds_checks(check_library, case):
    CASES[case]()


@pytest.mark.parametrize("window", [0, 16, 300])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1, 129, 0, 190], [500, 33, 1217], [2048 + 65], [1, 2, 3, 31] * 40, [1133] * 8])
def test_waves_without_queries_compute_nothing(check_library, lens, d, window):
    """The last tile of a prompt may have waves whose queries all lie behind its end: nothing is loaded for
    them, and they form no scores of what the LDS held before (a condition of the debug library's kernels)."""
    bounds = [0] + list(ta.np.cumsum(lens))
    host, dv = ta.prefill_case(bounds[-1], 4, 2, d, BF, 51)
    o = ta.gdn.gdn_attn_prefill(*dv, cu_seqlens=torch.tensor(bounds).cuda(), window=window)
    ta.check_prefill(o, host, bounds, window, None, BF, d)
