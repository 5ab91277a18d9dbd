"""The attention entry points without a GPU: what include/gdn_attn.h declares is
exported, bad arguments are rejected before any launch, the binding refuses
what it cannot marshal, and the kernels' index arithmetic stays within the
tensors for malformed offsets, lengths and page tables (built for the host
under the sanitizers)."""
import ctypes
import os
import re
import shutil
import subprocess
import sys
import sysconfig

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_gdn_amd", "csrc")
HIP_INCLUDE = "/opt/rocm/include"

gdn = pytest.importorskip("gated_delta_rule_gdn_amd")

NAMES = ["gdn_attn_abi_version", "gdn_attn_decode", "gdn_attn_decode_workspace_size",
         "gdn_attn_prefill", "gdn_kv_append", "gdn_qk_norm_rope"]


def test_header_and_exports():
    text = open(os.path.join(ROOT, "include", "gdn_attn.h")).read()
    assert sorted(set(re.findall(r"^\S.*?\b(gdn_[a-z_]+)\s*\(", text, flags=re.M))) == NAMES
    for lib in ("libgdn.so", "libgdn_check.so"):
        path = os.path.join(os.path.dirname(gdn.gdn.LIB_PATH), lib)
        out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True,
                             check=True).stdout
        assert set(NAMES) <= set(re.findall(r"\sT\s(gdn_\w+)$", out, flags=re.M))
    assert gdn.attn_abi_version() == 1


def _addr(i, off=0):
    return ctypes.c_void_p(0x7f0000000000 + i * (1 << 36) + off)


BF, F32 = gdn.GDN_BF16, gdn.GDN_F32


class Call:
    """One entry point: descriptor class, defaults, pointer names in order."""

    def __init__(self, fn, cls, desc, ptrs, optional=(), tail=()):
        self.fn, self.cls, self.desc, self.ptrs, self.optional, self.tail = fn, cls, desc, ptrs, optional, tail

    def __call__(self, ptrs=None, **kw):
        tail = kw.pop("tail", self.tail)
        p = {n: _addr(i) for i, n in enumerate(self.ptrs)}
        p.update(ptrs or {})
        return self.fn(ctypes.byref(self.cls(**{**self.desc, **kw})), *[p[n] for n in self.ptrs], *tail, None)


CALLS = {
    "norm_rope": Call(gdn.lib.gdn_qk_norm_rope, gdn.GdnQkDesc,
                      dict(rows=10, ld_q=512, ld_k=256, H_q=4, H_k=2, d=128, rope_dim=64, rope_mode=0, io_dtype=BF,
                           rope_scale=1.0, eps=1e-6),
                      ["q_raw", "k_raw", "q_weight", "k_weight", "positions", "inv_freq", "q", "k"],
                      optional=["q_weight", "k_weight"]),
    "append": Call(gdn.lib.gdn_kv_append, gdn.GdnKvAppendDesc,
                   dict(N=3, total_T=9, ld_k=256, ld_v=256, num_pages=20, max_pages=5, H_k=2, d=128, page_size=16,
                        rope_dim=64, rope_mode=1, io_dtype=BF, rope_scale=1.0, eps=1e-6),
                   ["cu_seqlens", "seq_lens", "page_table", "k_raw", "v_raw", "k_weight", "inv_freq", "k_cache",
                    "v_cache", "k_scale", "v_scale"], optional=["k_weight", "cu_seqlens"]),
    "prefill": Call(gdn.lib.gdn_attn_prefill, gdn.GdnAttnPrefillDesc,
                    dict(N=3, total_T=9, ld_q=512, ld_k=256, ld_v=256, window=0, H_q=4, H_k=2, d=128, io_dtype=BF,
                         scale=0.1), ["cu_seqlens", "q", "k", "v", "o"], optional=["cu_seqlens"]),
    "decode": Call(gdn.lib.gdn_attn_decode, gdn.GdnAttnDecodeDesc,
                   dict(N=3, num_pages=20, max_pages=500, window=0, H_q=4, H_k=2, d=128, page_size=16, io_dtype=BF,
                        scale=0.1),
                   ["q", "k_cache", "v_cache", "k_scale", "v_scale", "page_table", "seq_lens", "o", "workspace"],
                   tail=(1 << 35,)),
}


@pytest.mark.parametrize("call,field,value,expected", [
    ("norm_rope", "rows", -1, 1), ("norm_rope", "H_q", -1, 1), ("norm_rope", "d", 0, 1), ("norm_rope", "d", 256, 2),
    ("norm_rope", "rope_dim", 8, 1), ("norm_rope", "rope_dim", 144, 1), ("norm_rope", "rope_dim", -16, 1),
    ("norm_rope", "rope_dim", 0, 1),                       # positions and frequencies without a rotation
    ("norm_rope", "rope_mode", 2, 1), ("norm_rope", "io_dtype", 2, 1), ("norm_rope", "rope_scale", float("inf"), 1),
    ("norm_rope", "eps", -1.0, 1), ("norm_rope", "eps", float("nan"), 1), ("norm_rope", "ld_q", 504, 1),
    ("norm_rope", "ld_q", 516, 1), ("norm_rope", "ld_k", 2 ** 31, 1), ("norm_rope", "rows", 2 ** 40, 2),
    ("norm_rope", "rows", 2 ** 60, 1), ("norm_rope", "H_q", 2 ** 16, 2),
    ("append", "N", -1, 1), ("append", "total_T", -1, 1), ("append", "H_k", 0, 1), ("append", "page_size", 0, 1),
    ("append", "page_size", 48, 2), ("append", "page_size", 256, 2), ("append", "num_pages", 0, 1),
    ("append", "num_pages", 2 ** 31, 1), ("append", "max_pages", 0, 1), ("append", "max_pages", 2 ** 60, 1),
    ("append", "ld_k", 128, 1), ("append", "ld_v", 260, 1), ("append", "total_T", 2 ** 33, 2),
    ("append", "rope_dim", 0, 1), ("append", "d", 96, 2),
    ("prefill", "N", -1, 1), ("prefill", "total_T", -1, 1), ("prefill", "window", -1, 1), ("prefill", "H_q", 3, 1),
    ("prefill", "H_k", 0, 1), ("prefill", "d", 32, 2), ("prefill", "scale", 0.0, 1),
    ("prefill", "scale", float("nan"), 1), ("prefill", "ld_q", 256, 1), ("prefill", "total_T", 2 ** 32, 2),
    ("decode", "N", -1, 1), ("decode", "window", -5, 1), ("decode", "H_q", 5, 1), ("decode", "scale", 0.0, 1),
    ("decode", "page_size", 8, 2), ("decode", "num_pages", 0, 1), ("decode", "io_dtype", 9, 1),
    ("decode", "N", 2 ** 30, 2),
])
def test_rejects_bad_descriptor(call, field, value, expected):
    assert CALLS[call](**{field: value}) == expected


@pytest.mark.parametrize("call,name", [(c, n) for c, x in CALLS.items() for n in x.ptrs])
def test_rejects_null_and_misaligned_pointers(call, name):
    c = CALLS[call]
    if name not in c.optional:
        assert c(ptrs={name: None}) == gdn.GDN_ERR_INVALID_ARG
    i = c.ptrs.index(name)
    assert c(ptrs={name: _addr(i, 2)}) == gdn.GDN_ERR_INVALID_ARG


@pytest.mark.parametrize("call,out,other", [
    ("norm_rope", "q", "k_raw"), ("norm_rope", "k", "q"), ("norm_rope", "q", "q_weight"),
    ("norm_rope", "k", "positions"), ("append", "k_cache", "v_cache"), ("append", "k_scale", "v_scale"),
    ("append", "v_cache", "v_raw"), ("append", "k_scale", "page_table"), ("append", "v_scale", "seq_lens"),
    ("prefill", "o", "q"), ("prefill", "o", "v"), ("prefill", "o", "cu_seqlens"), ("decode", "o", "q"),
    ("decode", "o", "workspace"), ("decode", "workspace", "k_cache"), ("decode", "o", "page_table")])
def test_rejects_overlaps(call, out, other):
    c = CALLS[call]
    assert c(ptrs={out: _addr(c.ptrs.index(other))}) == gdn.GDN_ERR_INVALID_ARG


def test_norm_rope_in_place_only_where_rows_are_dense():
    c = CALLS["norm_rope"]
    assert c(ptrs={"q": _addr(0)}, ld_q=640) == gdn.GDN_ERR_INVALID_ARG
    assert c(ptrs={"q": _addr(0, 256)}) == gdn.GDN_ERR_INVALID_ARG


def test_absent_operands_take_no_pointers():
    c = CALLS["norm_rope"]
    assert c(H_k=0) == gdn.GDN_ERR_INVALID_ARG             # k pointers without key heads
    assert c(H_q=0, H_k=0) == gdn.GDN_ERR_INVALID_ARG


def test_nothing_to_do_returns_ok_without_a_launch():
    none = {n: None for n in CALLS["norm_rope"].ptrs}
    assert CALLS["norm_rope"](rows=0, ptrs=none) == gdn.GDN_OK
    for name in ("append", "prefill"):
        none = {n: None for n in CALLS[name].ptrs}
        assert CALLS[name](N=0, ptrs=none) == gdn.GDN_OK
        assert CALLS[name](total_T=0, ptrs=none) == gdn.GDN_OK
        assert CALLS[name](total_T=10, ptrs={"cu_seqlens": None}) == gdn.GDN_ERR_INVALID_ARG   # 10 % 3
    assert CALLS["decode"](N=0, ptrs={n: None for n in CALLS["decode"].ptrs}) == gdn.GDN_OK


def test_decode_workspace_is_needed_in_full():
    c = CALLS["decode"]
    need = gdn.lib.gdn_attn_decode_workspace_size(ctypes.byref(c.cls(**c.desc)))
    assert need > 0 and need % 4 == 0
    assert c(tail=(need - 1,)) == gdn.GDN_ERR_INVALID_ARG
    one = gdn.GdnAttnDecodeDesc(**{**c.desc, "max_pages": 1})
    assert gdn.lib.gdn_attn_decode_workspace_size(ctypes.byref(one)) == 0
    assert gdn.lib.gdn_attn_decode_workspace_size(ctypes.byref(c.cls(**{**c.desc, "d": 3}))) == 0


def test_binding_rejects_host_tensors():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="device tensor"):
        gdn.gdn_qk_norm_rope(x)
    with pytest.raises(ValueError, match="device tensor"):
        gdn.gdn_attn_prefill(x, x, x)
    with pytest.raises(ValueError, match="must be given"):
        gdn.gdn_qk_norm_rope(None)


def _run(tmp_path, name, sources, include_hip):
    exe = str(tmp_path / name)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    if include_hip:
        cmd += ["-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE]
    subprocess.run(cmd + sources + ["-o", exe], check=True, capture_output=True, text=True, timeout=600)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("ok "), r.stdout


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE),
                    reason="needs g++ and the HIP headers")
def test_validation_clean_under_asan_and_ubsan(tmp_path):
    here = os.path.join(ROOT, "tests", "abi_check")
    _run(tmp_path, "attn_check", [os.path.join(CSRC, "attn_api.cpp"), os.path.join(here, "attn_stubs.cpp"),
                                  os.path.join(here, "attn_check.cpp")], True)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_index_arithmetic_stays_within_the_tensors(tmp_path):
    _run(tmp_path, "attn_index_check", [os.path.join(ROOT, "tests", "abi_check", "attn_index_check.cpp")], False)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_decode_shares_are_equal_and_complete(tmp_path):
    _run(tmp_path, "attn_share_check", [os.path.join(ROOT, "tests", "abi_check", "attn_share_check.cpp")], False)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_decode_plan_holds_for_windows_of_any_size(tmp_path):
    _run(tmp_path, "attn_plan_check", [os.path.join(ROOT, "tests", "abi_check", "attn_plan_check.cpp")], False)


@pytest.mark.parametrize("window", [2 ** 40, 2 ** 63 - 33, 2 ** 63 - 32, 2 ** 63 - 1])
def test_decode_workspace_of_a_window_that_hides_nothing(window):
    """A window beyond the cache is none: the call shares the same work in the same way."""
    size = lambda w: gdn.lib.gdn_attn_decode_workspace_size(ctypes.byref(  # noqa: E731
        gdn.GdnAttnDecodeDesc(1, 4096, 2048, w, 32, 4, 128, 64, BF, 0.1)))
    assert size(window) == size(0) > 0


def _python(code):
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


@pytest.mark.parametrize("how", ["missing", "other torch"])
def test_package_works_without_the_extension_module(how):
    """The delta rule needs libgdn.so alone; the attention calls say what is missing."""
    stand_in = "None" if how == "missing" else "types.SimpleNamespace(torch_version='0.0.1')"
    out = _python(f"""
import sys, types, torch
sys.modules["gated_delta_rule_gdn_amd._attn_native"] = {stand_in}
if {how == "other torch"}:
    import importlib.machinery
    sys.modules["gated_delta_rule_gdn_amd._attn_native"].__spec__ = importlib.machinery.ModuleSpec("x", None)
import gated_delta_rule_gdn_amd as gdn
assert gdn.abi_version() > 0 and gdn.attn_abi_version() == 1
x = torch.zeros(4, 2, 64)
try:
    gdn.gdn_kv_append(x, x, x, x, x, x, x, x)
except ImportError as e:
    print("refused:", e)
""")
    assert "refused:" in out and "build.py" in out


def test_extension_module_names_the_python_and_torch_it_is_for():
    from gated_delta_rule_gdn_amd import attn
    assert attn._native.__file__.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert attn._native.torch_version == torch.__version__.split("+")[0]
