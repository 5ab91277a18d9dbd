"""The entry points of include/gdn_hybrid.h without a GPU: what the header declares
is exported, bad arguments are rejected before any launch, the binding refuses what
it cannot marshal, and the validation is clean under the sanitizers."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_gdn_amd", "csrc")
HIP_INCLUDE = "/opt/rocm/include"

gdn = pytest.importorskip("gated_delta_rule_gdn_amd")

NAMES = ["gdn_add_norm", "gdn_add_norm_backward", "gdn_add_norm_backward_workspace_size", "gdn_attn_backward",
         "gdn_attn_backward_workspace_size", "gdn_attn_prefill_save", "gdn_hybrid_abi_version",
         "gdn_qk_norm_rope_backward", "gdn_qk_norm_rope_backward_workspace_size"]
BF, F32 = gdn.GDN_BF16, gdn.GDN_F32
BIG = 1 << 35


def test_header_and_exports():
    text = open(os.path.join(ROOT, "include", "gdn_hybrid.h")).read()
    assert sorted(set(re.findall(r"^\S.*?\b(gdn_[a-z_]+)\s*\(", text, flags=re.M))) == NAMES
    for lib in ("libgdn.so", "libgdn_check.so"):
        path = os.path.join(os.path.dirname(gdn.gdn.LIB_PATH), lib)
        out = subprocess.run(["nm", "-D", "--defined-only", path], capture_output=True, text=True, check=True).stdout
        assert set(NAMES) <= set(re.findall(r"\sT\s(gdn_\w+)$", out, flags=re.M))
    assert gdn.hybrid_abi_version() == 1


def _addr(i, off=0):
    return ctypes.c_void_p(0x7f0000000000 + i * (1 << 38) + off)


class Call:
    """One entry point: descriptor class, defaults, pointer names in order (`ws`: the workspace, its bytes behind it)."""

    def __init__(self, fn, cls, desc, ptrs, optional=()):
        self.fn, self.cls, self.desc, self.ptrs, self.optional = fn, cls, desc, ptrs, optional

    def __call__(self, ptrs=None, bytes_=BIG, **kw):
        p = {n: _addr(i) for i, n in enumerate(self.ptrs)}
        p.update(ptrs or {})
        args = []
        for n in self.ptrs:
            args.append(p[n])
            if n == "ws":
                args.append(bytes_)
        return self.fn(ctypes.byref(self.cls(**{**self.desc, **kw})), *args, None)

    def none(self):
        return {n: None for n in self.ptrs}


L = gdn.lib
CALLS = {
    "save": Call(L.gdn_attn_prefill_save, gdn.GdnAttnPrefillDesc,
                 dict(N=3, total_T=9, ld_q=512, ld_k=256, ld_v=256, window=0, H_q=4, H_k=2, d=128, io_dtype=BF, scale=0.1),
                 ["cu", "q", "k", "v", "o", "stats"], ["cu"]),
    "backward": Call(L.gdn_attn_backward, gdn.GdnAttnBwdDesc,
                     dict(N=3, total_T=9, ld_q=512, ld_k=256, ld_v=256, ld_dq=512, ld_dk=256, ld_dv=256, window=0, H_q=4,
                          H_k=2, d=128, io_dtype=BF, grad_dtype=BF, scale=0.1),
                     ["cu", "q", "k", "v", "o", "d_o", "stats", "ws", "dq", "dk", "dv"], ["cu"]),
    "rope": Call(L.gdn_qk_norm_rope_backward, gdn.GdnQkBwdDesc,
                 dict(rows=10, ld_q=512, ld_k=256, ld_dq=512, ld_dk=256, H_q=4, H_k=2, d=128, rope_dim=64, rope_mode=0,
                      io_dtype=BF, grad_dtype=BF, rope_scale=1.0, eps=1e-6),
                 ["dq", "dk", "q_raw", "k_raw", "q_weight", "k_weight", "positions", "inv_freq", "ws", "dq_raw", "dk_raw",
                  "dq_weight", "dk_weight"], ["dq_weight", "dk_weight"]),
    "norm": Call(L.gdn_add_norm, gdn.GdnAddNormDesc,
                 dict(rows=10, ld_x=256, C=256, io_dtype=BF, res_dtype=F32, group=-1, eps=1e-6),
                 ["x", "res", "weight", "res_out", "y", "y_scale"], ["res", "weight", "res_out"]),
    "norm_bwd": Call(L.gdn_add_norm_backward, gdn.GdnAddNormBwdDesc,
                     dict(rows=10, ld_dx=256, C=256, io_dtype=BF, res_dtype=F32, eps=1e-6),
                     ["dy", "r", "weight", "d_res_out", "ws", "dx", "d_res", "d_weight"],
                     ["weight", "d_res_out", "dx", "d_res", "d_weight"]),
}
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("call,field,value,expected", [
    ("save", "N", -1, 1), ("save", "H_q", 3, 1), ("save", "d", 32, 2), ("save", "scale", 0.0, 1), ("save", "ld_v", 128, 1),
    ("save", "total_T", 2 ** 32, 2), ("save", "window", -1, 1), ("save", "io_dtype", 2, 1),
    ("backward", "N", -1, 1), ("backward", "total_T", -1, 1), ("backward", "window", -1, 1), ("backward", "H_q", 3, 1),
    ("backward", "H_k", 0, 1), ("backward", "d", 256, 2), ("backward", "scale", NAN, 1), ("backward", "scale", 1e-30, 2),
    ("backward", "scale", 1e30, 2), ("backward", "ld_q", 256, 1), ("backward", "ld_dq", 504, 1), ("backward", "ld_dk", 260, 1),
    ("backward", "ld_dv", 2 ** 31, 1), ("backward", "grad_dtype", 2, 1), ("backward", "io_dtype", F32, 2),
    ("backward", "io_dtype", -1, 1), ("backward", "total_T", 2 ** 32, 2), ("backward", "N", 2 ** 33, 2),
    ("rope", "rows", -1, 1), ("rope", "H_q", -1, 1), ("rope", "d", 96, 2), ("rope", "rope_dim", 8, 1),
    ("rope", "rope_dim", 0, 1), ("rope", "rope_mode", 3, 1), ("rope", "rope_scale", INF, 1), ("rope", "eps", -1.0, 1),
    ("rope", "ld_dq", 256, 1), ("rope", "ld_dk", 252, 1), ("rope", "ld_q", 500, 1), ("rope", "io_dtype", F32, 2),
    ("rope", "grad_dtype", 7, 1), ("rope", "rows", 2 ** 40, 2),
    ("norm", "rows", -1, 1), ("norm", "C", 0, 1), ("norm", "C", 260, 1), ("norm", "ld_x", 248, 1), ("norm", "ld_x", 260, 1),
    ("norm", "eps", NAN, 1), ("norm", "group", -2, 1), ("norm", "group", 16, 2), ("norm", "group", 0, 1),
    ("norm", "io_dtype", 4, 1), ("norm", "res_dtype", -1, 1), ("norm", "rows", 2 ** 40, 2),
    ("norm_bwd", "rows", -1, 1), ("norm_bwd", "C", 12, 1), ("norm_bwd", "ld_dx", 128, 1), ("norm_bwd", "eps", -0.5, 1),
    ("norm_bwd", "res_dtype", 3, 1), ("norm_bwd", "rows", 2 ** 40, 2)])
def test_rejects_bad_descriptor(call, field, value, expected):
    kw = {"ptrs": {"y_scale": None}} if call == "norm" else {}
    assert CALLS[call](**{field: value}, **kw) == expected


def test_rejects_types_and_widths_that_are_not_built():
    norm = CALLS["norm"]
    assert norm(C=16392, ld_x=16392, ptrs={"y_scale": None}) == gdn.GDN_ERR_UNSUPPORTED
    assert norm(io_dtype=F32, res_dtype=BF, ptrs={"y_scale": None}) == gdn.GDN_ERR_UNSUPPORTED
    assert norm(group=64, C=96, ld_x=96) == gdn.GDN_ERR_INVALID_ARG
    assert norm(group=64, ptrs={"y_scale": None}) == gdn.GDN_ERR_INVALID_ARG
    assert norm() == gdn.GDN_ERR_INVALID_ARG                         # a scale without a group
    assert CALLS["norm_bwd"](io_dtype=F32, res_dtype=BF) == gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,name", [(c, n) for c, x in CALLS.items() for n in x.ptrs])
def test_rejects_null_and_misaligned_pointers(call, name):
    c = CALLS[call]
    kw = dict(group=32) if call == "norm" else {}
    if name not in c.optional:
        assert c(ptrs={name: None}, **kw) == gdn.GDN_ERR_INVALID_ARG
    assert c(ptrs={name: _addr(c.ptrs.index(name), 2)}, **kw) == gdn.GDN_ERR_INVALID_ARG


@pytest.mark.parametrize("call,out,other", [
    ("save", "o", "q"), ("save", "stats", "v"), ("save", "stats", "o"), ("save", "o", "cu"),
    ("backward", "dq", "q"), ("backward", "dk", "o"), ("backward", "dv", "d_o"), ("backward", "dq", "dk"),
    ("backward", "dk", "dv"), ("backward", "dq", "ws"), ("backward", "ws", "stats"), ("backward", "dv", "cu"),
    ("rope", "dq_raw", "q_raw"), ("rope", "dk_raw", "dq_raw"), ("rope", "dq_raw", "dk"), ("rope", "dk_raw", "dq"),
    ("rope", "dq_weight", "q_weight"), ("rope", "dq_weight", "dk_weight"), ("rope", "ws", "dk_weight"),
    ("rope", "ws", "dq"), ("rope", "dq_raw", "positions"), ("rope", "dk_raw", "inv_freq"),
    ("norm", "res_out", "x"), ("norm", "y", "res"), ("norm", "y", "x"), ("norm", "y", "res_out"), ("norm", "y_scale", "x"),
    ("norm", "y_scale", "y"), ("norm", "y", "weight"),
    ("norm_bwd", "dx", "r"), ("norm_bwd", "d_res", "r"), ("norm_bwd", "dx", "d_res"), ("norm_bwd", "dx", "d_res_out"),
    ("norm_bwd", "d_res", "dy"), ("norm_bwd", "d_weight", "weight"), ("norm_bwd", "d_weight", "dy"),
    ("norm_bwd", "ws", "dx"), ("norm_bwd", "ws", "d_weight")])
def test_rejects_overlaps(call, out, other):
    c = CALLS[call]
    kw = dict(group=32) if call == "norm" else {}
    assert c(ptrs={out: _addr(c.ptrs.index(other))}, **kw) == gdn.GDN_ERR_INVALID_ARG


def test_statistics_end_behind_their_bytes():
    """9 tokens, 4 heads of 128: 288 bytes, and in bf16 4608 behind them."""
    save, back = CALLS["save"], CALLS["backward"]
    for io, size in ((BF, 4896), (F32, 288)):
        assert save(ptrs={"o": _addr(5, size - 16)}, io_dtype=io) == gdn.GDN_ERR_INVALID_ARG
        assert back(ptrs={"dq": _addr(6, size - 16)}, io_dtype=io, grad_dtype=io) == gdn.GDN_ERR_INVALID_ARG
        assert back(ptrs={"ws": _addr(6, size - 16)}, io_dtype=io, grad_dtype=io) == gdn.GDN_ERR_INVALID_ARG


def test_in_place_only_where_rows_are_the_same():
    c = CALLS["rope"]
    at = {"dq_raw": _addr(0)}
    assert c(ptrs=at, ld_dq=640) == gdn.GDN_ERR_INVALID_ARG
    assert c(ptrs={"dq_raw": _addr(0, 512)}) == gdn.GDN_ERR_INVALID_ARG
    n = CALLS["norm"]
    assert n(ptrs={"y": _addr(0), "y_scale": None}, ld_x=264) == gdn.GDN_ERR_INVALID_ARG
    assert n(ptrs={"res_out": _addr(1, 64), "y_scale": None}) == gdn.GDN_ERR_INVALID_ARG
    b = CALLS["norm_bwd"]
    assert b(ptrs={"dx": _addr(0)}, ld_dx=264) == gdn.GDN_ERR_INVALID_ARG
    assert b(ptrs={"d_res": _addr(3, 32)}) == gdn.GDN_ERR_INVALID_ARG


def test_column_blocks_must_not_meet():
    """dq, dk, dv in one buffer of 1024 columns of 2 bytes: blocks of 512, 256 and 256 columns."""
    c = CALLS["backward"]
    wide = dict(ld_dq=1024, ld_dk=1024, ld_dv=1024)
    at = lambda a, b: {"dk": _addr(8, a), "dv": _addr(8, b)}  # noqa: E731
    for a, b in ((1008, 1536), (1024, 1520), (1024, 1552), (1536, 1536)):
        assert c(ptrs=at(a, b), **wide) == gdn.GDN_ERR_INVALID_ARG, (a, b)
    assert c(ptrs=at(1024, 1536), **{**wide, "ld_dv": 1032}) == gdn.GDN_ERR_INVALID_ARG


def test_absent_operands_take_no_pointers():
    c = CALLS["rope"]
    assert c(H_k=0) == gdn.GDN_ERR_INVALID_ARG
    assert c(H_q=0, H_k=0) == gdn.GDN_ERR_INVALID_ARG
    assert c(ptrs={"q_weight": None}) == gdn.GDN_ERR_INVALID_ARG       # a weight's gradient without the weight


def test_nothing_to_do_returns_ok_without_a_launch():
    for name in ("save", "backward"):
        c = CALLS[name]
        assert c(N=0, ptrs=c.none(), bytes_=0) == gdn.GDN_OK
        assert c(total_T=0, ptrs=c.none(), bytes_=0) == gdn.GDN_OK
        assert c(total_T=10, ptrs={"cu": None}) == gdn.GDN_ERR_INVALID_ARG      # 10 % 3
    for name in ("rope", "norm", "norm_bwd"):
        assert CALLS[name](rows=0, ptrs=CALLS[name].none(), bytes_=0) == gdn.GDN_OK
    b = CALLS["norm_bwd"]
    assert b(ptrs={"dx": None, "d_res": None, "d_weight": None}) == gdn.GDN_OK


def test_workspaces_are_needed_in_full():
    for name, size in (("backward", L.gdn_attn_backward_workspace_size),
                       ("rope", L.gdn_qk_norm_rope_backward_workspace_size),
                       ("norm_bwd", L.gdn_add_norm_backward_workspace_size)):
        c = CALLS[name]
        need = size(ctypes.byref(c.cls(**c.desc)))
        assert need > 0 and need % 4 == 0
        assert c(bytes_=need - 1) == gdn.GDN_ERR_INVALID_ARG
        field = "C" if name == "norm_bwd" else "d"
        assert size(ctypes.byref(c.cls(**{**c.desc, field: 3}))) == 0


@pytest.mark.parametrize("heads", [(1, 1), (0, 1), (4, 2), (8190, 2), (8192, 1), (1, 16384), (65536, 65536)])
def test_no_row_needs_no_workspace(heads):
    """And so no workgroup of the gradient's kernel, which would read frequencies that a call without rows need not
    give: also where there are more heads than it has workgroups."""
    size = L.gdn_qk_norm_rope_backward_workspace_size
    desc = dict(rows=0, ld_q=2 ** 22, ld_k=2 ** 22, ld_dq=2 ** 22, ld_dk=2 ** 22, H_q=heads[0], H_k=heads[1], d=64, rope_dim=64,
                rope_mode=0, io_dtype=BF, grad_dtype=BF, rope_scale=1.0, eps=1e-6)
    assert size(ctypes.byref(gdn.GdnQkBwdDesc(**desc))) == 0
    assert size(ctypes.byref(gdn.GdnQkBwdDesc(**{**desc, "rows": 1}))) >= 256 * (sum(heads) // 2)


@pytest.mark.parametrize("window", [1, 2 ** 40, 2 ** 63 - 1])
def test_windows_of_any_size_have_a_plan(window):
    size = L.gdn_attn_backward_workspace_size
    desc = {**CALLS["backward"].desc, "total_T": 5000}
    a = size(ctypes.byref(gdn.GdnAttnBwdDesc(**{**desc, "window": window})))
    assert a >= 16 * 5000 * 4 and (window < 5000 or a == size(ctypes.byref(gdn.GdnAttnBwdDesc(**desc))))


def test_binding_rejects_host_tensors_and_what_does_not_fit():
    x = torch.zeros(4, 2, 64)
    r = torch.zeros(4, 64)
    for call in (lambda: gdn.gdn_attn_prefill_save(x, x, x), lambda: gdn.gdn_attn_backward(x, x, x, x, x, x),
                 lambda: gdn.gdn_qk_norm_rope_backward(x, None), lambda: gdn.gdn_add_norm(r),
                 lambda: gdn.gdn_add_norm_backward(r, r)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="must be given"):
        gdn.gdn_qk_norm_rope_backward(None, None)


@pytest.mark.parametrize("source", ["norm_ops.hip", "join_parts.hpp", "attn_rope_backward.hip", "attn_backward.hip"])
def test_debug_kernels_begin_with_nan_in_all_their_lds(source):
    """Every shared array is filled in the debug library, where reads of what was not written show as NaN."""
    text = open(os.path.join(CSRC, source)).read()
    arrays = [n for d in re.findall(r"__shared__\s+([^;]+);", text) for n in re.findall(r"(\w+)\[", d.split("=")[0])]
    arrays = [n for n in arrays if n.startswith("s")]
    filled = re.findall(r"lds_nan_fill\((\w+), sizeof \1\);", text)
    assert arrays and sorted(arrays) == sorted(filled)
    assert len(re.findall(r"\blds_check\(", text)) >= len(set(arrays))


def _run(tmp_path, name, sources):
    exe = str(tmp_path / name)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE]
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
    _run(tmp_path, "hybrid_check", [os.path.join(CSRC, "hybrid_api.cpp"), os.path.join(here, "hybrid_check.cpp")])


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_shares_of_the_backward_walks_are_equal_and_complete(tmp_path):
    _run(tmp_path, "attn_walk_check", [os.path.join(ROOT, "tests", "abi_check", "attn_walk_check.cpp")])
