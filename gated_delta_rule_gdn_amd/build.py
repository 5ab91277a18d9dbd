"""Build libgdn.so (and its debug twin libgdn_check.so) in-tree with hipcc for gfx950,
and the Python extension module that marshals the attention calls.

    python gated_delta_rule_gdn_amd/build.py [-v]

(Run as a script: importing the package first would load the library.)

Every HIP source is compiled with packed-fp32 instructions disabled
(``-Xclang -target-feature -Xclang -packed-fp32-ops``); hipcc's host pass warns
that it does not know that feature, which is harmless.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgdn.so")
LIB_CHECK = os.path.join(PKG, "libgdn_check.so")
MODULE = os.path.join(PKG, "_attn_native" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["gdn_api.cpp", "decode.hip", "chunk_fwd.hip", "chunk_fwd_sb.hip", "layer_ops.hip",
           "backward.hip", "noalloc.hip", "attn_api.cpp", "attn_rope.hip", "attn_prefill.hip",
           "attn_decode.hip", "hybrid_api.cpp", "attn_backward.hip", "attn_rope_backward.hip",
           "norm_ops.hip"]
ARCH = os.environ.get("GDN_OFFLOAD_ARCH", "gfx950")

COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", INCLUDE, "-I", CSRC, "-Wall", "-Wno-unused-function"]


# Flags of single sources.  attn_prefill.hip, attn_backward.hip: products take and
# leave their sums in vector registers; otherwise kernels that fill a CU's LDS with
# one workgroup keep them in accumulation registers and move them there and back in
# every tile.
SOURCE_FLAGS = {"attn_prefill.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
                "attn_backward.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}

# The product library and its debug twin (-DGDN_CHECK: LDS filled with NaN
# at kernel start, LDS accesses and block indices checked, every call waits
# for its kernels and reports GDN_ERR_CHECK on a violation).
VARIANTS = [(LIB, BUILD_DIR, []),
            (LIB_CHECK, os.path.join(BUILD_DIR, "check"), ["-DGDN_CHECK"])]
MAX_JOBS = 8


def module_command() -> list:
    """g++ on csrc/attn_bind.cpp against this interpreter's and torch's headers."""
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-attributes",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", inc,
            "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I", os.path.join(rocm, "include"), os.path.join(CSRC, "attn_bind.cpp"),
            "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
            "-L", os.path.join(rocm, "lib"), "-lamdhip64"]


def build(verbose: bool = False) -> str:
    jobs = [(MODULE, "attn_bind.cpp", None, [*module_command(), "-o", MODULE + ".tmp"])]
    for lib, bdir, flags in VARIANTS:
        os.makedirs(bdir, exist_ok=True)
        for src in SOURCES:
            obj = os.path.join(bdir, os.path.splitext(src)[0] + ".o")
            lang = ["-x", "hip"] if src.endswith(".hip") else []
            cmd = ["hipcc", *COMMON, *flags, *SOURCE_FLAGS.get(src, []), *lang, "-c", os.path.join(CSRC, src), "-o", obj]
            jobs.append((lib, src, obj, cmd))
    failed = []
    running = []

    def reap(entry):
        lib, src, obj, p = entry
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        noise = "is not a recognized feature for this target"
        lines = [ln for ln in text.splitlines() if noise not in ln]
        if lines and (verbose or p.returncode):
            print("\n".join(lines), file=sys.stderr)
        if p.returncode:
            failed.append((os.path.basename(lib), src))

    for lib, src, obj, cmd in jobs:
        if len(running) >= MAX_JOBS:
            reap(running.pop(0))
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append((lib, src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                        stderr=subprocess.STDOUT)))
    for entry in running:
        reap(entry)
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    for lib, bdir, _ in VARIANTS:
        objs = [os.path.join(bdir, os.path.splitext(src)[0] + ".o") for src in SOURCES]
        tmp = lib + ".tmp"
        cmd = ["hipcc", f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, lib)
    os.replace(MODULE + ".tmp", MODULE)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
