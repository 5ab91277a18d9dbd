"""What the compiler gave the prompt kernels of libgdn.so, as their code objects say it:
scratch in the tile loop of a kernel that serves costs every call."""
import os
import re
import shutil
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
READELF = shutil.which("llvm-readelf") or "/opt/rocm/llvm/bin/llvm-readelf"
OBJCOPY = shutil.which("llvm-objcopy") or "/opt/rocm/llvm/bin/llvm-objcopy"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def scratch(path, tmp_path):
    """Bytes of scratch to a lane of every kernel of a library built here, by its mangled name."""
    fat = tmp_path / "fat"
    subprocess.run([OBJCOPY, f"--dump-section=.hip_fatbin={fat}", path, os.devnull], check=True)
    blob, found, at = fat.read_bytes(), {}, 0
    while (at := blob.find(MAGIC, at)) >= 0:
        n, = struct.unpack_from("<Q", blob, at + len(MAGIC))
        entry = at + len(MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<3Q", blob, entry)
            target = blob[entry + 24:entry + 24 + length]
            entry += 24 + length
            if b"gfx950" in target and size:
                one = tmp_path / "one"
                one.write_bytes(blob[at + offset:at + offset + size])
                notes = subprocess.run([READELF, "--notes", one], check=True, capture_output=True, text=True).stdout
                for name, bytes_ in re.findall(r"\.name:\s+(_Z\S+)\n\s+\.private_segment_fixed_size:\s+(\d+)", notes):
                    found[name] = int(bytes_)
        at += len(MAGIC)
    return found


@pytest.mark.skipif(not os.path.exists(READELF) or not os.path.exists(OBJCOPY), reason="needs llvm-readelf and llvm-objcopy")
def test_prompt_kernels_that_serve_hold_no_scratch_for_statistics(tmp_path):
    """All without scratch but that of heads of 64 with three workgroups to a CU, which has 3 words outside its loop."""
    found = scratch(os.path.join(ROOT, "gated_delta_rule_gdn_amd", "libgdn.so"), tmp_path)
    plain = {}
    for name, bytes_ in found.items():
        m = re.search(r"prefill_(bf16|f32)_kernelI((?:L[ib]\d+E)+)E", name)
        if m:       # (head size, split, window and, in fp32, head size, waves); then whether it leaves statistics
            args = [int(x) for x in re.findall(r"L[ib](\d+)E", m[2])]
            own = 3 if m[1] == "bf16" else 2
            if args[own:] != [1]:
                plain[(m[1], *args[:own])] = bytes_
    assert len(plain) == 12, plain
    for kernel, bytes_ in plain.items():
        assert bytes_ <= (12 if kernel == ("bf16", 64, 1, 0) else 0), (kernel, bytes_)
