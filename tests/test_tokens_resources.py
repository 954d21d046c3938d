"""What the compiler gave the attention kernels, read from the library as it was
built: no registers spilled to memory.

A spilled register is reloaded through the same counter that the copies to
shared memory are waited for by, so that each reload waits for the copies on
their way (a forward kernel with 29 of them took twice its time)."""

import os
import re
import shutil
import struct
import subprocess

import pytest

from memory_bound_cnn_amd import binding

READELF = shutil.which("llvm-readelf") or "/opt/rocm/llvm/bin/llvm-readelf"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(blob):
    """The gfx950 code objects of a library's bundles."""
    at = blob.find(MAGIC)
    while at >= 0:
        p = at + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", blob, at + len(MAGIC))[0]):
            offset, size, length = struct.unpack_from("<QQQ", blob, p)
            if blob[p + 24:p + 24 + length].endswith(b"gfx950"):
                yield blob[at + offset:at + offset + size]
            p += 24 + length
        at = blob.find(MAGIC, at + 1)


def kernels(tmp_path):
    """{kernel: {resource: number}} of the library's attention kernels."""
    found = {}
    for i, code in enumerate(code_objects(open(binding.LIB_PATH, "rb").read())):
        if b"k_attn_" not in code:
            continue
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        notes = subprocess.run([READELF, "--notes", str(path)], capture_output=True, text=True, check=True).stdout
        for entry in re.split(r"\n  - \.", notes):
            name = re.search(r"\.name:\s+(\S*k_attn_\S+)\n", entry)
            if name:
                found[name.group(1)] = {k: int(v) for k, v in re.findall(r"\.?(\w+):\s+(\d+)\n", entry)}
    return found


@pytest.mark.skipif(not os.path.exists(READELF), reason="no llvm-readelf")
def test_attention_kernels_spill_no_registers(tmp_path):
    found = kernels(tmp_path)
    assert len([k for k in found if "k_attn_join" not in k]) == 24    # three kernels, four widths, two types
    bad = {k: v for k, v in found.items() if v["private_segment_fixed_size"] or v["vgpr_spill_count"]}
    assert not bad, bad
