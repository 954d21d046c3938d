"""What the compiler gave the kernels of the experts' products and of the gated
scan, read from the library as it was built: no registers spilled to memory.

In the products a spilled register is reloaded through the counter that the
copies to shared memory are waited for by; in the scan, whose time is its
traffic, spills are more of it (a backward pass with them moved half as much again)."""

import os
import re
import subprocess

import pytest

from memory_bound_cnn_amd import binding
from tests.test_tokens_resources import READELF, code_objects


@pytest.mark.skipif(not os.path.exists(READELF), reason="no llvm-readelf")
def test_kernels_spill_no_registers(tmp_path):
    found = {}
    for i, code in enumerate(code_objects(open(binding.LIB_PATH, "rb").read())):
        if b"k_product_" not in code and b"k_scan_" not in code:
            continue
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        notes = subprocess.run([READELF, "--notes", str(path)], capture_output=True, text=True, check=True).stdout
        for entry in re.split(r"\n  - \.", notes):
            name = re.search(r"\.name:\s+(\S*k_(?:product|scan)_\S+)\n", entry)
            if name:
                found[name.group(1)] = {k: int(v) for k, v in re.findall(r"\.?(\w+):\s+(\d+)\n", entry)}
    assert sum("k_product_rows" in k for k in found) >= 6 and sum("k_scan_backward" in k for k in found) == 4
    bad = {k: v for k, v in found.items() if v["private_segment_fixed_size"] or v["vgpr_spill_count"]}
    assert not bad, bad
