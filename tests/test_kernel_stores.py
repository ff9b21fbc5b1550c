"""What the compiler makes of stores past the caches: large 16-bit outputs of dequant_mx4 go past them,
32-bit ones, whose lanes store two pieces 32 bytes apart, do not."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from w8a8_int8_quantized_qk_amd import build


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    try:
        cc = build.hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("listing") / "mx4_quant.s"
    subprocess.run([cc, *build.FLAGS, "-S", "--cuda-device-only", os.path.join(build.CSRC, "mx4_quant.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    kernels, name = {}, None
    for line in out.read_text().splitlines():
        if m := re.match(r"(_Z\w*mx4_dequant_kernel\w*):", line):
            name = m.group(1)
            kernels[name] = []
        elif "s_endpgm" in line:
            name = None
        elif name and re.search(r"\b(global|flat|buffer)_store", line):
            kernels[name].append(line.split())
    return kernels


def test_the_way_back_stores_as_it_says(listing):
    # <type, past the caches>: 0 binary32, 1 bf16, 2 binary16
    found = {re.search(r"ILi(\d)ELb(\d)E", k).groups(): v for k, v in listing.items()}
    assert set(found) == {("0", "0"), ("1", "0"), ("1", "1"), ("2", "0"), ("2", "1")}
    for (dtype, past), stores in found.items():
        assert stores and all(("nt" in s) == (past == "1") for s in stores), (dtype, past, stores)
