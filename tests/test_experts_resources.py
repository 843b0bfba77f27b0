"""The registers of the experts' kernels, from their gfx950 assembly (no GPU):
none keeps registers in scratch but the instance whose comment says so."""
import os
import re

import pytest

from combine_ep_prepare_amd import _build
from test_kernel_asm import _device_asm

# few_rows_kernel<bf16, 4-bit, groups of 32, zero points>: three blocks a CU and
# 6 registers in scratch against two blocks and none, 45.6 against 49.1 us.
SCRATCH = {"few_rows_kernelILi0ELb1ELi32ELb1E": 28}


@pytest.mark.parametrize("source", ["ep_linear.hip", "ep_decode.hip", "ep_swiglu.hip"])
def test_no_kernel_spills(tmp_path, source):
    text = "\n".join(_device_asm(os.path.join(_build.CSRC, source), str(tmp_path)))
    kernels = re.findall(r"^\s*\.amdhsa_kernel (\S+)\n.*?\.amdhsa_private_segment_fixed_size (\d+)",
                         text, flags=re.M | re.S)
    assert len(kernels) >= 6
    for name, scratch in kernels:
        allowed = max((n for part, n in SCRATCH.items() if part in name), default=0)
        assert int(scratch) <= allowed, f"{name}: {scratch} bytes of scratch a lane"
