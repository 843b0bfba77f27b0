"""Which kernel a product of 8-bit operands runs with, the assembly of its loads into
LDS, its registers (no GPU)."""
import os
import re
import subprocess

import pytest

from combine_ep_prepare_amd import _build
from test_experts_asm import LOAD, _kernels
from test_experts_asm_m0 import check as check_m0
from test_experts_asm_waits import STATES, early
from test_experts_choice import FEW, PROGRAM, T64, T128, T128_ONCE, T256, T256_ONCE
from test_kernel_asm import _device_asm, _instructions

SOURCES = ("ep_scaled.hip", "ep_layer.hip", "ep_norm.hip", "ep_swiglu.hip")


@pytest.fixture(scope="module")
def kernel(tmp_path_factory):
    work = tmp_path_factory.mktemp("choice")
    source, program = work / "choice.hip", work / "choice"
    source.write_text(PROGRAM.replace("epmi::kernel_of((epmi::Product)n(1), d, n(7), 256)",
                                      "epmi::scaled_kernel_of(d, n(7), 256)"))
    subprocess.run([_build.hipcc(), "-std=c++17", f"--offload-arch={_build.ARCH}", "-I",
                    os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, "-o", str(program),
                    str(source)], check=True, capture_output=True)

    def choose(T, K, E, H, N, cap=None):
        args = [str(v) for v in (0, T, K, E, T * K if cap is None else cap, H, N, 0)]
        return int(subprocess.run([str(program), *args], check=True, capture_output=True).stdout)
    return choose


RING64, RING128, RING64x128 = range(6, 9)


def test_rules_at_their_borders(kernel):
    def rows(r, H=2048, N=1536, E=128):
        return kernel(r * E // 8, 8, E, H, N)
    assert [rows(r) for r in (0, 1, 6, 7, 40, 41, 104, 105, 192, 193)] == \
        [FEW, FEW, FEW, RING64x128, RING64x128, T128_ONCE, T128_ONCE, T256_ONCE, T256_ONCE, T256]
    assert [rows(r, 7168, 4096, 64) for r in (6, 40, 41, 193)] == \
        [FEW, RING64x128, T256_ONCE, T256]
    # eight experts of 4096 x 4096: two tiles of 64 a CU, one of 128, one of 256 for two
    assert [rows(r, 4096, 4096, 8) for r in (7, 56, 57, 117, 118, 128, 129)] == \
        [RING64, RING64, RING128, RING128, T128, T128, T256_ONCE]
    # one expert
    assert [kernel(r, 1, 1, 4096, 4096) for r in (32, 33, 240, 241, 512)] == \
        [FEW, T64, T64, RING64, RING64]
    # a share of the experts: the capacity tells
    assert kernel(64, 8, 32, 7168, 4096, cap=80) == FEW
    assert kernel(32768, 8, 32, 7168, 4096, cap=41000) == T256


def test_loads_into_lds(tmp_path):
    text = "\n".join(_device_asm(os.path.join(_build.CSRC, "ep_scaled.hip"), str(tmp_path)))
    kernels = _kernels(text, "scaled_product_kernel") + _kernels(text, "scaled_ring_kernel")
    assert len(kernels) == 16
    for name, body in kernels:
        check_m0(name, body)
        ins = list(_instructions(body.splitlines()))
        loads = [i for i, s in enumerate(ins) if LOAD.match(s)]
        assert loads
        for i in loads:
            assert ins[i - 2].startswith("s_add_u32 m0, ") and ins[i - 1] == f"s_nop {STATES - 2}"
        ends = [i for i, s in enumerate(ins) if s == "s_endpgm"]
        for i in ends:
            before = [j for j in loads if j < i]
            assert not before or any(re.match(r"^s_waitcnt .*vmcnt\(0\)", x)
                                     for x in ins[before[-1]:i]), name


@pytest.mark.parametrize("source", SOURCES)
def test_scalar_registers_and_scratch(tmp_path, source):
    lines = _device_asm(os.path.join(_build.CSRC, source), str(tmp_path))
    assert early(_instructions(lines)) == []
    text = "\n".join(lines)
    kernels = re.findall(r"^\s*\.amdhsa_kernel (\S+)\n.*?\.amdhsa_private_segment_fixed_size (\d+)",
                         text, flags=re.M | re.S)
    assert kernels
    for name, scratch in kernels:
        # the large tile keeps a few values in scratch between its tiles
        large = "scaled_product_kernelILi0ELi256" in name or "scaled_product_kernelILi1ELi256" in name
        assert int(scratch) <= (20 if large else 0), f"{name}: {scratch} bytes of scratch a lane"
    # and none of them inside the steps, where a wait for it would be one for every load
    for name, body in _kernels(text, "scaled_product_kernel"):
        assert "v_mfma" in body
        for block in re.split(r"^\.LBB\S+:.*$", body, flags=re.M):
            if block.count("v_mfma") >= 4:
                assert "scratch_" not in block, name
