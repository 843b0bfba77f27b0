"""Wait states in the gfx950 assembly of the experts' kernels (no GPU).

A vector memory instruction may read a scalar register five wait states after a
vector instruction wrote it (a lane read back, a comparison), no sooner; in
between it sees the old value. The compiler keeps to it for its own instructions
and not for those of an asm statement. Checked here: no memory instruction reads
such a register too early, and each load into LDS, which all stand in asm
statements, has the five wait states right before it, whatever comes ahead: the
write of m0 that gives its place, and four more.
"""
import os
import re

import pytest

from combine_ep_prepare_amd import _build
from test_experts_asm import LOAD
from test_kernel_asm import _device_asm, _instructions

MEMORY = re.compile(r"^(buffer|global|flat|scratch)_")
SCALAR = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(vcc)\b")
STATES = 5


def scalars(text):
    out = set()
    for a, b, one, vcc in SCALAR.findall(text):
        out |= {"vcc"} if vcc else {int(one)} if one else set(range(int(a), int(b) + 1))
    return out


def written(ins):
    """Scalar registers that a vector instruction writes: its first operand, and
    the second where that is a carry or a comparison's."""
    if not ins.startswith("v_"):
        return set()
    operands = ins.split(None, 1)[1].split(",") if " " in ins else []
    out = scalars(operands[0]) if operands else set()
    if re.match(r"v_\w*(_co_|div_scale|mad_[ui]64)", ins) and len(operands) > 1:
        out |= scalars(operands[1])
    return out


def early(ins):
    """(instruction, what wrote its register) of each that reads too early."""
    ins, found = list(ins), []
    for i, s in enumerate(ins):
        if not MEMORY.match(s):
            continue
        need, waited, j = scalars(s), 0, i - 1
        while need and j >= 0 and waited < STATES:
            if written(ins[j]) & need:
                found.append((s, ins[j]))
                break
            nop = re.match(r"^s_nop (\d+)", ins[j])
            waited += int(nop.group(1)) + 1 if nop else 1
            j -= 1
    return found


@pytest.mark.parametrize("source", ["ep_linear.hip", "ep_decode.hip", "ep_swiglu.hip"])
def test_scalar_registers_are_read_in_time(tmp_path, source):
    ins = list(_instructions(_device_asm(os.path.join(_build.CSRC, source), str(tmp_path))))
    assert early(ins) == []
    loads = [i for i, s in enumerate(ins) if LOAD.match(s)]
    assert bool(loads) == (source == "ep_linear.hip")
    for i in loads:
        assert ins[i - 2].startswith("s_add_u32 m0, "), ins[i - 2:i + 1]
        assert ins[i - 1] == f"s_nop {STATES - 2}", ins[i - 2:i + 1]


def test_the_check_sees_what_would_be_wrong():
    load = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds"
    for wrong in (["v_readlane_b32 s6, v134, 7", load],
                  ["v_readfirstlane_b32 s4, v2", "s_mov_b32 m0, s9", "s_nop 2", load],
                  ["v_cmp_lt_u32_e64 s[4:5], v1, v2", "s_nop 3", load],
                  ["v_add_co_u32 v1, s[6:7], v1, v2", "global_load_dword v0, v1, s[6:7]"]):
        assert len(early(wrong)) == 1, wrong
    for right in (["v_readlane_b32 s6, v134, 7", "s_nop 4", load],
                  ["v_readlane_b32 s8, v134, 7", load], ["s_mov_b32 s6, s9", load],
                  ["v_readlane_b32 s6, v134, 7", "s_mov_b32 m0, s9", "s_nop 3", load]):
        assert early(right) == [], right
