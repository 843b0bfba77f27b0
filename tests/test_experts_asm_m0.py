"""m0 in the gfx950 assembly of the grouped product (no GPU).

Its loads into LDS take their place there from m0, which their asm statements
write. The compiler does not know of these writes. Checked here,
for every kernel built from the file: m0 appears in them and nowhere else, each
load has its own write, and no branch target lies between the two.
"""
import os
import re

from combine_ep_prepare_amd import _build
from test_experts_asm import LOAD, _kernels
from test_kernel_asm import _device_asm

WRITE = re.compile(r"^(s_mov_b32 m0, \S+|s_add_u32 m0, \S+, \S+)$")


def check(name, body):
    pending = None     # the write that the next load will use
    for line in body.splitlines():
        s = line.split(";")[0].strip()
        if s.endswith(":") and pending:
            raise AssertionError(f"{name}: a branch target between {pending!r} and its load")
        if LOAD.match(s):
            assert pending, f"{name}: {s!r} without a write of m0 of its own"
            pending = None
        elif re.search(r"\bm0\b", s):
            assert WRITE.match(s), f"{name}: another use of m0, {s!r}"
            assert pending is None, f"{name}: {s!r} behind {pending!r}, with no load between"
            pending = s
    assert pending is None, f"{name}: {pending!r} without a load"


def test_m0_is_the_loads_alone(tmp_path):
    lines = _device_asm(os.path.join(_build.CSRC, "ep_linear.hip"), str(tmp_path))
    kernels = _kernels("\n".join(lines), "grouped_product_kernel")
    assert kernels
    for name, body in kernels:
        check(name, body)


def test_the_check_sees_what_would_be_wrong():
    load = "buffer_load_dwordx4 v1, s[0:3], 0 offen lds\n"
    write, nop = "s_mov_b32 m0, s7\n", "s_nop 0\n"
    check("right", (write + nop + load) * 2)
    for wrong in (write + nop + load + load, write + "s_mov_b32 m0, s8\n" + nop + load,
                  write + nop + ".LBB0_1:\n" + load, write + nop + load + write,
                  write + nop + "s_movrels_b32 s1, s2\ns_add_u32 s1, m0, s2\n" + load):
        try:
            check("wrong", wrong)
        except AssertionError:
            continue
        raise RuntimeError(f"not seen: {wrong!r}")
