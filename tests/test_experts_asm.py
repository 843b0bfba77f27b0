"""The gfx950 assembly of the grouped product, checked on the host (no GPU).

Its loads into LDS are written out in asm statements, so the compiler neither
counts them nor knows that they read m0. Checked here, for every kernel built
from the file: an instruction stands between each write of m0 and the load that
uses it, and no such load is left in flight where a wavefront ends (a late one
would write into the LDS of the block that follows): after the last load on the
straight line to an end of the program comes a wait for all of them.
"""
import os
import re

from combine_ep_prepare_amd import _build
from test_kernel_asm import _device_asm, _instructions

LOAD = re.compile(r"^buffer_load_dwordx4 .*\blds$")


def _kernels(text, name):
    return re.findall(r"^(_Z\S*" + name + r"\S*):[^\n]*\n(.*?)^\.Lfunc_end", text,
                      flags=re.M | re.S)


def test_loads_into_lds(tmp_path):
    lines = _device_asm(os.path.join(_build.CSRC, "ep_linear.hip"), str(tmp_path))
    kernels = _kernels("\n".join(lines), "grouped_product_kernel")
    assert kernels
    for name, body in kernels:
        ins = list(_instructions(body.splitlines()))
        loads = [i for i, s in enumerate(ins) if LOAD.match(s)]
        assert loads, f"{name}: no load into LDS"
        for i in loads:
            assert not re.match(r"^s_\w+ m0,", ins[i - 1]), \
                f"{name}: {ins[i - 1]!r} right before {ins[i]!r}"
        for i, s in enumerate(ins):
            if s == "s_endpgm":
                before = [j for j in loads if j < i]
                if before:
                    waits = [x for x in ins[before[-1]:i] if re.match(r"^s_waitcnt .*vmcnt\(0\)", x)]
                    assert waits, f"{name}: a load in flight at the end of the program"
