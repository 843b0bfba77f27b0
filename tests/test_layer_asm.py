"""The gfx950 assembly of the layer for a few tokens, checked on the host (no GPU).

Its second product's blocks hand their sums to each other, perhaps across XCDs: stores
and loads of agent scope (sc1), which pass the L2 by, and one relaxed add a tile. What
orders them is a wait for the stores written out in an asm statement, then a barrier,
then the add: the compiler is told of no order between them. Checked for every kernel
of the second product: sums are stored and loaded with sc1, and each add has the barrier
ahead of it and the wait ahead of that, with no such store in between.
"""
import os
import re

from combine_ep_prepare_amd import _build
from test_experts_asm import _kernels
from test_kernel_asm import _device_asm

STORE = re.compile(r"^global_store_\S+ .*\bsc1\b")
LOAD = re.compile(r"^global_load_\S+ .*\bsc1\b")
ADD = re.compile(r"^global_atomic_add")


def marked(body):
    """The instructions, a wait out of an asm statement as WAIT."""
    in_asm = False
    for line in body.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            in_asm = "#ASMSTART" in line
            continue
        s = line.split(";")[0].strip()
        if not s or s.endswith(":") or s.startswith("."):
            continue
        yield "WAIT" if in_asm and s == "s_waitcnt vmcnt(0)" else s


def check(ins):
    """What is amiss with the order of the adds, in the order of the program's text:
    the loop's add comes ahead of its stores there, and its wait is at the loop's top."""
    adds = [i for i, s in enumerate(ins) if ADD.match(s)]
    if len(adds) != 2:
        return f"{len(adds)} adds"
    for i in adds:
        waits = [j for j in range(i) if ins[j] == "WAIT"]
        if not waits or "s_barrier" not in ins[waits[-1]:i]:
            return f"no wait and barrier ahead of {ins[i]!r}"
        if any(STORE.match(s) for s in ins[waits[-1]:i]):
            return f"a store between the wait and {ins[i]!r}"
    if not any(STORE.match(s) for s in ins[adds[0]:adds[1]]):
        return "no store between the loop's add and the last one"
    return None


def test_sums_between_blocks(tmp_path):
    text = "\n".join(_device_asm(os.path.join(_build.CSRC, "ep_layer.hip"), str(tmp_path)))
    kernels = [(n, b) for n, b in _kernels(text, "layer_kernel") if "ELb0E" in n]
    assert len(kernels) == 6
    for name, body in kernels:
        ins = list(marked(body))
        assert check(ins) is None, f"{name}: {check(ins)}"
        assert sum(bool(STORE.match(s)) for s in ins) >= 2, name
        assert sum(bool(LOAD.match(s)) for s in ins) >= 4, name   # in the loop and after it


def test_the_check_itself():
    good = ["WAIT", "s_barrier", "global_atomic_add v0, v1, v2, s[0:1] sc0",
            "global_store_dwordx2 v[0:1], v[2:3], off sc1", "s_barrier", "WAIT", "s_barrier",
            "global_atomic_add v0, v1, v2, s[0:1] sc0"]
    assert check(good) is None
    for i in range(len(good)):
        if i != 4:
            assert check(good[:i] + good[i + 1:]) is not None, good[i]
