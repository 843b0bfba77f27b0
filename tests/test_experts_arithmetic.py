"""The row arithmetic of the experts' kernels next to 2^31 rows, where a layout
ends (no GPU): the helpers of ep_experts.h, compiled for the host."""
import os
import subprocess

from combine_ep_prepare_amd import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "ep_experts.h"
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    const int32_t n = (int32_t)std::strtoll(argv[i + 1], nullptr, 10);
    const long long m = std::strtoll(argv[i + 2], nullptr, 10);
    std::printf("%d\n", argv[i][0] == 'p' ? epmi::pieces(n, (int32_t)m)
                                          : epmi::rest_after(n, (uint32_t)m));
  }
}
"""


def test_pieces_and_rest(tmp_path):
    source, program = tmp_path / "arithmetic.hip", tmp_path / "arithmetic"
    source.write_text(PROGRAM)
    subprocess.run([_build.hipcc(), "-std=c++17", f"--offload-arch={_build.ARCH}",
                    "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, "-o",
                    str(program), str(source)], check=True, capture_output=True)
    top = 2 ** 31 - 1
    sizes = (16, 32, 64, 128, 256)
    cuts = [(n, m) for n in (0, 1, 63, 64, 65, 1000, top - 256, top - 63, top - 1, top)
            for m in sizes]
    # a step's first value, up to two steps past the last one
    starts = [(n, at) for n, m in cuts for at in (-(-n // m) * m, (-(-n // m) + 1) * m)]
    args = [str(v) for what, pairs in (("p", cuts), ("l", starts)) for pair in pairs
            for v in (what, *pair)]
    out = subprocess.run([str(program), *args], check=True, capture_output=True, text=True)
    assert [int(v) for v in out.stdout.split()] == \
        [-(-n // m) for n, m in cuts] + [n - at for n, at in starts]
